// Products of NVFP4 tokens and NVFP4 weights on the block-scaled tensor cores.
//
//   Y[t][r] = cast( gx[t] * gw[m] * sum_j vx[t][j] vw[m][r][j] sum_{i in block j} qx[t][i] qw[m][r][i] )
//
// for the tokens t of group m (one matrix per group: the experts of a bank, or one
// matrix and all tokens), with E2M1 values q, E4M3 block scales v and FP32 global
// scales g: W4A4 inference with the weights that lh_quantize_nvfp4 exports.
//
// Two kernels, both with one warp-specialised CTA per SM: pairs of CTAs that walk over tiles of
// 256 channels x up to 256 tokens, and, for few tiles of few tokens, clusters of CTAs that
// share the columns of one tile. Warp 0 fills a ring of stages by TMA (128 bytes = 256 values
// of each row, and the scale tiles of those columns), warp 1 copies the scales to TMEM and
// issues tcgen05.mma kind::mxf4nvf4 (K = 64 a step), the others read the accumulators and
// store. Channels are the M side, so the N side, the tokens, can be cut to the 16
// rows that a ragged group's last tile needs.
#include <climits>
#include <mutex>
#include <type_traits>

#include <cudaTypedefs.h>

#include "common.cuh"
#include "scale_tiles.cuh"
#include "tcgen05.cuh"
#include "token_block.cuh"
#include "tokens.cuh"

namespace lh {
namespace {

using namespace tc;

constexpr int kM = 128;            // channels of a tile
constexpr int kStageK = 256;       // columns of a stage: 128 bytes of E2M1 pairs
constexpr int kRowBytes = kStageK / 2;
constexpr int kThreads = 192;      // producer, MMA, four epilogue warps

// Set by an expired wait; read and cleared by lh_nvfp4_status.
__device__ unsigned int product_status;

struct ProdArgs {
    const int64_t* offsets;  // groups of tokens, or null: one group of all
    int64_t G, n_rows, c_out, ld_y;
    int mtiles;              // channel tiles per matrix (of 128, or of 256 for CTA pairs)
    int mtiles128;           // rows of scale tiles per matrix
    int stages_k;            // stages along c_in
    int steps;               // 64-column steps along c_in
    int box;                 // tokens of one TMA copy: a tile of a pair brings the rows it has, rounded up to these
    const uint8_t* xs;       // scale tiles of the tokens
    const uint8_t* ws;       // scale tiles of the weights
    const float* xg;         // [n_rows]
    const float* wg;         // [G]
    void* Y;
    const void* X;           // the tokens themselves (from_tokens), [n_rows][ld_x], and their given amax or null
    int64_t ld_x;
    const float* gamax;
    int J;
    bool wide_x;
    bool early;              // the kernel before leaves weights, scales and offsets alone: no need to wait for those
};

constexpr int kT = 128;            // tokens of a tile: one scale tile

struct Shape {
    static constexpr int kA = kM * kRowBytes, kB = kT * kRowBytes, kSa = 4 * kTileBytes, kSb = 4 * kTileBytes;
    static constexpr int kStageBytes = kA + kB + kSa + kSb;
    static constexpr int kStages = 6;
    // TMEM: the accumulator, then the scales of two stages (addresses of scales are
    // multiples of 4 columns, so a tile starts with a scale tile)
    static constexpr int kScaleCol = kT, kSetCols = 32, kTmemCols = 512;  // all
    static_assert(kScaleCol + 2 * kSetCols <= kTmemCols, "TMEM columns");
    static_assert(kStages * kStageBytes >= 2 * kT * kM * 4, "split: the partial sums reuse the ring");
};

constexpr int kFewTokens = 4;  // most tokens that the product quantises itself

struct Control {
    uint32_t amax[4][kFewTokens];  // of the tokens, by warp
    float gscale[kFewTokens];
    uint64_t full[Shape::kStages], empty[Shape::kStages], tfull, done, sums;
    uint32_t tmem;
    int abort_flag;
};

struct Tile {
    int64_t g, lo, row0;
    int rows, mt, sub;  // rows left in the group from row0 (at most T); sub: row0 - lo
};

// Walks over the tiles of all groups in order; every warp of the CTA does so by itself.
// Groups are looked at 32 at a time, one per lane.
struct Walk {
    int T;  // tokens of a tile
    int64_t g = 0;
    int64_t base = 0;  // tiles before group g
    __device__ void range(const ProdArgs& p, int64_t i, int64_t& lo, int64_t& hi) const {
        lo = __ldg(p.offsets + i);
        hi = __ldg(p.offsets + i + 1);
        lo = lo < 0 ? 0 : (lo > p.n_rows ? p.n_rows : lo);
        hi = hi < 0 ? 0 : (hi > p.n_rows ? p.n_rows : hi);
    }
    __device__ bool find(const ProdArgs& p, int64_t u, Tile& t) {
        if (!p.offsets) {
            const uint32_t tt = (uint32_t)u / (uint32_t)p.mtiles;
            t.g = t.lo = 0;
            t.mt = (int)((uint32_t)u - tt * p.mtiles);
            t.row0 = (int64_t)tt * T;
            t.sub = (int)t.row0;
            t.rows = p.n_rows - t.row0 < T ? (int)(p.n_rows - t.row0) : T;
            return t.row0 < p.n_rows;
        }
        const int lane = threadIdx.x & 31;
        while (g < p.G) {
            int64_t lo = 0, hi = 0;
            if (g + lane < p.G) range(p, g + lane, lo, hi);
            // sums stop at 2^32 - 1: groups that overlap (decreasing offsets) can have more tiles
            uint32_t inc = hi > lo ? ((uint32_t)(hi - lo + T - 1) / (uint32_t)T) * p.mtiles : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
                if (lane >= o) inc = inc + v < v ? 0xFFFFFFFFu : inc + v;
            }
            const uint32_t hit = __ballot_sync(0xFFFFFFFFu, base + inc > u);
            if (hit) {
                const int l = __ffs(hit) - 1;
                const uint32_t before = __shfl_sync(0xFFFFFFFFu, inc, l ? l - 1 : 0);
                base += l ? before : 0;
                g += l;
                lo = __shfl_sync(0xFFFFFFFFu, lo, l);
                hi = __shfl_sync(0xFFFFFFFFu, hi, l);
                const int i = (int)(u - base);
                const int tt = i / p.mtiles;
                t.g = g;
                t.lo = lo;
                t.mt = i - tt * p.mtiles;
                t.row0 = lo + (int64_t)tt * T;
                t.sub = (int)(t.row0 - lo);
                t.rows = hi - t.row0 < T ? (int)(hi - t.row0) : T;
                return true;
            }
            base += __shfl_sync(0xFFFFFFFFu, inc, 31);
            g += 32;
        }
        return false;
    }
};

// Waits for the phase of `parity`; false after `limit` (1 s), or when another warp gave up. The timer
// is read only after many tries: reading it takes longer than most waits.
__device__ __forceinline__ bool lane_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                          uint64_t limit = kTimeoutNs) {
    uint64_t t0 = 0;
    for (uint32_t it = 1; !mbar_try(bar, parity); ++it) {
        if ((it & 255) != 0) continue;
        const uint64_t now = global_ns();
        if (t0 == 0) t0 = now;
        if (*abort_flag || now - t0 > limit) return false;
    }
    return true;
}
// The same with one answer for the warp.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    return __all_sync(0xFFFFFFFFu, lane_wait(bar, parity, abort_flag));
}
__device__ __forceinline__ void give_up(volatile int* flag) {
    *flag = 1;
    atomicExch(&product_status, (unsigned)LH_ERR_TIMEOUT);
}

// That wait and its report on a barrier that nothing arrives on (arrive == 0), or that is completed first.
__global__ void product_wait_kernel(uint64_t limit, int arrive) {
    __shared__ uint64_t bar;
    __shared__ int abort_flag;
    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&bar), 1);
        abort_flag = 0;
        mbar_init_fence();
    }
    __syncthreads();
    if (arrive && threadIdx.x == 0) mbar_arrive(smem_u32(&bar));
    if (!__all_sync(0xFFFFFFFFu, lane_wait(smem_u32(&bar), 0, &abort_flag, limit))) give_up(&abort_flag);
}

__device__ __forceinline__ void store_out(float* y, float v) { *y = v; }
__device__ __forceinline__ void store_out(__nv_bfloat16* y, float v) { *y = __float2bfloat16_rn(v); }

// A warp's part of a finished tile: 32 channels (its TMEM lanes) x up to 128 tokens, into
// registers and from there to Y. Row-major Y wants a token's channels side by side. In f32
// a lane per channel does that (128 bytes a store). In bf16 the values are taken in the
// layout of mma fragments and turned by stmatrix through shared memory, 32 tokens at a time,
// in rows of 128 bytes that two warps with neighbouring channels share (their 16-byte pieces
// swapped as TMA's 128-byte swizzle does, which keeps both ways free of bank conflicts).
// One TMA store takes each turn to Y, while the next is written to the other half of the buffer if
// it holds two (kTurns); what is less than 32 tokens of 64 channels, where a group or the
// channels end, is stored by the lanes, 8 channels each (a TMA store writes past the end of
// an odd row: its bounds are not those of single elements).
constexpr int kTurnRow = 128, kTurnBytes = 32 * kTurnRow;

template <typename Tout>
struct Part;

template <>
struct Part<float> {
    uint32_t r[4][32];
    __device__ void take(uint32_t src, int n) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (32 * j < n) tmem_ld32(src + 32 * j, r[j]);
#pragma unroll
        for (int j = 0; j < 4; ++j) tmem_wait32(r[j]);
    }
    // gx[j]: this lane's token 32 j + lane; y: the first token's row, number `row`; ch0: the warp's first channel
    template <int kTurns>
    __device__ void put(const float (&gx)[4], int n, float* y, int64_t ld, int64_t ch0, int64_t c_out, uint8_t*, uint32_t&,
                        const CUtensorMap*, int) {
        const int64_t ch = ch0 + (threadIdx.x & 31);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (32 * j >= n) break;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const float s = __shfl_sync(0xFFFFFFFFu, gx[j], i);
                if (32 * j + i < n && ch < c_out) y[(int64_t)(32 * j + i) * ld + ch] = __uint_as_float(r[j][i]) * s;
            }
        }
    }
};

template <>
struct Part<__nv_bfloat16> {
    uint32_t r[4][32];  // [2 (token / 64) + lane / 16]
    __device__ void take(uint32_t src, int n) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (64 * (j >> 1) < n) tmem_ld16x64(src + 64 * (j >> 1) + ((uint32_t)(16 * (j & 1)) << 16), r[j]);
#pragma unroll
        for (int j = 0; j < 4; ++j) tmem_wait32(r[j]);
    }
    __device__ static uint32_t pack(uint32_t lo, float sl, uint32_t hi, float sh) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(lo) * sl, __uint_as_float(hi) * sh);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    // turn: the buffer of two warps; half: which half of it comes next
    template <int kTurns>
    __device__ void put(const float (&gx)[4], int n, __nv_bfloat16* y, int64_t ld, int64_t ch0, int64_t c_out,
                        uint8_t* turn, uint32_t& half, const CUtensorMap* ymap, int row) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int p0 = (warp & 1) * 4;  // the warp's first piece of a row
        const uint32_t dst = smem_u32(turn) + (lane & 7) * kTurnRow + (((p0 + (lane >> 3)) ^ (lane & 7)) << 4);
        const int64_t ch = ch0 + 8 * (lane & 3);
#pragma unroll
        for (int c = 0; c < 4; ++c) {  // 32 tokens
            if (32 * c >= n) break;
            const uint32_t at = kTurns == 2 ? half * kTurnBytes : 0;
            const bool leads = (warp & 1) == 0;
            if constexpr (kTurns == 1) {
                if (leads && elect_one()) tma_store_read<0>();
                asm volatile("bar.sync %0, 64;" ::"r"(warp >> 1) : "memory");
            }
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // 8 tokens
                const float s0 = __shfl_sync(0xFFFFFFFFu, gx[c], 8 * j + 2 * (lane & 3));
                const float s1 = __shfl_sync(0xFFFFFFFFu, gx[c], 8 * j + 2 * (lane & 3) + 1);
                const uint32_t* a = r[2 * (c >> 1)] + 16 * (c & 1) + 4 * j;
                const uint32_t* b = r[2 * (c >> 1) + 1] + 16 * (c & 1) + 4 * j;
                stmatrix4_trans(dst + at + 8 * j * kTurnRow, pack(a[0], s0, a[1], s1), pack(a[2], s0, a[3], s1),
                                pack(b[0], s0, b[1], s1), pack(b[2], s0, b[3], s1));
            }
            const bool whole = 32 * c + 32 <= n && ch0 - 8 * p0 + 64 <= c_out;
            fence_proxy_async();
            if (kTurns == 2 && leads && elect_one()) tma_store_read<0>();  // the other half is free from here on
            asm volatile("bar.sync %0, 64;" ::"r"(warp >> 1) : "memory");
            if (whole && leads && elect_one())
                tma_store_2d(ymap, (int)ch0, row + 32 * c, smem_u32(turn) + at);
            half ^= 1;
            if (whole) continue;
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int i = 8 * q + (lane >> 2);
                const uint4 v = *reinterpret_cast<const uint4*>(turn + at + i * kTurnRow + (((p0 + (lane & 3)) ^ (i & 7)) << 4));
                if (32 * c + i >= n) continue;
                __nv_bfloat16* to = y + (int64_t)(32 * c + i) * ld + ch;
                if (ch + 8 <= c_out) {
                    *reinterpret_cast<uint4*>(to) = v;
                } else {
                    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (ch + e < c_out) to[e] = __ushort_as_bfloat16((uint16_t)(u[e >> 1] >> (16 * (e & 1))));
                }
            }
        }
    }
};

// The tokens of a fused product (at most kFewTokens, by four warps): their global scales,
// and the stages ks0 .. ks1 of their codes, in the 128-byte swizzle that the products read
// (the 16-byte pieces of a row swapped by the row's number), with the scale tiles.
template <typename Tin>
__device__ void write_tokens(const ProdArgs& p, Control& C, uint32_t ring, int ks0, int ks1, volatile int* abort_flag) {
    using S = Shape;
    const int th = threadIdx.x - 64, warp = th >> 5, lane = th & 31;
    const int n = (int)p.n_rows;
    const Tin* X = static_cast<const Tin*>(p.X);
    Held<Tin> h;
    for (int r = 0; r < n; ++r) {
        uint32_t m = 0;
        for (int j = th; j < p.J; j += 128) {
            h.load(X + r * p.ld_x + 16 * (int64_t)j, p.wide_x);
            m = max(m, h.max_bits());
        }
        m = __reduce_max_sync(0xFFFFFFFFu, m);
        if (lane == 0) C.amax[warp][r] = m;
    }
    asm volatile("bar.sync 1, 128;" ::: "memory");
    const int r = th >> 4, jj = th & 15;  // a thread per block of a stage
    const bool mine = r < n;
    uint32_t m = 0;
    if (mine) m = max(max(C.amax[0][r], C.amax[1][r]), max(C.amax[2][r], C.amax[3][r]));
    const bool bad = m >= 0x7F800000u;
    const RowScale rs(p.gamax ? __ldg(p.gamax) : __uint_as_float(m));
    if (mine && jj == 0) C.gscale[r] = bad ? rs.nan : rs.g;
    int stage = 0;
    uint32_t phase = 0;
    for (int ks = ks0; ks < ks1; ++ks) {
        const int j = 16 * ks + jj;
        uint32_t code = 0, word[2] = {0u, 0u};
        if (mine && j < p.J) {  // blocks past c_in: zeros
            float o[16];
            h.load(X + r * p.ld_x + 16 * (int64_t)j, p.wide_x);
            code = quantize_held<false, true>(h, h.max_bits(), rs, bad && !p.gamax, o, word);
        }
        if (!warp_wait(smem_u32(&C.empty[stage]), phase ^ 1, abort_flag)) {
            give_up(abort_flag);
            break;
        }
        if (mine) {
            const uint32_t b = ring + stage * S::kStageBytes + S::kA, sb = b + S::kB + S::kSa;
            asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(b + r * kRowBytes + ((((jj >> 1) ^ r) & 7) << 4) + (jj & 1) * 8),
                         "r"(word[0]), "r"(word[1])
                         : "memory");
            asm volatile("st.shared.u8 [%0], %1;" ::"r"(sb + (jj >> 2) * kTileBytes + r * 16 + (jj & 3)), "r"(code) : "memory");
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&C.full[stage]));
        if (++stage == S::kStages) { stage = 0; phase ^= 1; }
    }
    asm volatile("bar.sync 1, 128;" ::: "memory");  // the scales are there for all
}

// ---------------------------------------------------------------- few tiles of few tokens
//
// A cluster of CTAs works on one tile of 128 channels and all tokens (at most 128), each on
// a part of c_in; the partial sums meet in distributed shared memory, each CTA adding up
// those of its share of the tokens in the order of the parts (the same sums every time).
//
// Tin: with few tokens of type Tin instead of quantised ones, every CTA
// quantises its part of them: the epilogue warps, idle until the sums are ready, take each
// token's largest |x| and write the codes and scales of a stage where TMA would put them,
// while the weights are on their way, in one launch instead of two.
template <typename Tout, typename Tin = void>
__global__ void __launch_bounds__(kThreads, 1) product_split_kernel(const __grid_constant__ CUtensorMap wmap,
                                                                    const __grid_constant__ CUtensorMap xmap,
                                                                    const __grid_constant__ CUtensorMap wsmap,
                                                                    const __grid_constant__ CUtensorMap xsmap,
                                                                    const ProdArgs p) {
    using S = Shape;
    constexpr bool kFused = !std::is_void_v<Tin>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base_p = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Control& C = *reinterpret_cast<Control*>(base_p + S::kStages * S::kStageBytes);
    const uint32_t ring = smem_u32(base_p);
    volatile int* abort_flag = &C.abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int parts = (int)cluster_size(), rank = (int)cluster_rank();
    const int mt = blockIdx.x / parts, rows = (int)p.n_rows;
    const int ks0 = p.stages_k * rank / parts, ks1 = p.stages_k * (rank + 1) / parts;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(smem_u32(&C.full[s]), kFused ? 5 : 1);  // TMA, and the warps that quantise
            mbar_init(smem_u32(&C.empty[s]), 1);
        }
        mbar_init(smem_u32(&C.tfull), 1);
        mbar_init(smem_u32(&C.done), 1);
        mbar_init(smem_u32(&C.sums), 1);
        C.abort_flag = 0;
        mbar_init_fence();
    }
    if (warp == 1) tmem_alloc(smem_u32(&C.tmem), S::kTmemCols);  // all columns: they begin at 0
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = C.tmem;
    // everything above overlaps the kernel before
    if (!p.early) asm volatile("griddepcontrol.wait;" ::: "memory");

    if (warp == 0) {
        int n = 0;  // stages on their way
        bool ok = true;
        if (elect_one()) {  // one lane for all of them
            const uint32_t bytes = S::kA + S::kSa + (kFused ? 0 : p.box * kRowBytes + S::kSb);
            auto weights = [&](int s, int ks) {
                const uint32_t bar = smem_u32(&C.full[s]), a = ring + s * S::kStageBytes;
                mbar_expect_tx(bar, bytes);
                tma_load_2d(a, &wmap, ks * kRowBytes, mt * kM, bar);
                // past the last step this brings other scales, or zeros, that no product uses
                tma_load_2d(a + S::kA + S::kB, &wsmap, 0, mt * p.steps + 4 * ks, bar);
            };
            int ahead = 0;  // stages whose weights are on their way
            if (p.early) {
                for (; ahead < ks1 - ks0 && ahead < S::kStages; ++ahead) weights(ahead, ks0 + ahead);
                asm volatile("griddepcontrol.wait;" ::: "memory");
            }
            int st = 0;
            uint32_t ph = 0;
            for (int ks = ks0; ks < ks1; ++ks, ++n) {
                ok = lane_wait(smem_u32(&C.empty[st]), ph ^ 1, abort_flag);
                if (!ok) break;
                if (n >= ahead) weights(st, ks);
                if constexpr (!kFused) {
                    const uint32_t bar = smem_u32(&C.full[st]), b = ring + st * S::kStageBytes + S::kA;
                    tma_load_2d(b, &xmap, ks * kRowBytes, 0, bar);
                    tma_load_2d(b + S::kB + S::kSa, &xsmap, 0, 4 * ks, bar);
                }
                if (++st == S::kStages) { st = 0; ph ^= 1; }
            }
            // the products' last arrivals on the ring come before the CTA ends
            for (int i = n < S::kStages ? 0 : n - S::kStages; ok && i < n; ++i)
                ok = lane_wait(smem_u32(&C.empty[i % S::kStages]), (i / S::kStages) & 1, abort_flag);
        }
        ok = __all_sync(0xFFFFFFFFu, ok);
        n = __reduce_max_sync(0xFFFFFFFFu, n);
        if (!ok) {  // the loads in flight land before the CTA ends
            give_up(abort_flag);
            for (int i = n < S::kStages ? 0 : n - S::kStages; i < n; ++i) {
                int none = 0;
                warp_wait(smem_u32(&C.full[i % S::kStages]), (i / S::kStages) & 1, &none);
            }
        }
    } else if (warp == 1) {
        // the bounded waits below begin when the tokens are there, not while they are quantised
        if (p.early) asm volatile("griddepcontrol.wait;" ::: "memory");
        bool ok = true;
        const uint64_t desc_a = desc_k_sw128(ring), desc_b = desc_k_sw128(ring + S::kA);
        const uint64_t desc_sa = desc_scales(ring + S::kA + S::kB), desc_sb = desc_scales(ring + S::kA + S::kB + S::kSa);
        const uint32_t n16 = (rows + 15) & ~15;
        // E2M1 x E2M1, E4M3 scales, N = n16, M = 128
        const uint32_t idesc = (1u << 7) | (1u << 10) | ((n16 >> 3) << 17) | ((uint32_t)(kM >> 7) << 27);
        // One lane runs the whole row: its own instructions bound a short stage, and a choice
        // of lane and an answer for the warp at every stage would add a third to them.
        if (elect_one()) {
            bool ready = false;
            int st = 0;
            uint32_t ph = 0, set = 0;
            for (int ks = ks0; ks < ks1; ++ks) {
                if (!ready && !lane_wait(smem_u32(&C.full[st]), ph, abort_flag)) {
                    ok = false;
                    break;
                }
                fence_after();
                const int nk = p.steps - 4 * ks < 4 ? p.steps - 4 * ks : 4;
                const uint32_t at = st * (S::kStageBytes >> 4);  // addresses in descriptors count 16 bytes
                const uint32_t ca = S::kScaleCol + set * S::kSetCols, cb = ca + 16, bar = smem_u32(&C.empty[st]);
                if (++st == S::kStages) { st = 0; ph ^= 1; }
                set ^= 1;
                // a first look at the next stage, answered while this one's products are issued
                ready = mbar_test(smem_u32(&C.full[st]), ph);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (k >= nk) break;
                    tmem_cp_scales(cb + 4 * k, desc_sb + (at + k * (kTileBytes >> 4)));
                    tmem_cp_scales(ca + 4 * k, desc_sa + (at + k * (kTileBytes >> 4)));
                    mma_nvfp4(0, desc_a + (at + 2 * k), desc_b + (at + 2 * k), idesc, ca + 4 * k, cb + 4 * k,
                              (ks > ks0 || k > 0) ? 1u : 0u);
                }
                mma_commit(bar);
            }
            if (ok) mma_commit(smem_u32(&C.tfull));
        }
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (__any_sync(0xFFFFFFFFu, !ok || *abort_flag)) {  // the products in flight end before the CTA does
            give_up(abort_flag);
            if (elect_one()) mma_commit(smem_u32(&C.done));
            __syncwarp();
            int none = 0;
            warp_wait(smem_u32(&C.done), 0, &none);
        }
    } else {
        if (p.early) asm volatile("griddepcontrol.wait;" ::: "memory");
        if constexpr (kFused) write_tokens<Tin>(p, C, ring, ks0, ks1, abort_flag);
        if (!warp_wait(smem_u32(&C.tfull), 0, abort_flag)) give_up(abort_flag);
    }
    // The ring is idle once all its products are done. Its first 64 KB take
    // this CTA's sums, [token][channel], the next 64 KB those of the other parts for this
    // CTA's tokens, [part][token][channel], sent by bulk copies.
    const int per = (rows + parts - 1) / parts, q = warp & 3;
    float* mine = reinterpret_cast<float*>(base_p);
    float* theirs = mine + kT * kM;
    auto tokens_of = [&](int r) {  // how many of its tokens the tile has
        const int n = rows - r * per;
        return n < 0 ? 0 : (n < per ? n : per);
    };
    const int64_t row0 = rank * per;
    float gx[2] = {0.0f, 0.0f};  // of this CTA's tokens, one per lane (two parts: 64 tokens)
    if (warp >= 2) {
        const float gw = __ldg(p.wg);
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (32 * j + lane < tokens_of(rank)) {
                if constexpr (kFused) gx[j] = gw * C.gscale[rank * per + 32 * j + lane];
                else gx[j] = gw * __ldg(p.xg + row0 + 32 * j + lane);
            }
        fence_after();
        for (int c = 0; c < rows; c += 32) {
            uint32_t r[32];
            tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + c, r);
            tmem_wait32(r);
#pragma unroll
            for (int i = 0; i < 32; ++i) mine[(c + i) * kM + q * 32 + lane] = __uint_as_float(r[i]);
        }
        fence_proxy_async();
    }
    __syncthreads();
    cluster_meet();  // the rings of all parts are idle
    if (warp >= 2) {
        const uint32_t bar = smem_u32(&C.sums), got = (parts - 1) * tokens_of(rank) * kM * 4;
        if (warp == 2 && elect_one()) {
            if (got) mbar_expect_tx(bar, got);
            for (int r = 0; r < parts; ++r)
                if (r != rank && tokens_of(r) > 0)
                    bulk_copy_cluster(cluster_addr(smem_u32(theirs + rank * per * kM), r), smem_u32(mine + r * per * kM),
                                      tokens_of(r) * kM * 4, cluster_addr(bar, r));
        }
        __syncwarp();
        if (got && !warp_wait(bar, 0, abort_flag)) give_up(abort_flag);
        if (tokens_of(rank) > 0) {
            const int64_t ch = (int64_t)mt * kM + q * 32 + lane;
            Tout* y = static_cast<Tout*>(p.Y) + row0 * p.ld_y + ch;
            const int n = tokens_of(rank);
            for (int i0 = 0; i0 < n; i0 += 8) {  // the additions of eight tokens overlap
                float v[8] = {};
                for (int s = 0; s < parts; ++s) {
                    const float* part = s == rank ? mine + rank * per * kM : theirs + s * per * kM;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (i0 + i < n) v[i] += part[(i0 + i) * kM + q * 32 + lane];
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float g = __shfl_sync(0xFFFFFFFFu, i0 < 32 ? gx[0] : gx[1], (i0 + i) & 31);
                    if (i0 + i < n && ch < p.c_out) store_out(y + (int64_t)(i0 + i) * p.ld_y, v[i] * g);
                }
            }
        }
    }
    __syncwarp();
    cluster_meet();  // nothing is in flight from or to a CTA that ends
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 1) tmem_dealloc(tmem, S::kTmemCols);
}

// ---------------------------------------------------------------- CTA pairs
//
// Tiles of 256 channels x T tokens, one per pair of CTAs (cta_group::2): each CTA loads its
// own 128 channels and half of the tokens, so for T = 256 a stage brings 38 KB for 128 x 256 x
// 256 products where a tile of one CTA, 128 x 128, brings 36 KB for half of them. The scales
// of all tokens go to both CTAs. The accumulator takes 256 TMEM columns and the scales 96,
// which leaves no room for a second one: eight epilogue warps take a whole accumulator into
// registers and free it, some 570 clocks in all, before they scale and store beside the next
// tile's products. 8192 x 4096 -> 12288 takes 155 us (5.3 PFLOP/s, 81 % of four times the
// measured bf16 rate): a stage takes 520 to 640 clocks of which the products need 512.
// T = 128 leaves room for seven stages instead of five and suits few or small tiles; a
// stage takes 480 clocks there, the issuing lane's own instructions.

constexpr int kPairWarps = 8;      // of the epilogue
constexpr int kPairThreads = 64 + 32 * kPairWarps;  // producer, MMA, epilogue
constexpr int kPairRows = 160;     // rows per group from which tiles of 256 tokens are taken

template <int T>  // tokens of a tile: 256 or 128
struct Pair {
    static constexpr int kA = kM * kRowBytes, kB = T / 2 * kRowBytes, kSa = 4 * kTileBytes, kSb = T / kTileRows * 4 * kTileBytes;
    static constexpr int kStageBytes = kA + kB + kSa + kSb;
    static constexpr int kStages = T == 256 ? 5 : 7;
    static constexpr int kTurns = T == 256 ? 2 : 1;  // of each two epilogue warps
    static constexpr int kScaleCol = T, kSetCols = 16 + 32;
    static_assert(kScaleCol + 2 * kSetCols <= 512, "TMEM columns");
    static constexpr int kTurnTotal = kPairWarps / 2 * kTurns * kTurnBytes;
};

struct PairControl {
    uint64_t full[Pair<128>::kStages], empty[Pair<128>::kStages], tfull, tempty, done;
    uint32_t tmem;
    int abort_flag;
};

template <int T, typename Tout>
__global__ void __launch_bounds__(kPairThreads, 1)
    product_pair_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                        const __grid_constant__ CUtensorMap wsmap, const __grid_constant__ CUtensorMap xsmap,
                        const __grid_constant__ CUtensorMap ymap,
                        const ProdArgs p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base_p = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    using S = Pair<T>;
    uint8_t* turn_p = base_p + S::kStages * S::kStageBytes;  // the epilogue warps' rows
    PairControl& C = *reinterpret_cast<PairControl*>(turn_p + S::kTurnTotal);
    const uint32_t ring = smem_u32(base_p);
    volatile int* abort_flag = &C.abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int first = blockIdx.x >> 1, step = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(smem_u32(&C.full[s]), 1);
            mbar_init(smem_u32(&C.empty[s]), 1);
        }
        mbar_init(smem_u32(&C.tfull), 1);
        mbar_init(smem_u32(&C.tempty), 16);  // the epilogue warps of both CTAs
        mbar_init(smem_u32(&C.done), 1);
        C.abort_flag = 0;
        mbar_init_fence();
    }
    if (warp == 1) tmem_alloc_pair(smem_u32(&C.tmem), 512);  // all columns: they begin at 0
    fence_before();
    __syncthreads();
    cluster_meet();  // the barriers of both CTAs are ready
    fence_after();
    const uint32_t tmem = C.tmem;
    // everything above overlaps the kernel before
    if (!p.early) asm volatile("griddepcontrol.wait;" ::: "memory");

    Walk walk{T};
    Tile t;
    if (warp == 0) {
        int stage = 0, ahead = 0;  // ahead: stages whose weights are on their way
        uint32_t phase = 0;
        int64_t issued = 0;
        bool ok = true;
        for (int64_t u = first; ok && walk.find(p, u, t); u += step) {
            const int half = ((t.rows + 15) & ~15) / 2;  // tokens of each CTA
            const int boxes = (half + p.box - 1) / p.box;
            const bool two = T > kTileRows && t.rows > kTileRows;  // scale tiles
            const uint32_t bytes = 2 * (S::kA + boxes * p.box * kRowBytes + S::kSa + (two ? 2 : 1) * 4 * kTileBytes);  // both CTAs
            const int wrow = (int)(t.g * p.c_out + (int64_t)t.mt * 2 * kM + rank * kM);
            const int xrow = (int)t.row0 + (int)rank * half;
            const int wsrow = (int)((t.g * p.mtiles128 + t.mt * 2 + rank) * p.steps);
            const int xsrow = (int)((group_tile(t.lo, t.g) + t.sub / kTileRows) * p.steps);
            auto weights = [&](int s, int ks) {
                const uint32_t bar = cluster_addr(smem_u32(&C.full[s]), 0), a = ring + s * S::kStageBytes;
                if (rank == 0) mbar_expect_tx(smem_u32(&C.full[s]), bytes);
                tma_load_2d_pair(a, &wmap, ks * kRowBytes, wrow, bar);
                // past the last step or tile these bring other scales, or zeros, that no product uses
                tma_load_2d_pair(a + S::kA + S::kB, &wsmap, 0, wsrow + 4 * ks, bar);
            };
            if (p.early && u == first) {
                ahead = p.stages_k < S::kStages ? p.stages_k : S::kStages;
                if (elect_one())
                    for (int i = 0; i < ahead; ++i) weights(i, i);
                __syncwarp();
                asm volatile("griddepcontrol.wait;" ::: "memory");
            }
            int n = 0;           // stages of this tile
            if (elect_one()) {  // one lane for all of them
                int st = stage;
                uint32_t ph = phase;
                for (int ks = 0; ks < p.stages_k; ++ks, ++n) {
                    ok = lane_wait(smem_u32(&C.empty[st]), ph ^ 1, abort_flag);
                    if (!ok) break;
                    const uint32_t bar = cluster_addr(smem_u32(&C.full[st]), 0);
                    const uint32_t b = ring + st * S::kStageBytes + S::kA, sb = b + S::kB + S::kSa;
                    if (n >= ahead) weights(st, ks);
                    for (int i = 0; i < boxes; ++i)
                        tma_load_2d_pair(b + i * p.box * kRowBytes, &xmap, ks * kRowBytes, xrow + i * p.box, bar);
                    tma_load_2d_pair(sb, &xsmap, 0, xsrow + 4 * ks, bar);
                    if (two) tma_load_2d_pair(sb + 4 * kTileBytes, &xsmap, 0, xsrow + p.steps + 4 * ks, bar);
                    if (++st == S::kStages) { st = 0; ph ^= 1; }
                }
            }
            ok = __all_sync(0xFFFFFFFFu, ok);
            n = __reduce_max_sync(0xFFFFFFFFu, n);
            ahead = 0;
            issued += n;
            stage += n;
            phase ^= (stage / S::kStages) & 1;
            stage %= S::kStages;
        }
        const int last = issued < S::kStages ? (int)issued : S::kStages;
        if (ok && elect_one()) {  // the products' last arrivals on this CTA's ring come before it ends
            int st = stage;
            uint32_t ph = phase;
            for (int i = 0; ok && i < last; ++i) {
                if (--st < 0) { st = S::kStages - 1; ph ^= 1; }
                ok = lane_wait(smem_u32(&C.empty[st]), ph, abort_flag);
            }
        }
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) {  // the loads in flight land before the CTAs end (both report to the first one's barriers)
            give_up(abort_flag);
            const int n = rank == 0 ? last : 0;
            for (int i = 0; i < n; ++i) {
                if (--stage < 0) { stage = S::kStages - 1; phase ^= 1; }
                int none = 0;
                warp_wait(smem_u32(&C.full[stage]), phase, &none);
            }
            // the second CTA's may be of stages that the first never came to: no barrier here tells, so they get
            // 1 ms, a thousand times what a load takes
            if (rank != 0)
                for (const uint64_t t0 = global_ns(); global_ns() - t0 < 1000000;) {}
        }
    } else if (warp == 1) {
        if (rank == 0) {
            // the bounded waits below begin when the tokens are there, not while they are quantised
            if (p.early) asm volatile("griddepcontrol.wait;" ::: "memory");
            int stage = 0;
            uint32_t phase = 0, aphase = 0, set = 0;
            bool ok = true;
            const uint64_t desc_a = desc_k_sw128(ring), desc_b = desc_k_sw128(ring + S::kA);
            const uint64_t desc_sa = desc_scales(ring + S::kA + S::kB), desc_sb = desc_scales(ring + S::kA + S::kB + S::kSa);
            for (int64_t u = first; ok && walk.find(p, u, t); u += step) {
                ok = warp_wait(smem_u32(&C.tempty), aphase ^ 1, abort_flag);
                if (!ok) break;
                fence_after();
                const uint32_t n16 = (t.rows + 15) & ~15;
                const uint32_t idesc = (1u << 7) | (1u << 10) | ((n16 >> 3) << 17) | (2u << 27);  // M = 256
                const bool two = T > kTileRows && t.rows > kTileRows;
                if (elect_one()) {  // one lane runs the whole row, as above
                    bool ready = false;
                    int st = stage;
                    uint32_t ph = phase, se = set;
                    for (int ks = 0; ks < p.stages_k; ++ks) {
                        if (!ready && !lane_wait(smem_u32(&C.full[st]), ph, abort_flag)) {
                            ok = false;
                            break;
                        }
                        fence_after();
                        const int nk = p.steps - 4 * ks < 4 ? p.steps - 4 * ks : 4;
                        const uint32_t at = st * (S::kStageBytes >> 4);  // addresses in descriptors count 16 bytes
                        const uint32_t ca = S::kScaleCol + se * S::kSetCols, cb = ca + 16, bar = smem_u32(&C.empty[st]);
                        if (++st == S::kStages) { st = 0; ph ^= 1; }
                        se ^= 1;
                        ready = mbar_test(smem_u32(&C.full[st]), ph);
                        // step by step: the copies of a step run beside the products of the one before
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if (k >= nk) break;
                            tmem_cp_scales_pair(cb + 8 * k, desc_sb + (at + k * (kTileBytes >> 4)));
                            if (two)
                                tmem_cp_scales_pair(cb + 8 * k + 4, desc_sb + (at + (4 + k) * (kTileBytes >> 4)));
                            tmem_cp_scales_pair(ca + 4 * k, desc_sa + (at + k * (kTileBytes >> 4)));
                            mma_nvfp4_pair(0, desc_a + (at + 2 * k), desc_b + (at + 2 * k), idesc, ca + 4 * k, cb + 8 * k,
                                           (ks | k) ? 1u : 0u);
                        }
                        mma_commit_pair(bar);
                    }
                    if (ok) mma_commit_pair(smem_u32(&C.tfull));
                }
                ok = __all_sync(0xFFFFFFFFu, ok);
                stage += p.stages_k;
                phase ^= (stage / S::kStages) & 1;
                stage %= S::kStages;
                set ^= p.stages_k & 1;
                aphase ^= 1;
            }
            // the second CTA's last arrivals come before this one ends
            if (ok) ok = warp_wait(smem_u32(&C.tempty), aphase ^ 1, abort_flag);
            if (__any_sync(0xFFFFFFFFu, !ok || *abort_flag)) {  // the products in flight end before the CTAs do
                give_up(abort_flag);
                if (elect_one()) mma_commit_pair(smem_u32(&C.done));
                __syncwarp();
                int none = 0;
                warp_wait(smem_u32(&C.done), 0, &none);
            }
        }
    } else {
        const int q = warp & 3;           // the TMEM lanes that this warp can read
        const int h = (warp - 2) >> 2;    // its half of the tokens
        uint8_t* turn = turn_p + ((warp - 2) >> 1) * S::kTurns * kTurnBytes;
        uint32_t half = 0;
        if (p.early) asm volatile("griddepcontrol.wait;" ::: "memory");
        uint32_t aphase = 0;
        bool ok = true;
        for (int64_t u = first; ok && walk.find(p, u, t); u += step) {
            const int64_t ch0 = (int64_t)t.mt * 2 * kM + rank * kM + q * 32;
            const float gw = __ldg(p.wg + t.g);
            const int c0 = h * (T / 2);
            const int n = t.rows - c0 < T / 2 ? t.rows - c0 : T / 2;  // tokens of this warp, if above 0
            float gx[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                gx[j] = 32 * j + lane < n ? gw * __ldg(p.xg + t.row0 + c0 + 32 * j + lane) : 0.0f;
            ok = warp_wait(smem_u32(&C.tfull), aphase, abort_flag);
            if (!ok) break;
            fence_after();
            Part<Tout> part;
            part.take(tmem + ((uint32_t)(q * 32) << 16) + c0, n);
            fence_before();
            __syncwarp();
            // the values are in registers: no memory is handed over
            if (lane == 0) mbar_arrive_cluster(cluster_addr(smem_u32(&C.tempty), 0));
            aphase ^= 1;
            part.template put<S::kTurns>(gx, n, static_cast<Tout*>(p.Y) + (t.row0 + c0) * p.ld_y, p.ld_y, ch0, p.c_out, turn,
                                    half, &ymap, (int)t.row0 + c0);
        }
        if (!ok) give_up(abort_flag);
        tma_store_wait();
    }
    fence_before();
    __syncthreads();
    cluster_meet();  // nothing of the pair is in flight to either CTA
    fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::call_once(once, [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    return fn;
}

// Packed E2M1 rows as bytes: boxes of 128 bytes x `box_rows` rows, 128-byte swizzle.
bool make_map(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap* map, const uint8_t* p, int64_t rows,
              int64_t row_bytes, int box_rows) {
    const cuuint64_t dims[2] = {(cuuint64_t)row_bytes, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)row_bytes};
    const cuuint32_t box[2] = {(cuuint32_t)kRowBytes, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(p), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scale tiles as rows of 512 bytes: boxes of the four steps of a stage.
bool make_scale_map(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap* map, const uint8_t* p, int64_t tiles) {
    const cuuint64_t dims[2] = {kTileBytes / 4, (cuuint64_t)tiles};
    const cuuint64_t strides[1] = {kTileBytes};
    const cuuint32_t box[2] = {kTileBytes / 4, 4};
    const cuuint32_t estr[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<uint8_t*>(p), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Y in bf16: boxes of 64 channels x 32 tokens, 128-byte swizzle.
bool make_out_map(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap* map, const ProdArgs& p) {
    const cuuint64_t dims[2] = {(cuuint64_t)p.c_out, (cuuint64_t)p.n_rows};
    const cuuint64_t strides[1] = {(cuuint64_t)p.ld_y * 2};
    const cuuint32_t box[2] = {kTurnRow / 2, kTurnBytes / kTurnRow};
    const cuuint32_t estr[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p.Y, dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename Tout, typename Tin = void>
lh_status launch_split(PFN_cuTensorMapEncodeTiled_v12000 encode, const uint8_t* X, const uint8_t* W, int64_t c_in,
                       ProdArgs p, int parts, cudaStream_t st) {
    using S = Shape;
    const int64_t xs_tiles = (p.n_rows / kTileRows + 1) * p.steps, ws_tiles = (int64_t)p.mtiles * p.steps;
    if (xs_tiles > INT_MAX - 512 || ws_tiles > INT_MAX - 512) return fail(LH_ERR_UNSUPPORTED, "too many scale tiles");
    p.box = 16;  // the power of 2 that takes all tokens (a copy costs its rows, used or not, about 1.3 ns each)
    while (p.box < p.n_rows) p.box *= 2;
    CUtensorMap wmap, xmap, wsmap, xsmap;
    bool ok = make_map(encode, &wmap, W, p.c_out, c_in / 2, kM) && make_scale_map(encode, &wsmap, p.ws, ws_tiles);
    if constexpr (std::is_void_v<Tin>)
        ok = ok && make_map(encode, &xmap, X, p.n_rows, c_in / 2, p.box) && make_scale_map(encode, &xsmap, p.xs, xs_tiles);
    else
        xmap = wmap, xsmap = wsmap;  // not used
    if (!ok) return fail(LH_ERR_CUDA, "cuTensorMapEncodeTiled failed");
    constexpr size_t smem = (size_t)S::kStages * S::kStageBytes + 1024 + sizeof(Control);
    static_assert(smem <= 227 * 1024, "shared memory");
    auto kernel = product_split_kernel<Tout, Tin>;
    static std::atomic<uint64_t> done{0};
    lh_status s = allow_shared((const void*)kernel, smem, done);
    if (s != LH_OK) return s;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.mtiles * parts));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)parts;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, wmap, xmap, wsmap, xsmap, p), "product_split_kernel launch");
}

int64_t pair_tiles(const ProdArgs& p, int T) {  // at most
    return (p.offsets ? p.n_rows / T + p.G : (p.n_rows + T - 1) / T) * ((p.mtiles128 + 1) / 2);
}

template <int T, typename Tout>
lh_status launch_pair(PFN_cuTensorMapEncodeTiled_v12000 encode, const uint8_t* X, const uint8_t* W, int64_t c_in,
                      ProdArgs p, int sms, cudaStream_t st) {
    using S = Pair<T>;
    p.mtiles = (p.mtiles128 + 1) / 2;
    // the power of 2 that takes half of a group of average size in one copy (a copy costs its
    // rows, used or not, about 1.3 ns each)
    p.box = 8;
    while (p.box < T / 2 && 2 * p.box * p.G < p.n_rows) p.box *= 2;
    const int64_t pairs = sms / 2, tiles = pair_tiles(p, T);
    const int64_t xs_tiles = (p.n_rows / kTileRows + p.G) * p.steps, ws_tiles = p.G * p.mtiles128 * p.steps;
    if (tiles > INT_MAX || xs_tiles > INT_MAX - 512 || ws_tiles > INT_MAX - 512)
        return fail(LH_ERR_UNSUPPORTED, "too many tiles");
    CUtensorMap wmap, xmap, wsmap, xsmap;
    if (!make_map(encode, &wmap, W, p.G * p.c_out, c_in / 2, kM) ||
        !make_map(encode, &xmap, X, p.n_rows, c_in / 2, p.box) ||
        !make_scale_map(encode, &wsmap, p.ws, ws_tiles) || !make_scale_map(encode, &xsmap, p.xs, xs_tiles))
        return fail(LH_ERR_CUDA, "cuTensorMapEncodeTiled failed");
    CUtensorMap ymap = wmap;  // f32: not used
    if (std::is_same_v<Tout, __nv_bfloat16> && !make_out_map(encode, &ymap, p))
        return fail(LH_ERR_CUDA, "cuTensorMapEncodeTiled failed");
    constexpr size_t smem = (size_t)S::kStages * S::kStageBytes + S::kTurnTotal + 1024 + sizeof(PairControl);
    static_assert(smem <= 227 * 1024, "shared memory");
    auto kernel = product_pair_kernel<T, Tout>;
    static std::atomic<uint64_t> done{0};
    lh_status s = allow_shared((const void*)kernel, smem, done);
    if (s != LH_OK) return s;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs)));
    cfg.blockDim = dim3(kPairThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, wmap, xmap, wsmap, xsmap, ymap, p), "product_pair_kernel launch");
}

// Parts of c_in for the tiles of one matrix and at most 128 tokens: as many as SMs allow, in
// cluster sizes that pack the GPCs (1 x 17408 -> 5120, 40 tiles: 12.6 us in two parts, 10.0 us
// in three).
int split_parts(const ProdArgs& p, int sms) {
    const int most = p.mtiles > 0 ? sms / p.mtiles : 1;
    for (const int parts : {8, 6, 4, 3, 2})
        if (parts <= most && parts <= p.stages_k) return parts;
    return 1;
}

// Which kernel. One matrix with tiles for at most half of the SMs: c_in split over clusters
// while that takes stages away from a row for at most four tokens each, since more tokens make
// the sums' way longer (4096 -> 4096, 12 of 16 stages: 32 tokens 5.9 us split and 6.8 us in
// pairs, 64 tokens 7.5 and 7.3 us; 17408 -> 5120, 45 of 68: 128 tokens 17.3 and 19.8 us). Else
// CTA pairs, with tiles of 256 tokens or, where these need more than 7/10 of the rounds of
// 128-token tiles or groups are small, of 128: 300 x 4096 -> 4096 8.1 us against 9.7 us. Of
// groups, whose sizes the host does not know, from 160 rows on average (64 experts 2048 -> 1536:
// 128 rows each 29.2 us in tiles of 128 and 30.0 us of 256, 192 rows 38.0 and 32.4 us).
template <typename Tout>
lh_status dispatch(PFN_cuTensorMapEncodeTiled_v12000 encode, const uint8_t* X, const uint8_t* W, int64_t c_in,
                   const ProdArgs& p, int sms, cudaStream_t st) {
    if (!p.offsets && p.n_rows <= kT) {
        const int parts = split_parts(p, sms), saved = p.stages_k - (p.stages_k + parts - 1) / parts;
        if (parts > 1 && p.n_rows <= (saved < 4 ? 16 : 4 * saved))
            return launch_split<Tout>(encode, X, W, c_in, p, parts, st);
    }
    const int64_t pairs = sms / 2;
    auto rounds = [&](int T) { return (pair_tiles(p, T) + pairs - 1) / pairs; };
    if (p.offsets ? p.n_rows < kPairRows * p.G : 7 * rounds(128) < 10 * rounds(256))
        return launch_pair<128, Tout>(encode, X, W, c_in, p, sms, st);
    return launch_pair<256, Tout>(encode, X, W, c_in, p, sms, st);
}

lh_status check_weights(const uint8_t* W_packed, const uint8_t* W_scales, const float* W_gscale, const int64_t* offsets,
                        int64_t n_groups, int64_t n_rows, int64_t c_out, int64_t c_in, const void* Y, lh_dtype out_dtype,
                        int64_t ld_y) {
    if (!valid_dtype(out_dtype)) return fail(LH_ERR_UNSUPPORTED, "out_dtype %d is not LH_BF16 or LH_F32", (int)out_dtype);
    if (n_rows < 0 || c_out < 0 || c_in < 0 || n_groups < 1)
        return fail(LH_ERR_INVALID_ARG, "sizes must be >= 0, n_groups >= 1");
    if (n_rows > 0 && c_out > 0 && (!W_packed || !W_scales || !W_gscale || !Y))
        return fail(LH_ERR_INVALID_ARG, "null pointer argument");
    if (!offsets && n_groups != 1) return fail(LH_ERR_INVALID_ARG, "several groups need offsets");
    if (c_in % 32 != 0 || c_in == 0)
        return fail(LH_ERR_UNSUPPORTED, "c_in=%lld is not a positive multiple of 32", (long long)c_in);
    // the tokens' limit: 2^20 stages of some 0.3 us, so that the wait for a tile stays well within its 1 s
    if (c_in > (1 << 28)) return fail(LH_ERR_UNSUPPORTED, "c_in must be at most 2^28");
    if (ld_y < c_out) return fail(LH_ERR_INVALID_ARG, "ld_y=%lld < c_out=%lld", (long long)ld_y, (long long)c_out);
    if (!aligned16(W_packed) || !aligned16(W_scales) || !aligned16(Y) || (ld_y * elem_bytes(out_dtype)) % 16 != 0)
        return fail(LH_ERR_ALIGNMENT, "W_packed, W_scales and Y must be 16-byte aligned, with 16-byte aligned rows of Y");
    // row and column coordinates of the TMA copies are 32-bit
    if (n_rows > INT_MAX - 512 || (c_out > 0 && n_groups > (INT_MAX - 512) / c_out))
        return fail(LH_ERR_UNSUPPORTED, "rows and n_groups * c_out must be below 2^31 - 512");
    return LH_OK;
}

}  // namespace
}  // namespace lh

namespace lh {
namespace {
ProdArgs product_args(const uint8_t* X_scales, const float* X_gscale, const uint8_t* W_scales, const float* W_gscale,
                      const int64_t* offsets, int64_t n_groups, int64_t n_rows, int64_t c_out, int64_t c_in, void* Y,
                      int64_t ld_y, bool early) {
    ProdArgs p = {};
    p.offsets = offsets; p.G = n_groups; p.n_rows = n_rows; p.c_out = c_out; p.ld_y = ld_y;
    p.mtiles = p.mtiles128 = (int)((c_out + kM - 1) / kM);
    p.stages_k = (int)((c_in + kStageK - 1) / kStageK);
    p.steps = (int)scale_steps(c_in);
    p.xs = X_scales; p.ws = W_scales; p.xg = X_gscale; p.wg = W_gscale; p.Y = Y; p.early = early;
    return p;
}

lh_status matmul(const uint8_t* X_packed, const uint8_t* X_scales, const float* X_gscale, const uint8_t* W_packed,
                 const uint8_t* W_scales, const float* W_gscale, const int64_t* offsets, int64_t n_groups,
                 int64_t n_rows, int64_t c_out, int64_t c_in, void* Y, lh_dtype out_dtype, int64_t ld_y, bool early,
                 void* stream) {
    clear_error();
    lh_status s = check_weights(W_packed, W_scales, W_gscale, offsets, n_groups, n_rows, c_out, c_in, Y, out_dtype, ld_y);
    if (s != LH_OK) return s;
    if (n_rows > 0 && c_out > 0 && (!X_packed || !X_scales || !X_gscale)) return fail(LH_ERR_INVALID_ARG, "null pointer argument");
    if (!aligned16(X_packed) || !aligned16(X_scales))
        return fail(LH_ERR_ALIGNMENT, "X_packed and X_scales must be 16-byte aligned");
    if (same_array(Y, X_packed) || same_array(Y, W_packed) || same_array(Y, X_scales) || same_array(Y, W_scales))
        return fail(LH_ERR_INVALID_ARG, "Y must not alias an input");
    if (n_rows == 0 || c_out == 0) return LH_OK;
    const int sms = sm_count();
    if (sms <= 0) return fail(LH_ERR_CUDA, "no CUDA device");
    auto encode = encode_fn();
    if (!encode) return fail(LH_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
    const ProdArgs p = product_args(X_scales, X_gscale, W_scales, W_gscale, offsets, n_groups, n_rows, c_out, c_in, Y,
                                    ld_y, early);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (out_dtype == LH_BF16) return dispatch<__nv_bfloat16>(encode, X_packed, W_packed, c_in, p, sms, st);
    return dispatch<float>(encode, X_packed, W_packed, c_in, p, sms, st);
}

// Whether the product takes the tokens themselves: one matrix in few tiles, and so little of
// them that every CTA can look at it all. From the tokens on, 1 x 4096 -> 4096 takes 6.5 us so
// and 6.4 us in two launches, 1 x 8192 -> 4096 7.8 and 8.0 us, 4 x 2048 -> 1536 5.9 and 6.0 us,
// with a launch less of the host's time each; 8 x 1024 -> 1024 takes 6.7 and 5.6 us,
// 4 x 4096 -> 4096 8.2 and 6.5 us.
bool can_fuse(const ProdArgs& p, int64_t c_in, const int32_t* rows, int sms) {
    return !rows && !p.offsets && p.n_rows <= kFewTokens && p.n_rows * c_in <= 8192 && split_parts(p, sms) > 1;
}

// The product of few tokens, from the tokens on. Arguments as lh_nvfp4_linear has checked them.
lh_status fused(ProdArgs p, const void* X, lh_dtype x_dtype, int64_t c_in, int64_t ld_x, const float* gamax,
                const uint8_t* W_packed, lh_dtype out_dtype, int sms, cudaStream_t st) {
    auto encode = encode_fn();
    if (!encode) return fail(LH_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
    p.X = X; p.ld_x = ld_x; p.gamax = gamax; p.J = (int)(c_in / 16);
    p.wide_x = (reinterpret_cast<uintptr_t>(X) & 31) == 0 && (ld_x * elem_bytes(x_dtype)) % 32 == 0;
    const int parts = split_parts(p, sms);
    if (x_dtype == LH_BF16)
        return out_dtype == LH_BF16
                   ? launch_split<__nv_bfloat16, uint16_t>(encode, nullptr, W_packed, c_in, p, parts, st)
                   : launch_split<float, uint16_t>(encode, nullptr, W_packed, c_in, p, parts, st);
    return out_dtype == LH_BF16
               ? launch_split<__nv_bfloat16, float>(encode, nullptr, W_packed, c_in, p, parts, st)
               : launch_split<float, float>(encode, nullptr, W_packed, c_in, p, parts, st);
}

}  // namespace
}  // namespace lh

extern "C" lh_status lh_nvfp4_matmul(const uint8_t* X_packed, const uint8_t* X_scales, const float* X_gscale,
                                     const uint8_t* W_packed, const uint8_t* W_scales, const float* W_gscale,
                                     const int64_t* offsets, int64_t n_groups, int64_t n_rows, int64_t c_out,
                                     int64_t c_in, void* Y, lh_dtype out_dtype, int64_t ld_y, void* stream) {
    return lh::matmul(X_packed, X_scales, X_gscale, W_packed, W_scales, W_gscale, offsets, n_groups, n_rows, c_out,
                      c_in, Y, out_dtype, ld_y, false, stream);
}

namespace lh {
namespace {
struct TokenWs {
    size_t packed, scales, gscale, total;
};
size_t up256(size_t b) { return (b + 255) & ~size_t(255); }
TokenWs token_ws(int64_t n_rows, int64_t c_in, int64_t n_groups) {
    TokenWs w;
    w.packed = 0;
    w.scales = up256((size_t)n_rows * (size_t)(c_in / 2));
    w.gscale = w.scales + up256(lh_nvfp4_token_scale_bytes(n_rows, c_in, n_groups));
    w.total = w.gscale + up256((size_t)n_rows * sizeof(float));
    return w;
}
}  // namespace
}  // namespace lh

extern "C" size_t lh_nvfp4_linear_workspace_bytes(int64_t n_rows, int64_t c_in, int64_t n_groups) {
    if (n_rows < 1 || n_groups < 1 || c_in < 32 || c_in % 32 != 0) return 0;
    return lh::token_ws(n_rows, c_in, n_groups).total;
}

extern "C" lh_status lh_nvfp4_linear(const void* X, lh_dtype x_dtype, int64_t n_src, int64_t c_in, int64_t ld_x,
                                     const int32_t* rows, int64_t row_div, int64_t n_rows, const int64_t* offsets,
                                     int64_t n_groups, const float* global_amax, const uint8_t* W_packed,
                                     const uint8_t* W_scales, const float* W_gscale, int64_t c_out, void* Y,
                                     lh_dtype out_dtype, int64_t ld_y, void* workspace, size_t workspace_bytes,
                                     void* stream) {
    using namespace lh;
    clear_error();
    lh_status s = check_weights(W_packed, W_scales, W_gscale, offsets, n_groups, n_rows, c_out, c_in, Y, out_dtype, ld_y);
    if (s != LH_OK) return s;
    if (same_array(Y, X) || same_array(Y, W_packed) || same_array(Y, W_scales) || same_array(Y, workspace))
        return fail(LH_ERR_INVALID_ARG, "Y must not alias an input or the workspace");
    const size_t need = lh_nvfp4_linear_workspace_bytes(n_rows, c_in, n_groups);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(LH_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need,
                    workspace ? workspace_bytes : (size_t)0);
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return fail(LH_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
    if (n_rows == 0 || c_out == 0) return LH_OK;
    const TokenWs w = token_ws(n_rows, c_in, n_groups);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    uint8_t* packed = ws + w.packed;
    uint8_t* scales = ws + w.scales;
    float* gscale = reinterpret_cast<float*>(ws + w.gscale);
    s = check_tokens(X, x_dtype, n_src, c_in, ld_x, rows, row_div, n_rows, offsets, n_groups, packed, scales, gscale,
                     nullptr, LH_F32);
    if (s != LH_OK) return s;
    const int sms = sm_count();
    if (sms <= 0) return fail(LH_ERR_CUDA, "no CUDA device");
    const ProdArgs few = product_args(nullptr, nullptr, W_scales, W_gscale, offsets, n_groups, n_rows, c_out, c_in, Y,
                                      ld_y, false);
    if (can_fuse(few, c_in, rows, sms))
        return fused(few, X, x_dtype, c_in, ld_x, global_amax, W_packed, out_dtype, sms,
                     reinterpret_cast<cudaStream_t>(stream));
    s = lh_quantize_tokens(X, x_dtype, n_src, c_in, ld_x, rows, row_div, n_rows, offsets, n_groups, global_amax, packed,
                           scales, gscale, nullptr, LH_F32, stream);
    if (s != LH_OK) return s;
    // the quantisation, if it ran, waited for everything before it and writes the workspace alone
    return matmul(packed, scales, gscale, W_packed, W_scales, W_gscale, offsets, n_groups, n_rows, c_out, c_in, Y,
                  out_dtype, ld_y, n_src > 0, stream);
}

extern "C" lh_status lh_debug_nvfp4_wait_timeout(int64_t timeout_us, int arrive, void* stream) {
    using namespace lh;
    clear_error();
    if (timeout_us < 1 || timeout_us > 1000000) return fail(LH_ERR_INVALID_ARG, "timeout_us must be in [1, 1e6]");
    if (sm_count() <= 0) return fail(LH_ERR_CUDA, "no CUDA device");
    product_wait_kernel<<<1, 32, 0, reinterpret_cast<cudaStream_t>(stream)>>>((uint64_t)timeout_us * 1000ull, arrive);
    return cuda_status(cudaGetLastError(), "product_wait_kernel launch");
}

extern "C" lh_status lh_nvfp4_status(void* stream) {
    using namespace lh;
    clear_error();
    void* word = nullptr;
    lh_status s = cuda_status(cudaGetSymbolAddress(&word, product_status), "cudaGetSymbolAddress");
    if (s != LH_OK) return s;
    unsigned int v = 0;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    s = cuda_status(cudaMemcpyAsync(&v, word, sizeof(v), cudaMemcpyDeviceToHost, st), "reading the product status");
    if (s == LH_OK) s = cuda_status(cudaStreamSynchronize(st), "cudaStreamSynchronize");
    if (s != LH_OK || v == 0) return s;
    s = cuda_status(cudaMemsetAsync(word, 0, sizeof(v), st), "clearing the product status");
    if (s != LH_OK) return s;
    return fail((lh_status)v, "a bounded wait inside the NVFP4 product gave up; its output is incomplete");
}
