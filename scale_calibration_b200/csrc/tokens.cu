// NVFP4 quantisation of tokens, and the scale tiles of exported weights.
//
// The two-level scale of "NVIDIA Model Optimizer Local-Hessian: 基于局部 Hessian 的
// NVFP4 逐块权重缩放算法实战指南" (xxmr.cn/news/266017), section "Local-Hessian 是什么",
// with max scaling (the pages' plain choice) applied to activations:
//   g   = fp32(amax / 2688)                     amax of the token, or of the tensor
//   v_b = E4M3_RNE_sat(fp32(fp32(amax_b / 6) / g)), at least code 1 (code 1 if g == 0)
//   q   = E2M1_RNE_sat(fp32(x / fp32(v_b g)))
// as lh_baseline_scales and lh_quantize_nvfp4 do for a matrix, in one pass over X.
#include <climits>

#include "scale_tiles.cuh"
#include "token_block.cuh"
#include "tokens.cuh"

namespace lh {
namespace {

// Blocks that a thread keeps in registers between the two passes (32 registers).
template <typename T>
constexpr int kHeld = 8 / (int)sizeof(T);

struct TokenArgs {
    int64_t n_src, ld;
    int n_rows, G, J, steps;
    uint32_t div_mul, div_shift;  // f / row_div = umulhi(f, div_mul) >> div_shift for f < 2^31; mul 0: row_div 1
    const int* rows;              // source of each row (over row_div), or null
    const int64_t* offsets;       // groups of rows, or null
    const float* gamax;           // amax of the tensor, or null (per token)
    bool wide_in, wide_out;       // rows of X, X_out 32-byte aligned
    uint8_t* packed;
    uint8_t* tiles;
    float* gscale;
};

// Largest group g with offsets[g] <= row, by the whole warp, 32 offsets a round; false
// when the row lies in no group.
__device__ __forceinline__ bool find_group(const TokenArgs& p, int row, int& g, int& lo) {
    g = 0;
    lo = 0;
    if (!p.offsets) return true;
    const int lane = threadIdx.x & 31;
    int span = p.G;  // offsets[g] <= row < offsets[g + span], if there is such a group
    while (span > 1) {
        const int step = (span + 31) >> 5;
        const bool le = lane * step < span && __ldg(p.offsets + g + lane * step) <= row;
        const uint32_t hit = __ballot_sync(0xFFFFFFFFu, le);
        const int l = hit ? 31 - __clz(hit) : 0;
        g += l * step;
        span = min(span - l * step, step);
    }
    const int64_t first = __ldg(p.offsets + g);
    lo = first < 0 ? 0 : (int)min(first, (int64_t)INT_MAX);
    return lo <= row && row < __ldg(p.offsets + g + 1);
}

__device__ __forceinline__ void store32(void* p, const uint32_t (&u)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]),
                 "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                 : "memory");
}
__device__ __forceinline__ void store16(uint16_t* p, const float (&o)[16], bool wide) {
    if (!wide) return Vec16<uint16_t>::store(p, o);
    uint32_t u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(o[2 * i], o[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    store32(p, u);
}
__device__ __forceinline__ void store16(float* p, const float (&o)[16], bool wide) {
    if (!wide) return Vec16<float>::store(p, o);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t u[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = __float_as_uint(o[8 * i + j]);
        store32(p + 8 * i, u);
    }
}

// kWarps warps per row. With the token's own scale each thread loads its blocks of the
// row and keeps them, the warps agree on the row's largest |x|, and the blocks are
// quantised from the registers; rows too wide for that are read twice (from L2). With a
// given scale one pass does.
// kGiven: the amax of the tensor is given.
template <typename Tin, typename Tout, bool kOut, bool kGiven, int kWarps>
__global__ void __launch_bounds__(256, sizeof(Tin) == 2 && !kOut ? 4 : 3)
    tokens_kernel(const Tin* __restrict__ X, TokenArgs p, Tout* __restrict__ out) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int kRows = 8 / kWarps;   // rows of a CTA
    constexpr int kSpan = 32 * kWarps;  // threads of a row
    constexpr int kN = kHeld<Tin>;
    __shared__ uint32_t red[kRows][kWarps];
    const int tid = threadIdx.x % kSpan, part = threadIdx.x / kSpan, warp = tid >> 5, lane = tid & 31;
    const int J = p.J;
    auto row_max = [&](uint32_t m) {
        m = __reduce_max_sync(0xFFFFFFFFu, m);
        if constexpr (kWarps > 1) {
            if (lane == 0) red[part][warp] = m;
            asm volatile("bar.sync %0, %1;" ::"r"(part + 1), "n"(kSpan) : "memory");
#pragma unroll
            for (int i = 0; i < kWarps; ++i) m = max(m, red[part][i]);
            asm volatile("bar.sync %0, %1;" ::"r"(part + 1), "n"(kSpan) : "memory");  // before the next row's
        }
        return m;
    };
    // unsigned: the step past the last of up to 2^31 - 513 rows would overflow an int
    for (uint32_t row = blockIdx.x * kRows + part; row < (uint32_t)p.n_rows; row += gridDim.x * kRows) {
        int g, lo;
        if (!find_group(p, (int)row, g, lo)) continue;
        int64_t src = row;
        if (p.rows) {
            const int f = __ldg(p.rows + row);
            src = f < 0 ? -1 : (int64_t)(p.div_mul ? __umulhi((uint32_t)f, p.div_mul) >> p.div_shift : (uint32_t)f);
        }
        if (src < 0 || src >= p.n_src) continue;
        const Tin* x = X + src * p.ld;
        Held<Tin> h[kN];
        uint32_t bb[kN], mb = 0;
        bool reload = true;
        if constexpr (!kGiven) {
            for (int j0 = tid; j0 - tid < J; j0 += kSpan * kN) {
#pragma unroll
                for (int i = 0; i < kN; ++i)
                    if (j0 + i * kSpan < J) h[i].load(x + 16 * (int64_t)(j0 + i * kSpan), p.wide_in);
#pragma unroll
                for (int i = 0; i < kN; ++i) {
                    bb[i] = j0 + i * kSpan < J ? h[i].max_bits() : 0;
                    mb = max(mb, bb[i]);
                }
            }
            mb = row_max(mb);
            reload = J > kSpan * kN;
        }
        const bool bad_token = mb >= 0x7F800000u;
        const RowScale rs(kGiven ? __ldg(p.gamax) : __uint_as_float(mb));
        const uint32_t r = row - lo, rt = r % kTileRows;
        uint8_t* tiles = p.tiles + (uint64_t)((uint32_t)lo / kTileRows + g + r / kTileRows) * ((uint32_t)p.steps * kTileBytes) +
                         (rt % 32) * 16 + rt / 32 * 4;
        const int64_t out0 = (int64_t)row * J;
        for (int j0 = tid; j0 - tid < 4 * p.steps; j0 += kSpan * kN) {
            if (reload) {
#pragma unroll
                for (int i = 0; i < kN; ++i)
                    if (j0 + i * kSpan < J) h[i].load(x + 16 * (int64_t)(j0 + i * kSpan), p.wide_in);
#pragma unroll
                for (int i = 0; i < kN; ++i) {
                    bb[i] = j0 + i * kSpan < J ? h[i].max_bits() : 0;
                    mb = max(mb, bb[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                const int j = j0 + i * kSpan;
                if (j - lane >= 4 * p.steps) break;  // the same for the warp
                uint32_t code = 0;
                if (j < J) {
                    float o[16];
                    uint32_t word[2];
                    code = quantize_held<kOut, kGiven>(h[i], bb[i], rs, bad_token, o, word);
                    reinterpret_cast<uint2*>(p.packed)[out0 + j] = make_uint2(word[0], word[1]);
                    if constexpr (kOut) store16(out + (out0 + j) * 16, o, p.wide_out);
                }
                // the four codes of a step, one word of the tile
                uint32_t v = code << (8 * (j & 3));
                v |= __shfl_xor_sync(0xFFFFFFFFu, v, 1);
                v |= __shfl_xor_sync(0xFFFFFFFFu, v, 2);
                if ((j & 3) == 0 && j < 4 * p.steps)
                    *reinterpret_cast<uint32_t*>(tiles + (int64_t)(j >> 2) * kTileBytes) = v;
            }
        }
        if constexpr (kGiven) mb = row_max(mb);
        if (tid == 0) p.gscale[row] = mb >= 0x7F800000u ? rs.nan : rs.g;
    }
}

// One thread per four scale bytes of a tile.
__global__ void __launch_bounds__(256) tile_scales_kernel(const uint8_t* __restrict__ scales, int64_t n_mats,
                                                          int64_t c_out, int64_t J, int64_t steps, int64_t row_tiles,
                                                          uint32_t* __restrict__ tiles) {
    const int64_t n = n_mats * row_tiles * steps * (kTileBytes / 4);
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
        const int w = (int)(i % (kTileBytes / 4));  // word of the tile: row w / 4 + 32 (w % 4)
        const int64_t t = i / (kTileBytes / 4);
        const int64_t k = t % steps, mt = t / steps;
        const int64_t m = mt / row_tiles, r = (mt - m * row_tiles) * kTileRows + (w >> 2) + 32 * (w & 3);
        uint32_t v = 0;
        if (r < c_out) {
            const uint8_t* s = scales + (m * c_out + r) * J;
#pragma unroll
            for (int b = 0; b < 4; ++b)
                if (4 * k + b < J) v |= (uint32_t)s[4 * k + b] << (8 * b);
        }
        tiles[i] = v;
    }
}

template <typename Tin, typename Tout, bool kOut, bool kGiven, int kWarps>
lh_status launch_tokens_w(const void* X, const TokenArgs& p, void* out, int sms, cudaStream_t st) {
    constexpr int kRows = 8 / kWarps;
    const int64_t need = (p.n_rows + kRows - 1) / kRows, cap = (int64_t)sms * 16;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(need < cap ? need : cap));
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, tokens_kernel<Tin, Tout, kOut, kGiven, kWarps>, (const Tin*)X, p, (Tout*)out),
                       "tokens_kernel launch");
}

template <typename Tin, typename Tout, bool kOut, bool kGiven>
lh_status launch_tokens_g(const void* X, const TokenArgs& p, void* out, int sms, cudaStream_t st) {
    // enough warps to hold the row (its own scale); more while there are few, which with a
    // given scale costs no reduction: up to 128 an SM, so that the loads in flight cover the
    // memory's latency (1777 x 17408 f32: 60 us with 16, 47 us with 128)
    int warps = 1;
    while (warps < 8 && ((!kGiven && p.J > 32 * kHeld<Tin> * warps) ||
                         (p.J > 32 * warps && p.n_rows * warps * 2 <= (kGiven ? 128 : 16) * (int64_t)sms)))
        warps *= 2;
    switch (warps) {
        case 1: return launch_tokens_w<Tin, Tout, kOut, kGiven, 1>(X, p, out, sms, st);
        case 2: return launch_tokens_w<Tin, Tout, kOut, kGiven, 2>(X, p, out, sms, st);
        case 4: return launch_tokens_w<Tin, Tout, kOut, kGiven, 4>(X, p, out, sms, st);
        default: return launch_tokens_w<Tin, Tout, kOut, kGiven, 8>(X, p, out, sms, st);
    }
}

template <typename Tin, typename Tout, bool kOut>
lh_status launch_tokens_o(const void* X, const TokenArgs& p, void* out, int sms, cudaStream_t st) {
    return p.gamax ? launch_tokens_g<Tin, Tout, kOut, true>(X, p, out, sms, st)
                   : launch_tokens_g<Tin, Tout, kOut, false>(X, p, out, sms, st);
}

template <typename Tin>
lh_status launch_tokens(const void* X, const TokenArgs& p, void* out, lh_dtype out_dtype, int sms, cudaStream_t st) {
    if (!out) return launch_tokens_o<Tin, float, false>(X, p, nullptr, sms, st);
    if (out_dtype == LH_BF16) return launch_tokens_o<Tin, uint16_t, true>(X, p, out, sms, st);
    return launch_tokens_o<Tin, float, true>(X, p, out, sms, st);
}

}  // namespace

lh_status check_tokens(const void* X, lh_dtype x_dtype, int64_t n_src, int64_t c_in, int64_t ld_x, const int32_t* rows,
                       int64_t row_div, int64_t n_rows, const int64_t* offsets, int64_t n_groups, const uint8_t* packed,
                       const uint8_t* scale_tiles, const float* token_scale, const void* X_out, lh_dtype out_dtype) {
    if (!valid_dtype(x_dtype) || (X_out && !valid_dtype(out_dtype))) return fail(LH_ERR_UNSUPPORTED, "unknown dtype");
    if (n_src < 0 || n_rows < 0 || c_in < 0 || n_groups < 1)
        return fail(LH_ERR_INVALID_ARG, "sizes must be >= 0, n_groups >= 1");
    if (n_rows > 0 && c_in > 0 && ((!X && n_src > 0) || !packed || !scale_tiles || !token_scale))
        return fail(LH_ERR_INVALID_ARG, "null pointer argument");
    if (row_div < 1) return fail(LH_ERR_INVALID_ARG, "row_div must be >= 1");
    if (n_rows > INT_MAX - 512 || n_groups > INT_MAX - 512)
        return fail(LH_ERR_UNSUPPORTED, "n_rows and n_groups must be below 2^31 - 512");
    if (row_div > INT_MAX) return fail(LH_ERR_UNSUPPORTED, "row_div must be below 2^31");
    if (!rows && (row_div != 1 || n_rows > n_src))
        return fail(LH_ERR_INVALID_ARG, "without rows, row_div must be 1 and n_rows at most n_src");
    if (!offsets && n_groups != 1) return fail(LH_ERR_INVALID_ARG, "several groups need offsets");
    if (c_in % 16 != 0) return fail(LH_ERR_UNSUPPORTED, "c_in=%lld is not a multiple of 16", (long long)c_in);
    if (ld_x < c_in) return fail(LH_ERR_INVALID_ARG, "ld_x=%lld < c_in=%lld", (long long)ld_x, (long long)c_in);
    if (!aligned16(X) || (ld_x * elem_bytes(x_dtype)) % 16 != 0)
        return fail(LH_ERR_ALIGNMENT, "X must be 16-byte aligned with 16-byte aligned rows");
    if (!aligned16(packed) || !aligned16(scale_tiles) || !aligned16(X_out))
        return fail(LH_ERR_ALIGNMENT, "packed, scale_tiles and X_out must be 16-byte aligned");
    if (c_in > (1 << 28)) return fail(LH_ERR_UNSUPPORTED, "c_in must be at most 2^28");  // a row of scale tiles: 2^31 bytes
    if (same_array(X, X_out) || same_array(X, packed) || same_array(X, scale_tiles) || same_array(packed, scale_tiles))
        return fail(LH_ERR_INVALID_ARG, "outputs must not alias X or one another");
    return LH_OK;
}

}  // namespace lh

extern "C" size_t lh_nvfp4_token_scale_bytes(int64_t n_rows, int64_t c_in, int64_t n_groups) {
    using namespace lh;
    if (n_rows < 0 || n_groups < 1 || c_in < 16 || c_in % 16 != 0) return 0;
    return (size_t)((n_rows / kTileRows + n_groups) * scale_steps(c_in) * kTileBytes);
}

extern "C" size_t lh_nvfp4_weight_scale_bytes(int64_t n_mats, int64_t c_out, int64_t c_in) {
    using namespace lh;
    if (n_mats < 1 || c_out < 0 || c_in < 16 || c_in % 16 != 0) return 0;
    return (size_t)(n_mats * ((c_out + kTileRows - 1) / kTileRows) * scale_steps(c_in) * kTileBytes);
}

extern "C" lh_status lh_nvfp4_tile_scales(const uint8_t* block_scales, int64_t n_mats, int64_t c_out, int64_t c_in,
                                          uint8_t* tiles, void* stream) {
    using namespace lh;
    clear_error();
    if (c_out != 0 && c_in != 0 && (!block_scales || !tiles)) return fail(LH_ERR_INVALID_ARG, "null pointer argument");
    if (n_mats < 1 || c_out < 0 || c_in < 0) return fail(LH_ERR_INVALID_ARG, "n_mats must be >= 1, sizes >= 0");
    if (c_in % 16 != 0) return fail(LH_ERR_UNSUPPORTED, "c_in=%lld is not a multiple of 16", (long long)c_in);
    if (!aligned16(tiles)) return fail(LH_ERR_ALIGNMENT, "tiles must be 16-byte aligned");
    if (same_array(block_scales, tiles)) return fail(LH_ERR_INVALID_ARG, "tiles must not alias block_scales");
    if (c_out == 0 || c_in == 0) return LH_OK;
    const int sms = sm_count();
    if (sms <= 0) return fail(LH_ERR_CUDA, "no CUDA device");
    const int64_t row_tiles = (c_out + kTileRows - 1) / kTileRows;
    const int64_t n = (int64_t)lh_nvfp4_weight_scale_bytes(n_mats, c_out, c_in) / 4;
    int64_t grid = (n + 255) / 256;
    if (grid > (int64_t)sms * 16) grid = (int64_t)sms * 16;
    tile_scales_kernel<<<(unsigned)grid, 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
        block_scales, n_mats, c_out, c_in / 16, scale_steps(c_in), row_tiles, reinterpret_cast<uint32_t*>(tiles));
    return cuda_status(cudaGetLastError(), "tile_scales_kernel launch");
}

extern "C" lh_status lh_quantize_tokens(const void* X, lh_dtype x_dtype, int64_t n_src, int64_t c_in, int64_t ld_x,
                                        const int32_t* rows, int64_t row_div, int64_t n_rows, const int64_t* offsets,
                                        int64_t n_groups, const float* global_amax, uint8_t* packed,
                                        uint8_t* scale_tiles, float* token_scale, void* X_out, lh_dtype out_dtype,
                                        void* stream) {
    using namespace lh;
    clear_error();
    const lh_status ok = check_tokens(X, x_dtype, n_src, c_in, ld_x, rows, row_div, n_rows, offsets, n_groups, packed,
                                      scale_tiles, token_scale, X_out, out_dtype);
    if (ok != LH_OK) return ok;
    if (n_rows == 0 || c_in == 0 || n_src == 0) return LH_OK;
    const int sms = sm_count();
    if (sms <= 0) return fail(LH_ERR_CUDA, "no CUDA device");
    TokenArgs p;
    p.n_src = n_src; p.ld = ld_x; p.n_rows = (int)n_rows;
    p.G = (int)n_groups; p.J = (int)(c_in / 16); p.steps = (int)scale_steps(c_in);
    p.div_shift = 0;  // with 2^(s-1) < row_div <= 2^s: ceil(2^(31+s) / row_div), exact for 31-bit dividends
    while ((int64_t(1) << p.div_shift) < row_div) ++p.div_shift;
    p.div_mul = row_div == 1 ? 0u : (uint32_t)(((uint64_t(1) << (31 + p.div_shift)) + row_div - 1) / row_div);
    if (row_div > 1) --p.div_shift;
    p.rows = (const int*)rows; p.offsets = offsets; p.gamax = global_amax;
    p.wide_in = (reinterpret_cast<uintptr_t>(X) & 31) == 0 && (ld_x * elem_bytes(x_dtype)) % 32 == 0;
    p.wide_out = (reinterpret_cast<uintptr_t>(X_out) & 31) == 0;
    p.packed = packed; p.tiles = scale_tiles; p.gscale = token_scale;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (x_dtype == LH_BF16) return launch_tokens<uint16_t>(X, p, X_out, out_dtype, sms, st);
    return launch_tokens<float>(X, p, X_out, out_dtype, sms, st);
}
