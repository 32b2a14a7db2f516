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

#include "nvfp4_block.cuh"
#include "scale_tiles.cuh"

namespace lh {
namespace {

constexpr int kTokThreads = 256;

struct TokenArgs {
    int64_t n_src, ld, row_div, n_rows, G, J, steps;
    const int* rows;         // source of each row (over row_div), or null
    const int64_t* offsets;  // groups of rows, or null
    const float* gamax;      // amax of the tensor, or null (per token)
    uint8_t* packed;
    uint8_t* tiles;
    float* gscale;
};

// Largest group g with offsets[g] <= row; false when the row lies in no group.
__device__ __forceinline__ bool find_group(const TokenArgs& p, int64_t row, int64_t& g, int64_t& lo) {
    if (!p.offsets) {
        g = 0;
        lo = 0;
        return true;
    }
    int64_t a = 0, b = p.G;  // offsets[a] <= row < offsets[b] if there is such a group
    while (b - a > 1) {
        const int64_t m = (a + b) >> 1;
        if (__ldg(p.offsets + m) <= row) a = m; else b = m;
    }
    g = a;
    lo = __ldg(p.offsets + a);
    lo = lo < 0 ? 0 : lo;
    return lo <= row && row < __ldg(p.offsets + a + 1);
}

__device__ __forceinline__ uint32_t block_max_bits(const float (&w)[16]) {
    uint32_t m = 0;  // as integers, infinities and NaN come out on top
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(w[i]) & 0x7FFFFFFFu);
    return m;
}

// One CTA per row: the row's largest |x|, then its blocks (from registers when a
// thread has one block at most, else read again, from L1 or L2).
template <typename Tin, typename Tout, bool kOut>
__global__ void __launch_bounds__(kTokThreads) tokens_kernel(const Tin* __restrict__ X, TokenArgs p,
                                                             Tout* __restrict__ out) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ uint32_t red[kTokThreads / 32];
    const int tid = threadIdx.x;
    for (int64_t row = blockIdx.x; row < p.n_rows; row += gridDim.x) {
        int64_t g, lo;
        if (!find_group(p, row, g, lo)) continue;
        const int64_t src = p.rows ? (int64_t)__ldg(p.rows + row) : row;
        if (src < 0 || src / p.row_div >= p.n_src) continue;
        const Tin* x = X + (src / p.row_div) * p.ld;
        float w[16];
        uint32_t mb = 0;
        for (int64_t j = tid; j < p.J; j += kTokThreads) {
            Vec16<Tin>::load(x + 16 * j, w);
            mb = max(mb, block_max_bits(w));
        }
        mb = __reduce_max_sync(0xFFFFFFFFu, mb);
        __syncthreads();
        if ((tid & 31) == 0) red[tid >> 5] = mb;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kTokThreads / 32; ++i) mb = max(mb, red[i]);
        const bool bad_row = mb >= 0x7F800000u;
        const float gs = __fdiv_rn(p.gamax ? __ldg(p.gamax) : __uint_as_float(mb), 2688.0f);
        const float nan = __int_as_float(0x7FFFFFFF);
        if (tid == 0) p.gscale[row] = bad_row ? nan : gs;
        const int64_t r = row - lo;
        const int64_t tile = group_tile(lo, g) + r / kTileRows;
        const int rt = (int)(r % kTileRows);
        for (int64_t j = tid; j < 4 * p.steps; j += kTokThreads) {
            uint32_t code = 0;
            if (j < p.J) {
                Vec16<Tin>::load(x + 16 * j, w);
                const uint32_t bb = block_max_bits(w);
                float s;
                if (bb >= 0x7F800000u || (bad_row && !p.gamax)) {
                    code = 0x7F;
                    s = nan;
                } else {
                    code = 1;
                    if (gs != 0.0f) {
                        const int c = e4m3_rne_code(__fdiv_rn(__fdiv_rn(__uint_as_float(bb), 6.0f), gs));
                        code = c < 1 ? 1 : c;
                    }
                    s = __fmul_rn(e4m3_value((int)code), gs);
                }
                float o[16];
                uint32_t word[2];
                quantize_block<kOut, true>(w, s, o, word);
                reinterpret_cast<uint2*>(p.packed)[row * p.J + j] = make_uint2(word[0], word[1]);
                if constexpr (kOut) Vec16<Tout>::store(out + (row * p.J + j) * 16, o);
            }
            p.tiles[scale_offset(tile, rt, j >> 2, p.steps) + (j & 3)] = (uint8_t)code;
        }
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

template <typename Tin, bool kOut>
lh_status launch_tokens(const void* X, const TokenArgs& p, void* out, lh_dtype out_dtype, int sms, cudaStream_t st) {
    const int64_t cap = (int64_t)sms * 8;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.n_rows < cap ? p.n_rows : cap));
    cfg.blockDim = dim3(kTokThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (out_dtype == LH_BF16)
        return cuda_status(cudaLaunchKernelEx(&cfg, tokens_kernel<Tin, uint16_t, kOut>, (const Tin*)X, p, (uint16_t*)out),
                           "tokens_kernel launch");
    return cuda_status(cudaLaunchKernelEx(&cfg, tokens_kernel<Tin, float, kOut>, (const Tin*)X, p, (float*)out),
                       "tokens_kernel launch");
}

}  // namespace
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
    if (!block_scales || !tiles) return fail(LH_ERR_INVALID_ARG, "null pointer argument");
    if (n_mats < 1 || c_out < 0 || c_in < 0) return fail(LH_ERR_INVALID_ARG, "n_mats must be >= 1, sizes >= 0");
    if (c_in % 16 != 0) return fail(LH_ERR_UNSUPPORTED, "c_in=%lld is not a multiple of 16", (long long)c_in);
    if (!aligned16(tiles)) return fail(LH_ERR_ALIGNMENT, "tiles must be 16-byte aligned");
    if (block_scales == tiles) return fail(LH_ERR_INVALID_ARG, "tiles must not alias block_scales");
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
    if (!valid_dtype(x_dtype) || (X_out && !valid_dtype(out_dtype))) return fail(LH_ERR_UNSUPPORTED, "unknown dtype");
    if (!X || !packed || !scale_tiles || !token_scale) return fail(LH_ERR_INVALID_ARG, "null pointer argument");
    if (n_src < 0 || n_rows < 0 || c_in < 0 || n_groups < 1)
        return fail(LH_ERR_INVALID_ARG, "sizes must be >= 0, n_groups >= 1");
    if (row_div < 1) return fail(LH_ERR_INVALID_ARG, "row_div must be >= 1");
    if (!rows && (row_div != 1 || n_rows > n_src))
        return fail(LH_ERR_INVALID_ARG, "without rows, row_div must be 1 and n_rows at most n_src");
    if (!offsets && n_groups != 1) return fail(LH_ERR_INVALID_ARG, "several groups need offsets");
    if (c_in % 16 != 0) return fail(LH_ERR_UNSUPPORTED, "c_in=%lld is not a multiple of 16", (long long)c_in);
    if (ld_x < c_in) return fail(LH_ERR_INVALID_ARG, "ld_x=%lld < c_in=%lld", (long long)ld_x, (long long)c_in);
    if (!aligned16(X) || (ld_x * elem_bytes(x_dtype)) % 16 != 0)
        return fail(LH_ERR_ALIGNMENT, "X must be 16-byte aligned with 16-byte aligned rows");
    if (!aligned16(packed) || !aligned16(scale_tiles) || !aligned16(X_out))
        return fail(LH_ERR_ALIGNMENT, "packed, scale_tiles and X_out must be 16-byte aligned");
    if (X == X_out || X == (const void*)packed || X == (const void*)scale_tiles || packed == scale_tiles)
        return fail(LH_ERR_INVALID_ARG, "outputs must not alias X or one another");
    if (n_rows == 0 || c_in == 0 || n_src == 0) return LH_OK;
    const int sms = sm_count();
    if (sms <= 0) return fail(LH_ERR_CUDA, "no CUDA device");
    TokenArgs p;
    p.n_src = n_src; p.ld = ld_x; p.row_div = row_div; p.n_rows = n_rows;
    p.G = n_groups; p.J = c_in / 16; p.steps = scale_steps(c_in);
    p.rows = (const int*)rows; p.offsets = offsets; p.gamax = global_amax;
    p.packed = packed; p.tiles = scale_tiles; p.gscale = token_scale;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (x_dtype == LH_BF16)
        return X_out ? launch_tokens<uint16_t, true>(X, p, X_out, out_dtype, sms, st)
                     : launch_tokens<uint16_t, false>(X, p, nullptr, LH_F32, sms, st);
    return X_out ? launch_tokens<float, true>(X, p, X_out, out_dtype, sms, st)
                 : launch_tokens<float, false>(X, p, nullptr, LH_F32, sms, st);
}
