// Tokens sorted by expert, and back.
//
// A bank of experts (one matrix per expert, as the Hessian, the sweep and the
// products take it) wants the rows of one expert next to one another, with
// offsets. These entry points make that order from the router's expert ids,
// copy rows into it, and bring the experts' results back to the tokens with the
// router's weights, with the gradient of that step.
//
//   flat index f = t * k + s (token t, slot s), expert ids[f];
//   order = the valid f sorted by (ids[f], f);  pos[order[p]] = p;
//   gather:   Xs[p] = X[order[p] / k]
//   combine:  Y[t]  = sum_s w[t][s] * Ys[pos[t][s]]
//   gradient: dYs[pos[t][s]] = w[t][s] * dY[t],  dw[t][s] = <dY[t], Ys[pos[t][s]]>
#include <climits>

#include "common.cuh"
#include "tcgen05.cuh"

namespace lh {
namespace {

// ---------------------------------------------------------------- route

constexpr int kRouteThreads = 1024;
constexpr int kRouteWarps = kRouteThreads / 32;
constexpr int kMaxExperts = 1024;  // one thread per expert in the scan
constexpr int kRouteCluster = 8;

using tc::cluster_rank;
using tc::cluster_size;
using tc::cluster_arrive;
using tc::cluster_sync;
using tc::cluster_wait;

__device__ __forceinline__ uint32_t ld_remote(const uint32_t* p, uint32_t rank) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(tc::cluster_addr(tc::smem_u32(p), rank)) : "memory");
    return v;
}

// A stable counting sort in one launch: one cluster, each CTA a contiguous chunk of
// the ids, each warp a contiguous run of its chunk. Every warp counts its run into a
// histogram of its own (lanes with the same expert find one another by a ballot for each
// bit of its number, the first of them adds; match.any, which does that in one instruction,
// takes longer than them all: 4096 ids 8.2 us), which also gives each id its rank in the run; the counts
// become prefixes over warps, CTAs (through distributed shared memory) and experts, and
// the ids take their places. No atomics: the order is that of the flat index. What
// bounds it is the chain of these steps, not the bytes; ranks stay in registers for the
// first kHeldIds of a lane, the others wait in pos.
constexpr int kHeldIds = 4;

__global__ void __launch_bounds__(kRouteThreads, 1) route_kernel(const int* __restrict__ ids, int n, int E,
                                                                 int64_t* __restrict__ offsets,
                                                                 int* __restrict__ order, int* __restrict__ pos) {
    extern __shared__ uint32_t sm[];
    const int stride = E | 1;      // odd: a column of the histograms touches every bank
    uint32_t* total = sm;          // [E] this CTA's count per expert
    uint32_t* base = total + E;    // [E] first place of this CTA's rows of an expert
    uint32_t* hist = base + E;     // [warps][stride]
    __shared__ uint32_t wsum[kRouteWarps];
    __shared__ uint32_t n_valid;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank(), ranks = cluster_size();
    for (int i = tid; i < kRouteWarps * stride; i += kRouteThreads) hist[i] = 0u;
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const int64_t per_warp = (((int64_t)n + ranks * kRouteThreads - 1) / (ranks * kRouteThreads)) * 32;
    const int64_t w0 = ((int64_t)rank * kRouteWarps + warp) * per_warp;
    const int f0 = (int)(w0 < n ? w0 : n);
    const int f1 = (int)(w0 + per_warp < n ? w0 + per_warp : n);
    uint32_t* mine = hist + warp * stride;
    auto expert_of = [&](int f) {
        const int e = f < f1 ? __ldg(ids + f) : -1;
        return e >= 0 && e < E ? e : -1;
    };
    const int bits = 32 - __clz(E - 1);
    auto count = [&](int e) {  // the id's rank in the run
        uint32_t same = __ballot_sync(0xFFFFFFFFu, e >= 0);
        for (int b = 0; b < bits; ++b) {
            const uint32_t set = __ballot_sync(0xFFFFFFFFu, (e >> b) & 1);
            same &= (e >> b) & 1 ? set : ~set;
        }
        const uint32_t before = e >= 0 ? mine[e] : 0;
        __syncwarp();
        if (e >= 0 && lane == __ffs(same) - 1) mine[e] = before + __popc(same);
        __syncwarp();
        return (int)(before + __popc(same & ((1u << lane) - 1u)));
    };
    int e_held[kHeldIds], r_held[kHeldIds];
#pragma unroll
    for (int i = 0; i < kHeldIds; ++i) e_held[i] = expert_of(f0 + 32 * i + lane);
#pragma unroll
    for (int i = 0; i < kHeldIds; ++i)
        if (f0 + 32 * i < f1) r_held[i] = count(e_held[i]);
    for (int f = f0 + 32 * kHeldIds + lane; f - lane < f1; f += 32) {
        const int r = count(expert_of(f));
        if (f < f1) pos[f] = r;
    }
    __syncthreads();
    for (int e = warp; e < E; e += kRouteWarps) {  // counts -> prefixes over the CTA's warps, a lane per warp
        const uint32_t c = hist[lane * stride + e];
        uint32_t inc = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
            if (lane >= o) inc += v;
        }
        hist[lane * stride + e] = inc - c;
        if (lane == 31) total[e] = inc;
    }
    if (ranks > 1) cluster_sync();
    else __syncthreads();
    uint32_t all = 0, before = 0;
    if (tid < E) {
        if (ranks == 1) {
            all = total[tid];
        } else {
            uint32_t c[kRouteCluster];
#pragma unroll
            for (uint32_t r = 0; r < kRouteCluster; ++r) c[r] = ld_remote(total + tid, r);
#pragma unroll
            for (uint32_t r = 0; r < kRouteCluster; ++r) {
                if (r < rank) before += c[r];
                all += c[r];
            }
        }
    }
    // inclusive scan of `all` over the experts
    uint32_t inc = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += v;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        uint32_t s = wsum[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, s, o);
            if (lane >= o) s += v;
        }
        wsum[lane] = s;
    }
    __syncthreads();
    if (ranks > 1) cluster_arrive();  // this CTA has read the others' counts
    inc += warp ? wsum[warp - 1] : 0u;
    if (tid < E) {
        base[tid] = inc - all + before;
        if (rank == 0) {
            offsets[tid + 1] = (int64_t)inc;
            if (tid == 0) offsets[0] = 0;
        }
        if (tid == E - 1) n_valid = inc;
    }
    __syncthreads();
    auto place = [&](int f, int e, int r) {
        if (f >= f1) return;
        const int p = e >= 0 ? (int)(base[e] + mine[e]) + r : -1;
        pos[f] = p;
        if (p >= 0) order[p] = f;
    };
#pragma unroll
    for (int i = 0; i < kHeldIds; ++i) place(f0 + 32 * i + lane, e_held[i], r_held[i]);
    for (int f = f0 + 32 * kHeldIds + lane; f - lane < f1; f += 32) place(f, expert_of(f), f < f1 ? pos[f] : 0);
    for (int64_t p = (int64_t)n_valid + rank * kRouteThreads + tid; p < n; p += ranks * kRouteThreads) order[p] = -1;
    if (ranks > 1) cluster_wait();  // a CTA's counts stay readable until every CTA has read them
}

// ---------------------------------------------------------------- rows

constexpr int kRowThreads = 256;

template <typename T>
struct Row16;  // 16 bytes of a row as floats
template <>
struct Row16<uint16_t> {
    static constexpr int kN = 8;
    __device__ static void unpack(const uint4& v, float (&x)[8]) {
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
    }
    __device__ static uint4 pack(const float (&x)[8]) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
    __device__ static float one(uint16_t v) { return bf16_bits_to_float(v); }
    __device__ static uint16_t rounded(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }
};
template <>
struct Row16<float> {
    static constexpr int kN = 4;
    __device__ static void unpack(const uint4& v, float (&x)[4]) {
        x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y);
        x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
    }
    __device__ static uint4 pack(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
    __device__ static float one(float v) { return v; }
    __device__ static float rounded(float x) { return x; }
};

// Rows are worked on as vectors of 32 bytes (16 where rows are not 32-byte aligned), one
// thread per vector of a row (gather: of kGatherRows rows), flat over the rows:
// neighbouring threads take neighbouring vectors, a few rows fill as many threads as they
// can, and every thread has its rows' loads in flight at once. The columns past the last
// whole vector go one by one to the thread after it. 32768 x 2048 bf16 gathered from 8192
// rows: 34.5 us with 16 bytes and four rows, 31.4 us with 32 bytes and two (25.6 us at the
// copy bandwidth).
constexpr int kGatherRows = 2;
constexpr int kSlots = 4;  // slots whose rows are loaded together
// CTAs per SM: few that stay suit the combination (8192 x 4 rows of 1536 bf16: 28 us with
// 32, 24 us with 4), whose threads each hold four rows' loads
constexpr int kCombineWaves = 4;

template <int kBytes>
struct Vec {
    uint4 q[kBytes / 16];
    __device__ __forceinline__ void load(const void* p) {
        if constexpr (kBytes == 32)
            asm("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                : "=r"(q[0].x), "=r"(q[0].y), "=r"(q[0].z), "=r"(q[0].w), "=r"(q[1].x), "=r"(q[1].y), "=r"(q[1].z),
                  "=r"(q[1].w)
                : "l"(p));
        else
            q[0] = __ldg(static_cast<const uint4*>(p));
    }
    // written once and not read here: kept from pushing the sources out of L2
    __device__ __forceinline__ void store(void* p) const {
        if constexpr (kBytes == 32)
            asm volatile("st.global.cs.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(q[0].x), "r"(q[0].y),
                         "r"(q[0].z), "r"(q[0].w), "r"(q[1].x), "r"(q[1].y), "r"(q[1].z), "r"(q[1].w)
                         : "memory");
        else
            __stcs(static_cast<uint4*>(p), q[0]);
    }
};

// This thread's (row, vector) with `per` vectors a row, of the CTA's vectors from `first`
// on: a division for each thread, of 32 bits where it can be (one of 64 bits takes as long
// as all the rest).
__device__ __forceinline__ void split(int64_t first, uint32_t per, int64_t& row, uint32_t& v) {
    if (first <= 0xFFFFFFFFll - kRowThreads) {
        const uint32_t i = (uint32_t)first + threadIdx.x, r = i / per;
        row = r;
        v = i - r * per;
    } else {
        const int64_t i = first + threadIdx.x;
        row = i / per;
        v = (uint32_t)(i - row * per);
    }
}

template <typename T, int kBytes>
__global__ void __launch_bounds__(kRowThreads) gather_kernel(const T* __restrict__ X, int64_t n_tok, int64_t c,
                                                             int64_t ld, const int* __restrict__ order, int64_t k,
                                                             int64_t n_rows, T* __restrict__ Xs, int64_t ld_s) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int V = kBytes / sizeof(T);
    const uint32_t nv = (uint32_t)(c / V), per = (uint32_t)((c + V - 1) / V);
    const int64_t n = (n_rows + kGatherRows - 1) / kGatherRows * per;
    for (int64_t i = (int64_t)blockIdx.x * kRowThreads; i < n; i += (int64_t)gridDim.x * kRowThreads) {
        int64_t p0;
        uint32_t v;
        split(i, per, p0, v);
        p0 *= kGatherRows;
        int64_t t[kGatherRows];
#pragma unroll
        for (int r = 0; r < kGatherRows; ++r) {
            const int f = p0 + r < n_rows ? __ldg(order + p0 + r) : -1;
            t[r] = f < 0 ? -1 : (int64_t)((uint32_t)f / (uint32_t)k);
            if (t[r] >= n_tok) t[r] = -1;
        }
        if (v < nv) {
            Vec<kBytes> x[kGatherRows];
#pragma unroll
            for (int r = 0; r < kGatherRows; ++r)
                if (t[r] >= 0) x[r].load(X + t[r] * ld + v * V);
#pragma unroll
            for (int r = 0; r < kGatherRows; ++r)
                if (t[r] >= 0) x[r].store(Xs + (p0 + r) * ld_s + v * V);
        } else {
            for (int r = 0; r < kGatherRows; ++r)
                if (t[r] >= 0)
                    for (int64_t j = (int64_t)nv * V; j < c; ++j) Xs[(p0 + r) * ld_s + j] = X[t[r] * ld + j];
        }
    }
}

// The sum runs over the slots in order, in FP32.
template <typename T, int kBytes>
__global__ void __launch_bounds__(kRowThreads) combine_kernel(const T* __restrict__ Ys, int64_t n_rows, int64_t c,
                                                              int64_t ld_s, const int* __restrict__ pos,
                                                              const float* __restrict__ w, int64_t n_tok, int k,
                                                              T* __restrict__ Y, int64_t ld) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int V = kBytes / sizeof(T), P = Row16<T>::kN;
    const uint32_t nv = (uint32_t)(c / V), per = (uint32_t)((c + V - 1) / V);
    for (int64_t i = (int64_t)blockIdx.x * kRowThreads; i < n_tok * per; i += (int64_t)gridDim.x * kRowThreads) {
        int64_t t;
        uint32_t v;
        split(i, per, t, v);
        if (t >= n_tok) continue;
        float acc[V] = {};
        for (int s0 = 0; s0 < k; s0 += kSlots) {
            int64_t p[kSlots];
            float ws[kSlots];
#pragma unroll
            for (int s = 0; s < kSlots; ++s) {
                p[s] = s0 + s < k ? __ldg(pos + t * k + s0 + s) : -1;
                if (p[s] >= n_rows) p[s] = -1;
                ws[s] = p[s] >= 0 && w ? __ldg(w + t * k + s0 + s) : 1.0f;
            }
            if (v < nv) {
                Vec<kBytes> x[kSlots];
#pragma unroll
                for (int s = 0; s < kSlots; ++s)
                    if (p[s] >= 0) x[s].load(Ys + p[s] * ld_s + v * V);
#pragma unroll
                for (int s = 0; s < kSlots; ++s) {
                    if (p[s] < 0) continue;
#pragma unroll
                    for (int h = 0; h < V / P; ++h) {
                        float f[P];
                        Row16<T>::unpack(x[s].q[h], f);
#pragma unroll
                        for (int j = 0; j < P; ++j) acc[h * P + j] = __fmaf_rn(ws[s], f[j], acc[h * P + j]);
                    }
                }
            } else {
                for (int s = 0; s < kSlots; ++s)
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        if (p[s] >= 0 && (int64_t)nv * V + j < c)
                            acc[j] = __fmaf_rn(ws[s], Row16<T>::one(Ys[p[s] * ld_s + (int64_t)nv * V + j]), acc[j]);
            }
        }
        T* dst = Y + t * ld;
        if (v < nv) {
            Vec<kBytes> y;
#pragma unroll
            for (int h = 0; h < V / P; ++h) {
                float f[P];
#pragma unroll
                for (int j = 0; j < P; ++j) f[j] = acc[h * P + j];
                y.q[h] = Row16<T>::pack(f);
            }
            y.store(dst + v * V);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if ((int64_t)nv * V + j < c) dst[(int64_t)nv * V + j] = Row16<T>::rounded(acc[j]);
        }
    }
}

// One CTA per token, kSlots slots at a time: dY[t] times each weight into the sorted
// rows, and the dot products with the rows, in FP32 in an order fixed by the threads.
constexpr int kGradThreads = 64;

template <typename T, int kBytes>
__global__ void __launch_bounds__(kGradThreads) combine_grad_kernel(const T* __restrict__ dY, int64_t n_tok, int k,
                                                                    int64_t c, int64_t ld, const T* __restrict__ Ys,
                                                                    int64_t ld_s, int64_t n_rows,
                                                                    const int* __restrict__ pos,
                                                                    const float* __restrict__ w, T* __restrict__ dYs,
                                                                    int64_t ld_d, float* __restrict__ dw) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int V = kBytes / sizeof(T), P = Row16<T>::kN;
    __shared__ float part[kGradThreads / 32][kSlots];
    const int tid = threadIdx.x, lane = tid & 31;
    const int64_t nv = c / V;
    for (int64_t t = blockIdx.x; t < n_tok; t += gridDim.x) {
        const T* dy = dY + t * ld;
        for (int s0 = 0; s0 < k; s0 += kSlots) {
            int64_t p[kSlots];
            float ws[kSlots], dot[kSlots] = {};
#pragma unroll
            for (int s = 0; s < kSlots; ++s) {
                p[s] = s0 + s < k ? __ldg(pos + t * k + s0 + s) : -1;
                if (p[s] >= n_rows) p[s] = -1;
                ws[s] = p[s] >= 0 && w ? __ldg(w + t * k + s0 + s) : 1.0f;
            }
            for (int64_t v = tid; v < nv; v += kGradThreads) {
                Vec<kBytes> x[kSlots], gv;
                gv.load(dy + v * V);
                if (dw) {
#pragma unroll
                    for (int s = 0; s < kSlots; ++s)
                        if (p[s] >= 0) x[s].load(Ys + p[s] * ld_s + v * V);
                }
                float g[V];
#pragma unroll
                for (int h = 0; h < V / P; ++h) {
                    float f[P];
                    Row16<T>::unpack(gv.q[h], f);
#pragma unroll
                    for (int j = 0; j < P; ++j) g[h * P + j] = f[j];
                }
#pragma unroll
                for (int s = 0; s < kSlots; ++s) {
                    if (p[s] < 0) continue;
                    Vec<kBytes> out;
#pragma unroll
                    for (int h = 0; h < V / P; ++h) {
                        float y[P], d[P];
                        if (dw) {
                            Row16<T>::unpack(x[s].q[h], y);
#pragma unroll
                            for (int j = 0; j < P; ++j) dot[s] = __fmaf_rn(g[h * P + j], y[j], dot[s]);
                        }
#pragma unroll
                        for (int j = 0; j < P; ++j) d[j] = g[h * P + j] * ws[s];
                        out.q[h] = Row16<T>::pack(d);
                    }
                    if (dYs) out.store(dYs + p[s] * ld_d + v * V);
                }
            }
            for (int64_t j = nv * V + tid; j < c; j += kGradThreads) {
                const float g = Row16<T>::one(dy[j]);
#pragma unroll
                for (int s = 0; s < kSlots; ++s) {
                    if (p[s] < 0) continue;
                    if (dw) dot[s] = __fmaf_rn(g, Row16<T>::one(Ys[p[s] * ld_s + j]), dot[s]);
                    if (dYs) dYs[p[s] * ld_d + j] = Row16<T>::rounded(g * ws[s]);
                }
            }
            if (!dw) continue;
#pragma unroll
            for (int s = 0; s < kSlots; ++s) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) dot[s] += __shfl_xor_sync(0xFFFFFFFFu, dot[s], o);
                if (lane == 0) part[tid >> 5][s] = dot[s];
            }
            __syncthreads();
            if (tid < kSlots && s0 + tid < k) {
                float d = 0.0f;
#pragma unroll
                for (int i = 0; i < kGradThreads / 32; ++i) d += part[i][tid];
                dw[t * k + s0 + tid] = d;
            }
            __syncthreads();
        }
    }
}

// CTAs for `items` of `per_cta`, at most `waves` CTAs per SM.
unsigned grid_for(int64_t items, int64_t per_cta, int sms, int waves) {
    const int64_t need = (items + per_cta - 1) / per_cta, cap = (int64_t)sms * waves;
    return (unsigned)(need < cap ? need : cap);
}

lh_status check_rows(const char* name, const void* p, lh_dtype t, int64_t c, int64_t ld) {
    if (c > INT_MAX) return fail(LH_ERR_UNSUPPORTED, "rows must have fewer than 2^31 columns");
    if (ld < c) return fail(LH_ERR_INVALID_ARG, "%s: leading dimension %lld < %lld columns", name, (long long)ld, (long long)c);
    if (!aligned16(p) || (ld * elem_bytes(t)) % 16 != 0)
        return fail(LH_ERR_ALIGNMENT, "%s must be 16-byte aligned with 16-byte aligned rows", name);
    return LH_OK;
}

// Whether the rows of p are 32-byte aligned.
bool wide_rows(const void* p, lh_dtype t, int64_t ld) {
    return (reinterpret_cast<uintptr_t>(p) & 31u) == 0 && (ld * elem_bytes(t)) % 32 == 0;
}

constexpr int64_t kMaxFlat = INT_MAX - 512;
static_assert(32 * kHeldIds + 32 <= 512 && kSlots <= 512, "steps past the last flat index");

lh_status check_slots(int64_t n_tok, int64_t k) {
    if (n_tok < 0 || k < 1) return fail(LH_ERR_INVALID_ARG, "n_tok must be >= 0 and k >= 1");
    // the kernels' 32-bit counters of flat indices and slots step past the last one
    if (k > kMaxFlat || (n_tok > 0 && n_tok > kMaxFlat / k))
        return fail(LH_ERR_UNSUPPORTED, "n_tok * k must be below 2^31 - 512");
    return LH_OK;
}

// Launch with programmatic serialisation: the kernels wait for the one before
// (griddepcontrol.wait) before they touch memory, so their start-up overlaps its end.
template <typename... P, typename... A>
lh_status launch_rows(const char* what, void (*kernel)(P...), unsigned grid, int threads, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, args...), what);
}

}  // namespace
}  // namespace lh

extern "C" lh_status lh_route_tokens(const int32_t* ids, int64_t n_tok, int64_t k, int64_t n_experts,
                                     int64_t* offsets, int32_t* order, int32_t* pos, void* stream) {
    using namespace lh;
    clear_error();
    lh_status s = check_slots(n_tok, k);
    if (s != LH_OK) return s;
    if (n_experts < 1) return fail(LH_ERR_INVALID_ARG, "n_experts must be >= 1");
    if (n_experts > kMaxExperts)
        return fail(LH_ERR_UNSUPPORTED, "n_experts=%lld is above %d", (long long)n_experts, kMaxExperts);
    if (!offsets || (n_tok > 0 && (!ids || !order || !pos))) return fail(LH_ERR_INVALID_ARG, "null pointer argument");
    if (n_tok > 0 && (order == pos || ids == order || ids == pos))
        return fail(LH_ERR_INVALID_ARG, "order, pos and ids must be different arrays");
    if (sm_count() <= 0) return fail(LH_ERR_CUDA, "no CUDA device");
    const int n = (int)(n_tok * k), E = (int)n_experts;
    const size_t smem = ((size_t)kRouteWarps * (E | 1) + 2 * (size_t)E) * sizeof(uint32_t);
    static std::atomic<uint64_t> done{0};  // for the largest number of experts
    s = allow_shared((const void*)route_kernel, (size_t)(kRouteWarps + 2) * (kMaxExperts + 1) * sizeof(uint32_t), done);
    if (s != LH_OK) return s;
    // one step of one CTA takes 1024 ids; more want the eight SMs of a cluster (4096 ids: 6.7 us in one CTA, 5.0 us)
    const unsigned ctas = n <= kRouteThreads ? 1 : kRouteCluster;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kRouteThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cuda_status(cudaLaunchKernelEx(&cfg, route_kernel, (const int*)ids, n, E, offsets, (int*)order, (int*)pos),
                       "route_kernel launch");
}

extern "C" lh_status lh_gather_tokens(const void* X, lh_dtype dtype, int64_t n_tok, int64_t c, int64_t ld_x,
                                      const int32_t* order, int64_t k, int64_t n_rows, void* Xs, int64_t ld_xs,
                                      void* stream) {
    using namespace lh;
    clear_error();
    if (!valid_dtype(dtype)) return fail(LH_ERR_UNSUPPORTED, "dtype %d is not LH_BF16 or LH_F32", (int)dtype);
    if (n_tok < 0 || c < 0 || k < 1 || n_rows < 0) return fail(LH_ERR_INVALID_ARG, "sizes must be >= 0, k >= 1");
    const bool nothing = n_tok == 0 || c == 0 || n_rows == 0;
    if (!nothing && (!X || !order || !Xs)) return fail(LH_ERR_INVALID_ARG, "null pointer argument");
    if (k > INT_MAX) return fail(LH_ERR_UNSUPPORTED, "k must be below 2^31");
    if (same_array(X, Xs)) return fail(LH_ERR_INVALID_ARG, "Xs must not alias X");
    lh_status s = check_rows("X", X, dtype, c, ld_x);
    if (s == LH_OK) s = check_rows("Xs", Xs, dtype, c, ld_xs);
    if (s != LH_OK) return s;
    if (nothing) return LH_OK;
    const int sms = sm_count();
    if (sms <= 0) return fail(LH_ERR_CUDA, "no CUDA device");
    const bool wide = wide_rows(X, dtype, ld_x) && wide_rows(Xs, dtype, ld_xs);
    const int bytes = wide ? 32 : 16;
    const int64_t per = (c * elem_bytes(dtype) + bytes - 1) / bytes;
    const unsigned grid = grid_for((n_rows + kGatherRows - 1) / kGatherRows * per, kRowThreads, sms, 32);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int* o = (const int*)order;
    if (dtype == LH_BF16)
        return launch_rows("gather_kernel launch", wide ? gather_kernel<uint16_t, 32> : gather_kernel<uint16_t, 16>, grid,
                           kRowThreads, st, (const uint16_t*)X, n_tok, c, ld_x, o, k, n_rows, (uint16_t*)Xs, ld_xs);
    return launch_rows("gather_kernel launch", wide ? gather_kernel<float, 32> : gather_kernel<float, 16>, grid,
                       kRowThreads, st, (const float*)X, n_tok, c, ld_x, o, k, n_rows, (float*)Xs, ld_xs);
}

extern "C" lh_status lh_combine_tokens(const void* Ys, lh_dtype dtype, int64_t n_rows, int64_t c, int64_t ld_ys,
                                       const int32_t* pos, const float* weights, int64_t n_tok, int64_t k, void* Y,
                                       int64_t ld_y, void* stream) {
    using namespace lh;
    clear_error();
    if (!valid_dtype(dtype)) return fail(LH_ERR_UNSUPPORTED, "dtype %d is not LH_BF16 or LH_F32", (int)dtype);
    lh_status s = check_slots(n_tok, k);
    if (s != LH_OK) return s;
    if (n_rows < 0 || c < 0) return fail(LH_ERR_INVALID_ARG, "sizes must be >= 0");
    const bool nothing = n_tok == 0 || c == 0;
    if (!nothing && ((!Ys && n_rows > 0) || !pos || !Y)) return fail(LH_ERR_INVALID_ARG, "null pointer argument");
    if (same_array(Y, Ys)) return fail(LH_ERR_INVALID_ARG, "Y must not alias Ys");
    s = check_rows("Ys", Ys, dtype, c, ld_ys);
    if (s == LH_OK) s = check_rows("Y", Y, dtype, c, ld_y);
    if (s != LH_OK) return s;
    if (nothing) return LH_OK;
    const int sms = sm_count();
    if (sms <= 0) return fail(LH_ERR_CUDA, "no CUDA device");
    const bool wide = wide_rows(Ys, dtype, ld_ys) && wide_rows(Y, dtype, ld_y);
    const int bytes = wide ? 32 : 16;
    const unsigned grid = grid_for(n_tok * ((c * elem_bytes(dtype) + bytes - 1) / bytes), kRowThreads, sms, kCombineWaves);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == LH_BF16)
        return launch_rows("combine_kernel launch", wide ? combine_kernel<uint16_t, 32> : combine_kernel<uint16_t, 16>,
                           grid, kRowThreads, st, (const uint16_t*)Ys, n_rows, c, ld_ys, (const int*)pos, weights, n_tok,
                           (int)k, (uint16_t*)Y, ld_y);
    return launch_rows("combine_kernel launch", wide ? combine_kernel<float, 32> : combine_kernel<float, 16>, grid,
                       kRowThreads, st, (const float*)Ys, n_rows, c, ld_ys, (const int*)pos, weights, n_tok, (int)k,
                       (float*)Y, ld_y);
}

extern "C" lh_status lh_combine_tokens_grad(const void* dY, lh_dtype dtype, int64_t n_tok, int64_t k, int64_t c,
                                            int64_t ld_dy, const void* Ys, int64_t ld_ys, int64_t n_rows,
                                            const int32_t* pos, const float* weights, void* dYs, int64_t ld_dys,
                                            float* dweights, void* stream) {
    using namespace lh;
    clear_error();
    if (!valid_dtype(dtype)) return fail(LH_ERR_UNSUPPORTED, "dtype %d is not LH_BF16 or LH_F32", (int)dtype);
    lh_status s = check_slots(n_tok, k);
    if (s != LH_OK) return s;
    if (n_rows < 0 || c < 0) return fail(LH_ERR_INVALID_ARG, "sizes must be >= 0");
    const bool no_rows = n_rows == 0 || c == 0;  // of Ys and dYs
    if (n_tok > 0) {
        if ((!dY && c > 0) || !pos) return fail(LH_ERR_INVALID_ARG, "null pointer argument");
        if (!dYs && !dweights && !no_rows) return fail(LH_ERR_INVALID_ARG, "one of dYs and dweights is needed");
        if (dweights && !Ys && !no_rows) return fail(LH_ERR_INVALID_ARG, "dweights needs Ys");
    }
    if (same_array(dYs, dY) || same_array(dYs, Ys)) return fail(LH_ERR_INVALID_ARG, "dYs must not alias an input");
    s = check_rows("dY", dY, dtype, c, ld_dy);
    if (s == LH_OK && dweights) s = check_rows("Ys", Ys, dtype, c, ld_ys);
    if (s == LH_OK && dYs) s = check_rows("dYs", dYs, dtype, c, ld_dys);
    if (s != LH_OK) return s;
    if (n_tok == 0 || (no_rows && !dweights)) return LH_OK;
    const int sms = sm_count();
    if (sms <= 0) return fail(LH_ERR_CUDA, "no CUDA device");
    const bool wide = wide_rows(dY, dtype, ld_dy) && (!dweights || wide_rows(Ys, dtype, ld_ys)) &&
                      (!dYs || wide_rows(dYs, dtype, ld_dys));
    const unsigned grid = grid_for(n_tok, 1, sms, 8);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == LH_BF16)
        return launch_rows("combine_grad_kernel launch",
                           wide ? combine_grad_kernel<uint16_t, 32> : combine_grad_kernel<uint16_t, 16>, grid,
                           kGradThreads, st, (const uint16_t*)dY, n_tok, (int)k, c, ld_dy, (const uint16_t*)Ys, ld_ys,
                           n_rows, (const int*)pos, weights, (uint16_t*)dYs, ld_dys, dweights);
    return launch_rows("combine_grad_kernel launch",
                       wide ? combine_grad_kernel<float, 32> : combine_grad_kernel<float, 16>, grid, kGradThreads, st,
                       (const float*)dY, n_tok, (int)k, c, ld_dy, (const float*)Ys, ld_ys, n_rows, (const int*)pos, weights,
                       (float*)dYs, ld_dys, dweights);
}
