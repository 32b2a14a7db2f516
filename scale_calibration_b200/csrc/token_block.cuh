// One block (16 values) of a token on its way to NVFP4, by one thread: its values in
// registers, its largest |x|, its scale's code under the row's global scale (internal
// header; the codes themselves are quantize_block's).
#pragma once

#include "nvfp4_block.cuh"

namespace lh {

// 16 values as they lie in memory.
template <typename T>
struct Held {
    uint32_t v[8 * (sizeof(T) / 2)];
    // wide: p is 32-byte aligned. A warp's 32-byte accesses fill whole sectors, where 16
    // bytes of every 32 or 64 make L2 handle each sector twice.
    __device__ void load(const T* p, bool wide) {
        if (wide) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
                uint32_t* u = v + 8 * i;
                asm("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                    : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
                    : "l"(reinterpret_cast<const uint32_t*>(p) + 8 * i));
            }
        } else {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T); ++i) {
                const uint4 u = __ldg(reinterpret_cast<const uint4*>(p) + i);
                v[4 * i] = u.x; v[4 * i + 1] = u.y; v[4 * i + 2] = u.z; v[4 * i + 3] = u.w;
            }
        }
    }
    __device__ void floats(float (&w)[16]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (sizeof(T) == 2) {
                w[2 * i] = __uint_as_float(v[i] << 16);
                w[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
            } else {
                w[2 * i] = __uint_as_float(v[2 * i]);
                w[2 * i + 1] = __uint_as_float(v[2 * i + 1]);
            }
        }
    }
    // Bits of the largest |x|; as integers, infinities and NaN come out on top.
    __device__ uint32_t max_bits() const {
        uint32_t m = 0;
        if constexpr (sizeof(T) == 2) {  // two bf16 at a time
#pragma unroll
            for (int i = 0; i < 8; ++i) m = __vmaxu2(m, v[i] & 0x7FFF7FFFu);
            return max(m << 16, m & 0xFFFF0000u);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) m = max(m, v[i] & 0x7FFFFFFFu);
            return m;
        }
    }
};

// A row's global scale, with its reciprocal where the quotient of a block needs no
// division: with g in [2^-85, 2^100], q = RN(a y) and RN(q + (a - q g) y) with y = RN(1/g)
// is the correctly rounded a / g for |a| >= 2^-100 (P. Markstein, IBM J. Res. Dev. 34(1),
// 1990: the residual is exact), and a smaller a gives less than 2^-14 either way, code 1.
// The same holds for a / 6, and for g itself.
struct RowScale {
    float g, ny, nan;
    bool fast;
    // From an amax >= 0 (or NaN).
    __device__ explicit RowScale(float amax) {
        nan = __int_as_float(0x7FFFFFFF);
        fast = amax >= 6.948286e-23f && amax <= 3.3230700e33f;  // 2688 * [2^-85, 2^100], rounded inwards
        if (fast) {
            g = quotient(amax, 2688.0f, -1.0f / 2688.0f);
            ny = -__frcp_rn(g);
        } else {
            g = __fdiv_rn(amax, 2688.0f);
            ny = 0.0f;
        }
    }
    __device__ static float quotient(float a, float d, float nyd) {
        const float nq = __fmul_rn(a, nyd);          // -q
        const float r = __fmaf_rn(nq, d, a);         // a - q d
        return -__fmaf_rn(r, nyd, nq);
    }
    // E4M3 code of a block whose largest |x| is a, and the block's scale.
    // kGiven: a may be above the row's amax.
    template <bool kGiven>
    __device__ uint32_t code(float a, float& s) const {
        uint32_t c = 1;
        if (fast)
            {
            const float sixth = quotient(a, 6.0f, -1.0f / 6.0f);
            c = (uint32_t)e4m3_rne_code(quotient(kGiven ? fminf(sixth, 512.0f * g) : sixth, g, ny));  // above: the largest code
        }
        else if (g != 0.0f)
            c = (uint32_t)e4m3_rne_code(__fdiv_rn(__fdiv_rn(a, 6.0f), g));
        c = c < 1 ? 1 : c;
        uint32_t h2;  // the code's value, exact in f16
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)c));
        s = __fmul_rn(__low2float(*reinterpret_cast<const __half2*>(&h2)), g);
        return c;
    }
};

// The codes of a block whose largest |x| has the bits bb: returns its scale's code, writes
// the packed E2M1 codes and (kOut) the values. not_finite: the token's own scale is not.
template <bool kOut, bool kGiven, typename T>
__device__ __forceinline__ uint32_t quantize_held(const Held<T>& h, uint32_t bb, const RowScale& rs, bool not_finite,
                                                  float (&o)[16], uint32_t (&word)[2]) {
    float s, w[16];
    uint32_t code = rs.template code<kGiven>(__uint_as_float(bb), s);
    if (bb >= 0x7F800000u || not_finite) {
        code = 0x7F;
        s = rs.nan;
    }
    h.floats(w);
    if constexpr (kGiven) {
        // far above the amax, the quotients of quantize_block would overflow
        const float far = 1.1529215e18f * s;
        if (s >= 2.524355e-29f && __uint_as_float(bb) > far) {
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = fminf(fmaxf(w[e], -far), far);
        }
    }
    quantize_block<kOut, true>(w, s, o, word);
    return code;
}

}  // namespace lh
