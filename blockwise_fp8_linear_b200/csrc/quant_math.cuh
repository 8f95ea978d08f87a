// quant_math.cuh -- the arithmetic of E4M3 quantization with FP32 scales: group scale,
// correctly rounded division by it, and the rounding onto E4M3.  Used by the
// quantizers and by the kernels that quantize their activations themselves.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace fp8bw {

// Two FP32 values -> two E4M3 codes (RNE, saturating); `lo` lands in the low byte.
__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Per-group division x / s, correctly rounded to binary32.
//
// Fast path (s in [2^-90, 2^90]): one correctly rounded reciprocal r = RN(1/s) per
// group, then per value q0 = RN(x*r), e = x - q0*s (exact by FMA) and
// q = RN(q0 + e*r).  By Markstein's theorem (P. Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", IBM J. Res. Dev. 34(1), 1990;
// also Muller et al., Handbook of Floating-Point Arithmetic, ch. 4) this is the
// correctly rounded quotient whenever no intermediate underflows; quotients small
// enough for that to matter lie far below half the smallest E4M3 subnormal (2^-10),
// where only the sign survives, and the sign is restored from x.  Outside that
// range of s the group falls back to the compiler's IEEE division.  The test suite
// checks the fast path against IEEE division for every (BF16 amax, BF16 x) pair.
struct GroupDiv {
    float s, r;
    bool fast;
    __device__ __forceinline__ explicit GroupDiv(float scale) : s(scale)
    {
        fast = scale >= 0x1p-90f && scale <= 0x1p90f;
        r = fast ? __frcp_rn(scale) : 0.0f;
    }
};

// The group scale amax / 448, correctly rounded to binary32, in three operations
// instead of a full division: q0 = RN(amax * RN(1/448)), then one correction step
// (Markstein's, as in GroupDiv below): d = RN(amax - q0 * 448) by FMA, s = RN(q0 + d *
// RN(1/448)).  amax is always a non-negative BF16 value widened to FP32 (32,640
// positive finite ones and zero); the sequence equals the IEEE quotient for every one
// of them, checked against the exact rational quotient on the host and against the
// oracle on the GPU for every BF16 amax.
__device__ __forceinline__ float scale_of_amax(float amax)
{
    constexpr float inv448 = 1.0f / 448.0f;
    const float q0 = __fmul_rn(amax, inv448);
    const float d = __fmaf_rn(-q0, 448.0f, amax);
    return __fmaf_rn(d, inv448, q0);
}

__device__ __forceinline__ float bf16lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Fast-path quotients of a pair of values by per-lane-half scales (r, -r and s given
// as packed pairs): q0 = x*r, d = q0*s - x (one FMA, exact), q = q0 - d*r.  The
// residual is taken as q0*s - x rather than x - q0*s so that zeros keep their sign
// with no fix-up: for x = +-0, q0 = +-0 and d = +0, so q = (-0) + (+-0) = +-0; when
// q0 underflows to a zero, d = -x exactly and q = x*r + q0 carries the sign of x; and
// q0 - d*r cannot cancel exactly to zero for a nonzero q0, because |d*r| is within
// an ulp of |q0 - x/s|, far below |q0|.
__device__ __forceinline__ float2 div2_fast(float2 x, float2 r, float2 neg_r, float2 s)
{
    const float2 q0 = __fmul2_rn(x, r);
    const float2 d = __ffma2_rn(q0, s, make_float2(-x.x, -x.y));
    return __ffma2_rn(d, neg_r, q0);
}

// |bf16| max over two packed words, as packed unsigned 16-bit halves (for
// non-negative BF16 values the integer order is the numeric order).
__device__ __forceinline__ uint32_t absmax2(uint32_t a, uint32_t b)
{
    return __vmaxu2(a & 0x7FFF7FFFu, b & 0x7FFF7FFFu);
}

__device__ __forceinline__ float halves_max_to_float(uint32_t m2)
{
    uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
    return __uint_as_float(m << 16);
}

// Eight BF16 values of one group (one uint4) -> eight E4M3 codes (one uint2), by the
// fast path (r = RN(1/s)) or by IEEE division.
__device__ __forceinline__ uint2 quant8_fast(uint4 v, float r, float s)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    const float2 r2 = make_float2(r, r), nr2 = make_float2(-r, -r), s2 = make_float2(s, s);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 q = div2_fast(make_float2(bf16lo(w[i]), bf16hi(w[i])), r2, nr2, s2);
        c[i] = cvt_e4m3x2(q.x, q.y);
    }
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

__device__ __forceinline__ uint2 quant8_ieee(uint4 v, float s)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c[i] = cvt_e4m3x2(__fdiv_rn(bf16lo(w[i]), s), __fdiv_rn(bf16hi(w[i]), s));
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

__device__ __forceinline__ uint2 quant8(uint4 v, const GroupDiv &d)
{
    return d.fast ? quant8_fast(v, d.r, d.s) : quant8_ieee(v, d.s);
}

} // namespace fp8bw
