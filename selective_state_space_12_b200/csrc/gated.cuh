// Arithmetic of the gated linear recurrence, shared by its kernels (gated.cu).
//
// For one channel with k = -c softplus(lam) <= 0, and gates r, i of a token:
//
//   s = k sigmoid(r)      a = exp(s)      m = sqrt(1 - a^2)
//   h <- a h + m sigmoid(i) x             (a reset token: a = 0, m = 1)
//
// a is close to 1 for channels that remember long, and an error of a is
// multiplied by that memory, so nothing here forms 1 - a by subtraction:
// with E = exp(s) - 1, a = 1 + E (one rounding) and m^2 = -E (2 + E). For
// s >= kSeries, E is its Taylor series s (1 + s/2 + ... + s^5/720), whose
// remainder is below s^6/5040 < 1e-9 relative; below, exp2 of the
// special-function unit (relative error about 2^-22) minus one, where
// |E| > 0.11. The series takes no special-function operation; those bind these
// kernels beside the memory (16 a clock and SM), so both sigmoids also share
// one reciprocal.
#pragma once

#include "common.cuh"
#include "tc_ptx.cuh"

namespace ssd {
namespace gated {

constexpr int kBlock = 64;          // SSD_GATED_BLOCK: tokens per saved state and 8-bit scale
constexpr float kSeries = -0.125f;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float rcp_approx(float v) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v));
    return y;
}
__device__ __forceinline__ float rsqrt_approx(float v) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v));
    return y;
}
__device__ __forceinline__ float min_nan(float a, float b) {  // a NaN stays one
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// k = -c softplus(lam), and sigmoid(lam) / softplus(lam) (its limit 1 where
// softplus underflows), by which the gradient of lam follows from that of log a.
__device__ __forceinline__ float softplus_full(float v) {
    return fmaxf(v, 0.f) + log1pf(expf(-fabsf(v)));
}
__device__ __forceinline__ float lam_ratio(float lam) {
    const float sp = softplus_full(lam);
    return sp > 0.f ? 1.f / ((1.f + expf(-lam)) * sp) : (lam == lam ? 1.f : lam);
}

// sigmoid(r) and sigmoid(i) from one reciprocal: 1/p = q/(pq). Exponents stop
// at 2^63, so that the product stays finite: a gate below 2^-63 reads 2^-63.
__device__ __forceinline__ void two_sigmoids(float r, float i, float &sr, float &si) {
    const float p = 1.f + tc::fast_exp2(min_nan(-r * kLog2e, 63.f));
    const float q = 1.f + tc::fast_exp2(min_nan(-i * kLog2e, 63.f));
    const float R = rcp_approx(p * q);
    sr = q * R;
    si = p * R;
}

// E = exp(s) - 1 for s <= 0. FAST: the caller knows that s >= kSeries.
template <bool FAST>
__device__ __forceinline__ float expm1_neg(float s) {
    float p = 1.f / 720.f;
    p = fmaf(p, s, 1.f / 120.f);
    p = fmaf(p, s, 1.f / 24.f);
    p = fmaf(p, s, 1.f / 6.f);
    p = fmaf(p, s, 0.5f);
    p = fmaf(p, s, 1.f);
    const float series = s * p;
    if (FAST) return series;
    return s >= kSeries ? series : tc::fast_exp2(s * kLog2e) - 1.f;
}

// A reset's decay is written -0: it passes nothing on, whatever stands before
// it (an infinity or a NaN times 0 would). Products of decays keep the mark,
// as decays are >= +0.
constexpr uint32_t kResetBits = 0x80000000u;
__device__ __forceinline__ float reset_decay() { return __uint_as_float(kResetBits); }
__device__ __forceinline__ float carry_on(float a, float h, float u) {  // a h + u
    return __float_as_uint(a) == kResetBits ? u : fmaf(a, h, u);
}

struct Gate {
    float sr, si;  // sigmoids
    float s;       // log a
    float a, m2;   // decay and m^2
    float rm;      // 1 / m (large where m = 0, with m2 * rm = 0 there)
    __device__ __forceinline__ float m() const { return m2 * rm; }
};

template <bool FAST>
__device__ __forceinline__ Gate gate(float r, float i, float k) {
    Gate g;
    two_sigmoids(r, i, g.sr, g.si);
    g.s = k * g.sr;
    const float E = expm1_neg<FAST>(g.s);
    g.a = 1.f + E;
    g.m2 = -E * (2.f + E);
    g.rm = rsqrt_approx(g.m2 < 1e-36f ? 1e-36f : g.m2);
    return g;
}

}  // namespace gated
}  // namespace ssd
