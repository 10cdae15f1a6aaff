// Arithmetic of the gated linear recurrence, shared by its kernels (gated.cu).
//
// For one channel with k = c softplus(lam) >= 0, and gates r, i of a token:
//
//   q = k sigmoid(r)      a = exp(-q)      m = sqrt(1 - a^2)
//   h <- a h + m sigmoid(i) x              (a reset token: a = 0, m = 1)
//
// a is close to 1 for channels that remember long, and an error of a is
// multiplied by that memory, so nothing here forms 1 - a by subtraction:
// with F = 1 - exp(-q), a = 1 - F (one rounding) and m^2 = F (1 + a). For
// q <= kSeries, F is its Taylor series q (1 - q/2 + ... + q^4/120), whose
// remainder is below q^5/720 < 5e-8 relative; above, one minus exp2 of the
// special-function unit (relative error about 2^-22), where F > 0.11. The
// series takes no special-function operation; those bind these kernels beside
// the memory (16 a clock and SM), so both sigmoids also share one reciprocal.
#pragma once

#include "common.cuh"
#include "tc_ptx.cuh"

namespace ssd {
namespace gated {

constexpr int kBlock = 64;          // SSD_GATED_BLOCK: tokens per saved state and 8-bit scale
constexpr float kSeries = 0.125f;
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

// softplus(lam), and sigmoid(lam) / softplus(lam) (its limit 1 where
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

// F = 1 - exp(-q) for q = -log a >= 0.
__device__ __forceinline__ float forget(float q) {
    float p = 1.f / 120.f;
    p = fmaf(p, q, -1.f / 24.f);
    p = fmaf(p, q, 1.f / 6.f);
    p = fmaf(p, q, -0.5f);
    p = fmaf(p, q, 1.f);
    return q <= kSeries ? q * p : 1.f - tc::fast_exp2(-q * kLog2e);
}

// A reset's decay is written -0: it passes nothing on, whatever stands before
// it (an infinity or a NaN times 0 would). Products of decays from a reset on
// keep the mark, as decays are >= +0.
constexpr uint32_t kResetBits = 0x80000000u;
__device__ __forceinline__ float reset_decay() { return __uint_as_float(kResetBits); }
__device__ __forceinline__ float carry_on(float a, float h, float u) {  // a h + u
    return __float_as_uint(a) == kResetBits ? u : fmaf(a, h, u);
}

__device__ __forceinline__ float chain_decay(float first, float next) {
    return __float_as_uint(next) == kResetBits ? next : first * next;
}

// One token's gate values (the step kernel).
struct Gate {
    float a, m, si;
};
__device__ __forceinline__ Gate gate(float r, float i, float k) {
    Gate g;
    float sr;
    two_sigmoids(r, i, sr, g.si);
    const float F = forget(k * sr);
    g.a = 1.f - F;
    const float m2 = fmaf(F, g.a, F) + 1e-36f;
    g.m = m2 * rsqrt_approx(m2);
    return g;
}

// The same for two channels at once in packed fp32 (half the instructions).
using tc::f2;
using tc::f2_add;
using tc::f2_fma;
using tc::f2_mul;
using tc::f2_pack;
using tc::f2_sub;
using tc::f2_unpack;

__device__ __forceinline__ f2 f2_both(float v) { return f2_pack(v, v); }

struct Gate2 {
    f2 sr, si;  // sigmoids
    f2 a;       // decay
    f2 m, rm;   // sqrt(1 - a^2) and its reciprocal (large where m = 0)
};

__device__ __forceinline__ f2 exp2_gate2(f2 v) {  // exp2(min(-v log2 e, 63))
    float lo, hi;
    f2_unpack(f2_mul(v, f2_both(-kLog2e)), lo, hi);
    return f2_pack(tc::fast_exp2(min_nan(lo, 63.f)), tc::fast_exp2(min_nan(hi, 63.f)));
}
__device__ __forceinline__ void two_sigmoids2(f2 r, f2 i, f2 &sr, f2 &si) {
    const f2 one = f2_both(1.f);
    const f2 p = f2_add(one, exp2_gate2(r)), q = f2_add(one, exp2_gate2(i));
    float lo, hi;
    f2_unpack(f2_mul(p, q), lo, hi);
    const f2 R = f2_pack(rcp_approx(lo), rcp_approx(hi));
    sr = f2_mul(q, R);
    si = f2_mul(p, R);
}
// F = 1 - exp(-q), q = -log a >= 0.
template <bool FAST>
__device__ __forceinline__ f2 forget2(f2 q) {
    f2 p = f2_both(1.f / 120.f);
    p = f2_fma(p, q, f2_both(-1.f / 24.f));
    p = f2_fma(p, q, f2_both(1.f / 6.f));
    p = f2_fma(p, q, f2_both(-0.5f));
    p = f2_fma(p, q, f2_both(1.f));
    const f2 series = f2_mul(q, p);
    if (FAST) return series;
    float f0, f1, q0, q1;
    f2_unpack(series, f0, f1);
    f2_unpack(q, q0, q1);
    return f2_pack(q0 <= kSeries ? f0 : 1.f - tc::fast_exp2(-q0 * kLog2e),
                   q1 <= kSeries ? f1 : 1.f - tc::fast_exp2(-q1 * kLog2e));
}
// a, m and 1 / m from F = 1 - a: m^2 = F (1 + a) = F + F a, kept off zero by
// 1e-36 (m = 1e-18 where a = 1).
__device__ __forceinline__ void decay_from2(f2 F, Gate2 &g) {
    g.a = f2_sub(f2_both(1.f), F);
    const f2 m2 = f2_add(f2_fma(F, g.a, F), f2_both(1e-36f));
    float lo, hi;
    f2_unpack(m2, lo, hi);
    g.rm = f2_pack(rsqrt_approx(lo), rsqrt_approx(hi));
    g.m = f2_mul(m2, g.rm);
}
template <bool FAST>
__device__ __forceinline__ Gate2 gate2(f2 r, f2 i, f2 k) {
    Gate2 g;
    two_sigmoids2(r, i, g.sr, g.si);
    decay_from2(forget2<FAST>(f2_mul(k, g.sr)), g);
    return g;
}

}  // namespace gated
}  // namespace ssd
