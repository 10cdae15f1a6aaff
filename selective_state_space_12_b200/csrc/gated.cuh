// Arithmetic of the gated linear recurrence, shared by its kernels (gated.cu).
//
// For one channel with k = c softplus(lam) >= 0, and gates r, i of a token:
//
//   q = k sigmoid(r)      a = exp(-q)      m = sqrt(1 - a^2)
//   h <- a h + m sigmoid(i) x              (a reset token: a = 0, m = 1)
//
// a is close to 1 for channels that remember long, and an error of a is
// multiplied by that memory, while of a small a the gradient of log a needs the
// leading bits. So of a and F = 1 - a the smaller is not formed from the other:
// for q <= kSeries, F is its Taylor series q (1 - q/2 + ... + q^4/120), whose
// remainder is below q^5/720 < 5e-8 relative, and a = 1 - F; above, a is exp2 of
// the special-function unit (relative error about 2^-22) and F = 1 - a > 0.11.
// m^2 = F (1 + a). The series takes no special-function operation; those bind
// these kernels beside the memory (16 a clock and SM).
#pragma once

#include "common.cuh"
#include "tc_ptx.cuh"

namespace ssd {
namespace gated {

constexpr int kBlock = 64;          // SSD_GATED_BLOCK: tokens per saved state and 8-bit scale
constexpr float kSeries = 0.125f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTiny = 1.2e-38f;   // keeps a root off zero (a normal number)

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
// softplus(lam), and sigmoid(lam) / softplus(lam) (its limit 1 where
// softplus underflows), by which the gradient of lam follows from that of log a.
__device__ __forceinline__ float softplus_full(float v) {
    return fmaxf(v, 0.f) + log1pf(expf(-fabsf(v)));
}
__device__ __forceinline__ float lam_ratio(float lam) {
    const float sp = softplus_full(lam);
    return sp > 0.f ? 1.f / ((1.f + expf(-lam)) * sp) : (lam == lam ? 1.f : lam);
}

// exp2 overflows to infinity and its reciprocal is then 0: a gate is right down to
// 2^-126 and shut below.
__device__ __forceinline__ float sigmoid(float v) {
    return rcp_approx(1.f + tc::fast_exp2(-v * kLog2e));
}

// a = exp(-q) and F = 1 - a, q >= 0.
struct Decay1 {
    float a, F;
};
__device__ __forceinline__ Decay1 decay(float q) {
    float p = 1.f / 120.f;
    p = fmaf(p, q, -1.f / 24.f);
    p = fmaf(p, q, 1.f / 6.f);
    p = fmaf(p, q, -0.5f);
    p = fmaf(p, q, 1.f);
    const float F = q * p, a = tc::fast_exp2(-q * kLog2e);
    return q <= kSeries ? Decay1{1.f - F, F} : Decay1{a, 1.f - a};
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
    const Decay1 d = decay(k * sigmoid(r));
    g.si = sigmoid(i);
    g.a = d.a;
    const float m2 = fmaf(d.F, d.a, d.F);
    g.m = m2 * rsqrt_approx(m2 + kTiny);
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

__device__ __forceinline__ f2 sigmoid2(f2 v) {
    float lo, hi;
    f2_unpack(f2_mul(v, f2_both(-kLog2e)), lo, hi);
    f2_unpack(f2_add(f2_both(1.f), f2_pack(tc::fast_exp2(lo), tc::fast_exp2(hi))), lo, hi);
    return f2_pack(rcp_approx(lo), rcp_approx(hi));
}
// sigmoid(r) and sigmoid(i) from one reciprocal: with p = 1 + exp(-r) and q = 1 + exp(-i),
// 1/p = q/(pq). Right where pq stays below kGatesTop (r + i above about -86): beyond,
// the reciprocal is flushed to 0, and the open gate with the shut one. Whoever takes it
// adds pq up in `top`, looks at that (gates_open), and takes the gates one by one where
// it is more. (Bounded exponents instead keep a masked token's m at 1e-9, which moves a
// state over a long masked stretch.)
constexpr float kGatesTop = 0x1p125f;
__device__ __forceinline__ void two_sigmoids2(f2 r, f2 i, f2 &sr, f2 &si, f2 &top) {
    float r0, r1, i0, i1;
    f2_unpack(f2_mul(r, f2_both(-kLog2e)), r0, r1);
    f2_unpack(f2_mul(i, f2_both(-kLog2e)), i0, i1);
    const f2 p = f2_add(f2_both(1.f), f2_pack(tc::fast_exp2(r0), tc::fast_exp2(r1)));
    const f2 q = f2_add(f2_both(1.f), f2_pack(tc::fast_exp2(i0), tc::fast_exp2(i1)));
    const f2 pq = f2_mul(p, q);
    top = f2_add(top, pq);
    float lo, hi;
    f2_unpack(pq, lo, hi);
    const f2 R = f2_pack(rcp_approx(lo), rcp_approx(hi));
    sr = f2_mul(q, R);
    si = f2_mul(p, R);
}
__device__ __forceinline__ bool gates_open(f2 top) {  // of the warp's; a NaN is not
    float lo, hi;
    f2_unpack(top, lo, hi);
    return __all_sync(0xffffffffu, lo < kGatesTop && hi < kGatesTop);
}
// F = 1 - exp(-q) by its series.
__device__ __forceinline__ f2 forget2(f2 q) {
    f2 p = f2_both(1.f / 120.f);
    p = f2_fma(p, q, f2_both(-1.f / 24.f));
    p = f2_fma(p, q, f2_both(1.f / 6.f));
    p = f2_fma(p, q, f2_both(-0.5f));
    p = f2_fma(p, q, f2_both(1.f));
    return f2_mul(q, p);
}
// What is not formed from the other: F where all q <= kSeries (FAST), else a.
template <bool FAST>
__device__ __forceinline__ f2 decay2(f2 q) {
    const f2 F = forget2(q);
    if (FAST) return F;
    float q0, q1, a0, a1;
    f2_unpack(q, q0, q1);
    f2_unpack(f2_sub(f2_both(1.f), F), a0, a1);
    return f2_pack(q0 <= kSeries ? a0 : tc::fast_exp2(-q0 * kLog2e),
                   q1 <= kSeries ? a1 : tc::fast_exp2(-q1 * kLog2e));
}
template <bool FAST>
__device__ __forceinline__ f2 decay_of(f2 v) {  // a from decay2's result
    return FAST ? f2_sub(f2_both(1.f), v) : v;
}
// a, m and 1 / m from decay2's result: m^2 = F (1 + a) = F + F a. Under the root it is
// kept off zero: m = 0 where a = 1, and within 1e-5 of its value from 3e-17 on.
template <bool FAST>
__device__ __forceinline__ void decay_from2(f2 v, f2 q, Gate2 &g) {
    f2 F = v;
    g.a = decay_of<FAST>(v);
    if (!FAST) {
        float q0, q1, s0, s1, d0, d1;
        f2_unpack(q, q0, q1);
        f2_unpack(forget2(q), s0, s1);
        f2_unpack(f2_sub(f2_both(1.f), v), d0, d1);
        F = f2_pack(q0 <= kSeries ? s0 : d0, q1 <= kSeries ? s1 : d1);
    }
    const f2 m2 = f2_fma(F, g.a, F);
    float lo, hi;
    f2_unpack(f2_add(m2, f2_both(kTiny)), lo, hi);
    g.rm = f2_pack(rsqrt_approx(lo), rsqrt_approx(hi));
    g.m = f2_mul(m2, g.rm);
}
// SHARED: the sigmoids by two_sigmoids2.
template <bool FAST, bool SHARED>
__device__ __forceinline__ Gate2 gate2(f2 r, f2 i, f2 k, f2 &top) {
    Gate2 g;
    if (SHARED) {
        two_sigmoids2(r, i, g.sr, g.si, top);
    } else {
        g.sr = sigmoid2(r);
        g.si = sigmoid2(i);
    }
    const f2 q = f2_mul(k, g.sr);
    decay_from2<FAST>(decay2<FAST>(q), q, g);
    return g;
}
template <bool FAST>
__device__ __forceinline__ Gate2 gate2(f2 r, f2 i, f2 k) {
    f2 unused = 0;
    return gate2<FAST, false>(r, i, k, unused);
}

}  // namespace gated
}  // namespace ssd
