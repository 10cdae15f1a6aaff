// Backward pass of the selective scan (scan.cu: diagonal A, one N-vector state
// per channel). With a = exp(dt A), w the input weight (dt, or the hold's
// (a - 1) / A) and r_t the gradient of the state h_t,
//
//   r_t = C_t dy_t + a_{t+1} r_{t+1}
//   dx  = Dskip dy + sum_n r w B        dB = sum_d r w x       dC = sum_d dy h_t
//   ddt = sum_n r a A h_{t-1} + r (dw/ddt) x B,  dw/ddt = 1 (Euler) or a (hold)
//   dA  = sum_t r dt a h_{t-1} + r (dw/dA) x B,  dw/dA  = (dt a - w) / A (hold)
//
// then ddt through the clamp (1 between its bounds, bounds included) and the
// softplus. With the hold, the state is carried as g = A h, which moves by
// E = exp(dt A) - 1 alone, without the cancellation of 1 - a:
//
//   g <- g + E (g + x B)   w = E / A   ddt = sum_n a r (g + x B)
//   dA = (1/A) sum_t [dt a r (g + x B) - r w x B]
//
// (the last difference is taken term by term, from series, where |A| < 2^-5). Every state entry takes an exponential a token and about a dozen
// fp32 operations, 16 or so times what a token's bytes need: the pass is bound
// by the arithmetic, and by keeping sums over states (dx, ddt), over channels
// (dB, dC) and over tokens (dA) all in registers.
//
// Time is cut into chunks of 64 tokens that run side by side:
//   1. scan_bwd_sums: each chunk's end state from a zero state, and the
//      gradient it hands to its left when none comes from its right;
//   2. scan_bwd_chain: the chains over chunks, forward and backward, leaving
//      the state entering each chunk and the gradient entering it from its right;
//   3. scan_bwd_main: the same again inside a chunk over its 16 pieces of four
//      tokens (a warp each), then each piece's states forward and gradients
//      back, from registers;
//   4. sums of dB and dC over blocks of channels, and of dA, dDskip and the
//      bias's gradient over batch and chunks. No atomics: every sum has one order.
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace ssd {
namespace {

constexpr float kLog2eB = 1.4426950408889634f;
constexpr int kChunk = 64;               // tokens of a chunk
constexpr int kPiece = 4;                // tokens of a piece
constexpr int kPieces = kChunk / kPiece;  // = warps of the main kernel
constexpr int kCh = 32;                  // channels of a tile
constexpr int kQ = 4;                    // states of a thread
constexpr int kRow = kChunk + 4;         // floats of a channel's row of tokens in shared memory
constexpr int kMainThreads = 32 * kPieces;

// Step preparation with its derivative. A step's side of the clamp's bounds is
// all or nothing for its gradient, so raw + bias is compared with the bounds'
// preimages under the softplus, both sums carried in two floats.
struct StepArgs {
    DtPreArgs pre;
    int on;               // any of bias, softplus, clamp
    float lo[2], hi[2];   // preimages of the bounds: value and remainder
};

__device__ __forceinline__ float div_approx(float a, float b) {
    float y;
    asm("div.approx.ftz.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// log(1 + e), e in [0, 1], as 2 atanh(z), z = e / (2 + e) <= 1/3: the series
// to z^13 (the next term is below 2 z^15 / 15 < 1e-8 relative to z).
__device__ __forceinline__ float log1p_unit(float e) {
    const float z = div_approx(e, 2.f + e), q = z * z;
    float p = 1.f / 13.f;
    p = fmaf(p, q, 1.f / 11.f);
    p = fmaf(p, q, 1.f / 9.f);
    p = fmaf(p, q, 1.f / 7.f);
    p = fmaf(p, q, 1.f / 5.f);
    p = fmaf(p, q, 1.f / 3.f);
    p = fmaf(p, q, 1.f);
    return 2.f * z * p;
}

// The prepared step, and d(step)/d(raw) where GRAD.
template <bool GRAD>
__device__ __forceinline__ float prepare_step(float raw, float bias, const StepArgs &s,
                                              float &slope) {
    if (GRAD) slope = 1.f;
    if (!s.on) return raw;
    const float v = raw + bias;
    float dt = v;
    if (s.pre.softplus) {
        const float e = tc::fast_exp2(-fabsf(v) * kLog2eB);
        dt = (v > 0.f ? v : 0.f) + log1p_unit(e);
        if (v != v) dt = v;
        if (GRAD) slope = div_approx(v >= 0.f ? 1.f : e, 1.f + e);
    }
    if (s.pre.dt_max > 0.f) {
        dt = fminf(fmaxf(dt, s.pre.dt_min), s.pre.dt_max);
        if (GRAD) {
            const float bb = v - raw;  // the sum's remainder
            const float rest = (raw - (v - bb)) + (bias - bb);
            const bool in = (v - s.lo[0]) + (rest - s.lo[1]) >= 0.f &&
                            (s.hi[0] - v) + (s.hi[1] - rest) >= 0.f;
            if (!in) slope = 0.f;
        }
    }
    return dt;
}

// One pair of state entries at one step: F is exp(dt A) (Euler) or
// E = exp(dt A) - 1 (hold), the latter by its series where |z| < 1/4, z = dt A
// (remainder below z^6 / 5040 < 5e-8 relative), else from exp2, whose error of
// 2^-22 is then at most 1e-6 of it.
using tc::f2;
using tc::f2_add;
using tc::f2_fma;
using tc::f2_mul;
using tc::f2_pack;
using tc::f2_sub;
using tc::f2_unpack;
__device__ __forceinline__ f2 f2_both(float v) { return f2_pack(v, v); }

template <bool ZOH>
struct Decay {
    f2 A, Al;  // A (hold: kept off zero) and A log2 e
    __device__ __forceinline__ f2 at(f2 dt) const {
        float z0, z1, l0, l1;
        f2_unpack(f2_mul(dt, Al), l0, l1);
        const f2 e = f2_pack(tc::fast_exp2(l0), tc::fast_exp2(l1));
        if (!ZOH) return e;
        const f2 z = f2_mul(dt, A);
        f2 p = f2_fma(f2_both(1.f / 720.f), z, f2_both(1.f / 120.f));
        p = f2_fma(p, z, f2_both(1.f / 24.f));
        p = f2_fma(p, z, f2_both(1.f / 6.f));
        p = f2_fma(p, z, f2_both(0.5f));
        p = f2_fma(p, z, f2_both(1.f));
        float s0, s1, e0, e1;
        f2_unpack(f2_mul(z, p), s0, s1);
        f2_unpack(f2_add(e, f2_both(-1.f)), e0, e1);
        f2_unpack(z, z0, z1);
        return f2_pack(fabsf(z0) < 0.25f ? s0 : e0, fabsf(z1) < 0.25f ? s1 : e1);
    }
};

// A as the hold uses it: |A| >= 2^-40, which changes no result by more than
// 2^-40 a token and lets g = A h carry the state of A = 0 too.
__device__ __forceinline__ float off_zero(float A) {
    return fabsf(A) < 0x1p-40f ? (A > 0.f ? 0x1p-40f : -0x1p-40f) : A;
}

struct BwdArgs {
    const void *x, *dt, *B, *C, *dy;
    const float *A, *Dskip;
    float *dx, *ddt, *dB, *dC;
    float *S, *R;        // (b, nc, D, N): per-chunk sums, then what enters each chunk
    float *steps;        // (b, nc, D): sum of the chunk's steps
    float *bc_part;      // (parts, b, L, N, 2) by group: dB and dC of a block of channels
    float *dA_part;      // (b, nc, D, N)
    float *d_part;       // (b, nc, D, 2): dDskip, dbias
    int64_t batch, L, D, G, nc;
    int64_t gch;         // channels of a group
    int tiles_per_group, tiles_per_block, blocks_per_group;
    StepArgs step;
};

// Shared memory of the staged tile, in floats.
template <int N>
struct __align__(16) Tile {
    static constexpr int kState = kCh * N;
    float x[kCh][kRow], dt[kCh][kRow], dy[kCh][kRow];
    float B[kChunk][N], C[kChunk][N];
};
template <int N>
struct MainTile : Tile<N> {
    float fac[kCh][kRow], dx[kCh][kRow];
    float S[kPieces][Tile<N>::kState], R[kPieces][Tile<N>::kState], P[kPieces][Tile<N>::kState];
};

struct Place {
    int64_t b, chunk, g;
    int part, tile0, tiles;  // tiles of channels [tile0, tile0 + tiles) of the group
    int64_t t0;
    int n;  // tokens
};
__device__ __forceinline__ Place place(const BwdArgs &a) {
    Place p;
    int64_t i = blockIdx.x;
    p.part = (int)(i % a.blocks_per_group);
    i /= a.blocks_per_group;
    p.g = i % a.G;
    i /= a.G;
    p.chunk = i % a.nc;
    p.b = i / a.nc;
    p.tile0 = p.part * a.tiles_per_block;
    p.tiles = min(a.tiles_per_block, a.tiles_per_group - p.tile0);
    p.t0 = p.chunk * kChunk;
    p.n = (int)(a.L - p.t0 < kChunk ? a.L - p.t0 : kChunk);
    return p;
}

// x, dt (prepared) and dy of a tile of channels as floats, tokens along a
// row; channels and tokens past the end are zeros (dt = 0: a = 1, w = 0).
template <typename T, int N, bool GRAD, int THREADS>
__device__ __forceinline__ void stage_channels(const BwdArgs &a, const Place &p, int64_t d0,
                                               int64_t dend, Tile<N> &s, float (*fac)[kRow]) {
    const T *x = static_cast<const T *>(a.x), *dt = static_cast<const T *>(a.dt),
            *dy = static_cast<const T *>(a.dy);
    const int c = threadIdx.x % kCh;
    const bool has = d0 + c < dend;
    const float bias = (has && a.step.pre.bias) ? a.step.pre.bias[d0 + c] : 0.f;
    const int64_t base = (p.b * a.L + p.t0) * a.D + d0 + c;
    for (int t = threadIdx.x / kCh; t < kChunk; t += THREADS / kCh) {
        float xv = 0.f, dv = 0.f, yv = 0.f, f = 0.f;
        if (has && t < p.n) {
            const int64_t off = base + t * a.D;
            xv = to_f(x[off]);
            yv = to_f(dy[off]);
            dv = prepare_step<GRAD>(to_f(dt[off]), bias, a.step, f);
        }
        s.x[c][t] = xv;
        s.dt[c][t] = dv;
        s.dy[c][t] = yv;
        if (GRAD) fac[c][t] = f;
    }
}
template <typename T, int N, int THREADS>
__device__ __forceinline__ void stage_rows(const BwdArgs &a, const Place &p, Tile<N> &s) {
    const T *B = static_cast<const T *>(a.B), *C = static_cast<const T *>(a.C);
    for (int i = threadIdx.x; i < kChunk * N; i += THREADS) {
        const int t = i / N, n = i % N;
        float bv = 0.f, cv = 0.f;
        if (t < p.n) {
            const int64_t off = ((p.b * a.L + p.t0 + t) * a.G + p.g) * N + n;
            bv = to_f(B[off]);
            cv = to_f(C[off]);
        }
        s.B[t][n] = bv;
        s.C[t][n] = cv;
    }
}

__device__ __forceinline__ void load4x(const float *p, f2 (&v)[2]) {
    const float4 q = *reinterpret_cast<const float4 *>(p);
    v[0] = f2_pack(q.x, q.y);
    v[1] = f2_pack(q.z, q.w);
}
__device__ __forceinline__ void store4x(float *p, const f2 (&v)[2]) {
    float4 q;
    f2_unpack(v[0], q.x, q.y);
    f2_unpack(v[1], q.z, q.w);
    *reinterpret_cast<float4 *>(p) = q;
}

// One token's move of the state: s <- a s + w x B, or with the hold g.
template <bool ZOH>
__device__ __forceinline__ f2 move(f2 F, f2 s, f2 in) {
    return ZOH ? f2_fma(F, f2_add(s, in), s) : f2_fma(F, s, in);
}
template <bool ZOH>
__device__ __forceinline__ f2 times_decay(f2 v, f2 F) {
    return ZOH ? f2_fma(v, F, v) : f2_mul(v, F);
}

// The map of a run of tokens for one thread's four states: end state S from
// zero, gradient R handed to the left when none comes from the right, product P.
template <int N, bool ZOH, int TOKENS>
__device__ __forceinline__ void run_sums(const Tile<N> &s, int c, int t0, int n0,
                                         const Decay<ZOH> (&A)[2], f2 (&S)[2], f2 (&R)[2],
                                         f2 (&P)[2]) {
#pragma unroll
    for (int k = 0; k < 2; ++k) S[k] = R[k] = f2_both(0.f), P[k] = f2_both(1.f);
#pragma unroll 1
    for (int t4 = t0; t4 < t0 + TOKENS; t4 += 4) {
        const float4 x4 = *reinterpret_cast<const float4 *>(&s.x[c][t4]);
        const float4 d4 = *reinterpret_cast<const float4 *>(&s.dt[c][t4]);
        const float4 y4 = *reinterpret_cast<const float4 *>(&s.dy[c][t4]);
        const float xs[4] = {x4.x, x4.y, x4.z, x4.w}, ds[4] = {d4.x, d4.y, d4.z, d4.w},
                    ys[4] = {y4.x, y4.y, y4.z, y4.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const f2 in = f2_both(ZOH ? xs[j] : xs[j] * ds[j]), dt = f2_both(ds[j]),
                     dy = f2_both(ys[j]);
            f2 B[2], C[2];
            load4x(&s.B[t4 + j][n0], B);
            load4x(&s.C[t4 + j][n0], C);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const f2 F = A[k].at(dt);
                S[k] = move<ZOH>(F, S[k], f2_mul(in, B[k]));
                P[k] = times_decay<ZOH>(P[k], F);
                R[k] = f2_fma(P[k], f2_mul(dy, C[k]), R[k]);
            }
        }
    }
}

// A of a thread's states, 1 / A and whether any is too near zero for the
// plain form of the hold's dA.
template <int N, bool ZOH>
__device__ __forceinline__ bool load_A(const BwdArgs &a, int64_t d, int n0, Decay<ZOH> (&A)[2],
                                       f2 (&raw)[2], f2 (&invA)[2]) {
    float v[kQ];
    bool tiny = false;
#pragma unroll
    for (int k = 0; k < kQ; ++k) {
        v[k] = a.A[d * N + n0 + k];
        if (ZOH) v[k] = off_zero(v[k]);
        tiny = tiny || fabsf(v[k]) < 0x1p-5f;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        raw[k] = A[k].A = f2_pack(v[2 * k], v[2 * k + 1]);
        A[k].Al = f2_mul(A[k].A, f2_both(kLog2eB));
        invA[k] = ZOH ? f2_pack(1.f / v[2 * k], 1.f / v[2 * k + 1]) : 0;
    }
    return ZOH && tiny;
}

template <typename T, int N, bool ZOH>
__global__ void __launch_bounds__(kCh *N / kQ) scan_bwd_sums(const BwdArgs a) {
    constexpr int kThreads = kCh * N / kQ, kLanes = N / kQ;
    extern __shared__ __align__(16) unsigned char raw[];
    Tile<N> &s = *reinterpret_cast<Tile<N> *>(raw);
    const Place p = place(a);
    const int64_t dend = (p.g + 1) * a.gch;
    stage_rows<T, N, kThreads>(a, p, s);
    for (int k = 0; k < p.tiles; ++k) {
        const int64_t d0 = p.g * a.gch + (int64_t)(p.tile0 + k) * kCh;
        __syncthreads();
        stage_channels<T, N, false, kThreads>(a, p, d0, dend, s, nullptr);
        __syncthreads();
        const int c = threadIdx.x / kLanes, n0 = (threadIdx.x % kLanes) * kQ;
        const bool has = d0 + c < dend;
        const int64_t d = has ? d0 + c : dend - 1;
        Decay<ZOH> A[2];
        f2 v[2], invA[2], S[2], R[2], P[2];
        load_A<N, ZOH>(a, d, n0, A, v, invA);
        run_sums<N, ZOH, kChunk>(s, c, 0, n0, A, S, R, P);
        if (has) {
            const int64_t at = (p.b * a.nc + p.chunk) * a.D + d;
            store4x(&a.S[at * N + n0], S);
            store4x(&a.R[at * N + n0], R);
            if (n0 == 0) {
                float sum = 0.f;
                for (int t = 0; t < kChunk; ++t) sum += s.dt[c][t];
                a.steps[at] = sum;
            }
        }
    }
}

// The chains over chunks: blockIdx.y 0 the states (with the hold g = A h), 1
// the gradients. Eight chunks' words are loaded at a time.
template <int N, bool ZOH>
__global__ void __launch_bounds__(128)
scan_bwd_chain(const BwdArgs a, const float *h0, const float *dh_final, float *dh0) {
    constexpr int kBatch = 8;
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t lane_len = a.D * N;
    if (i >= a.batch * lane_len) return;
    const int64_t b = i / lane_len, dn = i % lane_len;
    const bool back = blockIdx.y == 1;
    float A = a.A[dn];
    if (ZOH) A = off_zero(A);
    const float Al = A * kLog2eB;
    const float *first = back ? dh_final : h0;
    const int64_t way = back ? -1 : 1, c0 = b * a.nc + (back ? a.nc - 1 : 0);
    float *S = (back ? a.R : a.S) + c0 * lane_len + dn;
    const float *steps = a.steps + c0 * a.D + dn / N;
    float h = first ? first[i] : 0.f;
    if (ZOH && !back) h *= A;
    for (int64_t j0 = 0; j0 < a.nc; j0 += kBatch) {
        float v[kBatch], t[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const bool has = j0 + j < a.nc;
            v[j] = has ? S[way * (j0 + j) * lane_len] : 0.f;
            t[j] = has ? steps[way * (j0 + j) * a.D] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            if (j0 + j >= a.nc) break;
            S[way * (j0 + j) * lane_len] = h;
            h = fmaf(tc::fast_exp2(t[j] * Al), h, v[j]);
        }
    }
    if (back && dh0) dh0[i] = h;
}

// Sum over the lanes of a channel (LANES a power of two), result in all.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sums of the piece's four values over a channel's LANES lanes: with 4 lanes,
// lane i ends with token i's, with 2 lane i with those of tokens 2i and 2i + 1.
template <int LANES>
__device__ __forceinline__ void share_sums(float (&u)[kPiece], float (&v)[kPiece], int lane) {
    if constexpr (LANES == 4) {
        const bool up = lane & 2;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float su = up ? u[j] : u[j + 2], sv = up ? v[j] : v[j + 2];
            u[j] = (up ? u[j + 2] : u[j]) + __shfl_xor_sync(0xffffffffu, su, 2);
            v[j] = (up ? v[j + 2] : v[j]) + __shfl_xor_sync(0xffffffffu, sv, 2);
        }
        const bool odd = lane & 1;
        const float su = odd ? u[0] : u[1], sv = odd ? v[0] : v[1];
        u[0] = (odd ? u[1] : u[0]) + __shfl_xor_sync(0xffffffffu, su, 1);
        v[0] = (odd ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, sv, 1);
    } else if constexpr (LANES == 2) {
        const bool up = lane & 1;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float su = up ? u[j] : u[j + 2], sv = up ? v[j] : v[j + 2];
            u[j] = (up ? u[j + 2] : u[j]) + __shfl_xor_sync(0xffffffffu, su, 1);
            v[j] = (up ? v[j + 2] : v[j]) + __shfl_xor_sync(0xffffffffu, sv, 1);
        }
    }
}

// The hold's dw/dA = (dt e^z - w) / A of a pair, for A near zero: with
// phi1 = (e^z - 1) / z and phi2 = (phi1 - 1) / z it is dt^2 (phi1 - phi2),
// where |z| < 1/4 from the series of phi2 (remainder below z^5/5040 < 2e-7).
__device__ __forceinline__ f2 slope(float dt, f2 A, f2 invA, f2 E) {
    float a[2], i[2], e[2], r[2];
    f2_unpack(A, a[0], a[1]);
    f2_unpack(invA, i[0], i[1]);
    f2_unpack(E, e[0], e[1]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float z = dt * a[k];
        float phi2 = 1.f / 720.f;
        phi2 = fmaf(phi2, z, 1.f / 120.f);
        phi2 = fmaf(phi2, z, 1.f / 24.f);
        phi2 = fmaf(phi2, z, 1.f / 6.f);
        phi2 = fmaf(phi2, z, 0.5f);
        r[k] = fabsf(z) < 0.25f ? dt * dt * (fmaf(z, phi2, 1.f) - phi2)
                                : (fmaf(dt, e[k], dt) - e[k] * i[k]) * i[k];
    }
    return f2_pack(r[0], r[1]);
}

template <typename T, int N, bool ZOH>
__global__ void __launch_bounds__(kMainThreads, 1) scan_bwd_main(const BwdArgs a) {
    constexpr int kLanes = N / kQ, kPerWarp = 32 / kLanes, kState = kCh * N;
    extern __shared__ __align__(16) unsigned char raw[];
    MainTile<N> &s = *reinterpret_cast<MainTile<N> *>(raw);
    const Place p = place(a);
    const int64_t dend = (p.g + 1) * a.gch;
    const int tid = threadIdx.x, lane = tid & 31, piece = tid >> 5;
    const int n0 = (lane % kLanes) * kQ, t0 = piece * kPiece;
    const f2 none = f2_both(0.f);
    f2 accB[kPiece][2], accC[kPiece][2];
#pragma unroll
    for (int t = 0; t < kPiece; ++t)
#pragma unroll
        for (int k = 0; k < 2; ++k) accB[t][k] = accC[t][k] = none;
    stage_rows<T, N, kMainThreads>(a, p, s);
    for (int tile = 0; tile < p.tiles; ++tile) {
        const int64_t d0 = p.g * a.gch + (int64_t)(p.tile0 + tile) * kCh;
        const int64_t row = (p.b * a.nc + p.chunk) * a.D;
        __syncthreads();
        stage_channels<T, N, true, kMainThreads>(a, p, d0, dend, s, s.fac);
        // this thread's state of the chain over pieces
        float h = 0.f, r = 0.f;
        const bool chain = tid < kState && d0 + tid / N < dend;
        if (chain) {
            h = a.S[(row + d0) * N + tid];
            r = a.R[(row + d0) * N + tid];
        }
        __syncthreads();
#pragma unroll 1
        for (int c = lane / kLanes; c < kCh; c += kPerWarp) {
            Decay<ZOH> A[2];
            f2 v[2], invA[2], S[2], R[2], P[2];
            load_A<N, ZOH>(a, d0 + c < dend ? d0 + c : dend - 1, n0, A, v, invA);
            run_sums<N, ZOH, kPiece>(s, c, t0, n0, A, S, R, P);
            store4x(&s.S[piece][c * N + n0], S);
            store4x(&s.R[piece][c * N + n0], R);
            store4x(&s.P[piece][c * N + n0], P);
        }
        __syncthreads();
        if (tid < kState) {
#pragma unroll 4
            for (int j = 0; j < kPieces; ++j) {
                const float v = s.S[j][tid];
                s.S[j][tid] = h;
                h = fmaf(s.P[j][tid], h, v);
            }
#pragma unroll 4
            for (int j = kPieces - 1; j >= 0; --j) {
                const float v = s.R[j][tid];
                s.R[j][tid] = r;
                r = fmaf(s.P[j][tid], r, v);
            }
        }
        __syncthreads();
#pragma unroll 1
        for (int c = lane / kLanes; c < kCh; c += kPerWarp) {
            const int64_t d = d0 + c < dend ? d0 + c : dend - 1;
            Decay<ZOH> A[2];
            f2 An[2], invA[2], st[2], carry[2], dA[2], dA2[2], F[kPiece][2], before[kPiece][2];
            const bool tiny = load_A<N, ZOH>(a, d, n0, A, An, invA);
            const float Ds = a.Dskip ? a.Dskip[d] : 0.f;
            load4x(&s.S[piece][c * N + n0], st);
            load4x(&s.R[piece][c * N + n0], carry);
            const float4 x4 = *reinterpret_cast<const float4 *>(&s.x[c][t0]);
            const float4 d4 = *reinterpret_cast<const float4 *>(&s.dt[c][t0]);
            const float4 y4 = *reinterpret_cast<const float4 *>(&s.dy[c][t0]);
            const float xs[kPiece] = {x4.x, x4.y, x4.z, x4.w}, ds[kPiece] = {d4.x, d4.y, d4.z, d4.w},
                        ys[kPiece] = {y4.x, y4.y, y4.z, y4.w};
#pragma unroll
            for (int t = 0; t < kPiece; ++t) {
                const f2 in = f2_both(ZOH ? xs[t] : xs[t] * ds[t]), dt = f2_both(ds[t]),
                         dy = f2_both(ys[t]);
                f2 B[2];
                load4x(&s.B[t0 + t][n0], B);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    F[t][k] = A[k].at(dt);
                    before[t][k] = st[k];
                    st[k] = move<ZOH>(F[t][k], st[k], f2_mul(in, B[k]));
                    const f2 h = ZOH ? f2_mul(st[k], invA[k]) : st[k];
                    accC[t][k] = f2_fma(dy, h, accC[t][k]);
                }
            }
            float vB[kPiece], vA[kPiece];
#pragma unroll
            for (int k = 0; k < 2; ++k) dA[k] = dA2[k] = none;
            auto back = [&](auto near_zero) {
#pragma unroll
                for (int t = kPiece - 1; t >= 0; --t) {
                    const f2 x = f2_both(xs[t]), dt = f2_both(ds[t]), dy = f2_both(ys[t]),
                             u = f2_both(xs[t] * ds[t]);
                    f2 B[2], C[2], sB = none, sA = none;
                    load4x(&s.B[t0 + t][n0], B);
                    load4x(&s.C[t0 + t][n0], C);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const f2 rv = f2_fma(dy, C[k], carry[k]);
                        const f2 ra = times_decay<ZOH>(rv, F[t][k]);
                        if (ZOH) {
                            const f2 rw = f2_mul(rv, f2_mul(F[t][k], invA[k]));
                            const f2 in = f2_mul(x, B[k]);
                            const f2 rt = f2_mul(ra, f2_add(before[t][k], in));
                            sB = f2_fma(rw, B[k], sB);
                            accB[t][k] = f2_fma(rw, x, accB[t][k]);
                            sA = f2_add(sA, rt);
                            if constexpr (decltype(near_zero)::value) {
                                // term by term: dt a r h + r x B dw/dA
                                dA[k] = f2_fma(f2_mul(ra, dt), f2_mul(before[t][k], invA[k]), dA[k]);
                                dA2[k] = f2_fma(f2_mul(rv, in), slope(ds[t], An[k], invA[k], F[t][k]),
                                                dA2[k]);
                            } else {
                                dA[k] = f2_fma(dt, rt, dA[k]);
                                dA2[k] = f2_fma(rw, in, dA2[k]);
                            }
                        } else {
                            const f2 t1 = f2_mul(ra, before[t][k]);
                            sB = f2_fma(rv, B[k], sB);
                            accB[t][k] = f2_fma(rv, u, accB[t][k]);
                            sA = f2_fma(An[k], t1, sA);
                            dA[k] = f2_fma(dt, t1, dA[k]);
                        }
                        carry[k] = ra;
                    }
                    float lo, hi;
                    f2_unpack(sB, lo, hi);
                    vB[t] = lo + hi;
                    f2_unpack(sA, lo, hi);
                    vA[t] = lo + hi;
                }
            };
            if (__any_sync(0xffffffffu, tiny)) {
                back(std::true_type{});
#pragma unroll
                for (int k = 0; k < 2; ++k) dA[k] = f2_add(dA[k], dA2[k]);
            } else {
                back(std::false_type{});
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    if (ZOH) dA[k] = f2_mul(invA[k], f2_sub(dA[k], dA2[k]));
            }
            // dx and ddt: each lane of the channel ends with the sums of its share of the tokens
            share_sums<kLanes>(vB, vA, lane);
            constexpr int kShare = kPiece / kLanes;
#pragma unroll
            for (int j = 0; j < kShare; ++j) {
                const int t = t0 + (lane % kLanes) * kShare + j;
                const float sB = vB[j], sA = vA[j];
                s.dx[c][t] = fmaf(Ds, s.dy[c][t], ZOH ? sB : sB * s.dt[c][t]);
                s.fac[c][t] *= ZOH ? sA : fmaf(s.x[c][t], sB, sA);  // ddt
            }
            store4x(&s.P[piece][c * N + n0], dA);
        }
        __syncthreads();
        if (chain) {
            float v = 0.f;
#pragma unroll
            for (int j = 0; j < kPieces; ++j) v += s.P[j][tid];
            a.dA_part[(row + d0) * N + tid] = v;
        }
        for (int i = tid; i < kChunk * kCh; i += kMainThreads) {
            const int t = i / kCh, c = i % kCh;
            if (t < p.n && d0 + c < dend) {
                const int64_t off = (p.b * a.L + p.t0 + t) * a.D + d0 + c;
                a.dx[off] = s.dx[c][t];
                a.ddt[off] = s.fac[c][t];
            }
        }
        // sums over the chunk's tokens: 16 lanes a channel
        {
            const int c = tid / 16, q = tid % 16;
            float dd = 0.f, db = 0.f;
            for (int t = q; t < kChunk; t += 16) {
                dd = fmaf(s.x[c][t], s.dy[c][t], dd);
                db += t < p.n ? s.fac[c][t] : 0.f;
            }
            dd = lanes_sum<16>(dd);
            db = lanes_sum<16>(db);
            if (q == 0 && d0 + c < dend) {
                a.d_part[(row + d0 + c) * 2] = dd;
                a.d_part[(row + d0 + c) * 2 + 1] = db;
            }
        }
    }
    // dB and dC of these channels: summed over the warp's channel lanes
#pragma unroll
    for (int t = 0; t < kPiece; ++t)
#pragma unroll
        for (int k = 0; k < kQ; ++k) {
            float b0, b1, c0, c1;
            f2_unpack(accB[t][k / 2], b0, b1);
            f2_unpack(accC[t][k / 2], c0, c1);
            float vb = k & 1 ? b1 : b0, vc = k & 1 ? c1 : c0;
#pragma unroll
            for (int o = kLanes; o < 32; o <<= 1) {
                vb += __shfl_xor_sync(0xffffffffu, vb, o);
                vc += __shfl_xor_sync(0xffffffffu, vc, o);
            }
            if (lane < kLanes && t0 + t < p.n) {
                const int64_t at =
                    (((int64_t)p.part * a.batch + p.b) * a.L + p.t0 + t0 + t) * a.G + p.g;
                a.bc_part[(at * N + n0 + k) * 2] = vb;
                a.bc_part[(at * N + n0 + k) * 2 + 1] = vc;
            }
        }
}

// dB and dC: the sum over blocks of channels.
__global__ void scan_bwd_rows(const float2 *__restrict__ part, float *__restrict__ dB,
                              float *__restrict__ dC, int parts, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= n) return;
    float b = 0.f, c = 0.f;
    for (int j = 0; j < parts; ++j) {
        const float2 v = part[j * n + i];
        b += v.x;
        c += v.y;
    }
    dB[i] = b;
    dC[i] = c;
}

// Sums over batch and chunks of rows of `width` floats; out2 takes the odd
// columns where given.
__global__ void scan_bwd_params(const float *__restrict__ part, float *__restrict__ out,
                                float *__restrict__ out2, bool pairs, int64_t rows, int64_t width) {
    __shared__ float red[8][33];
    const int64_t i = (int64_t)blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    if (i < width)
        for (int64_t j = threadIdx.y; j < rows; j += 8) s += part[j * width + i];
    red[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && i < width) {
        for (int j = 1; j < 8; ++j) s += red[j][threadIdx.x];
        float *to = pairs ? ((i & 1) ? out2 : out) : out;
        if (to) to[pairs ? i / 2 : i] = s;
    }
}

int64_t chunks(const Problem &pr) { return (pr.seqlen + kChunk - 1) / kChunk; }

// Tiles of channels that one CUDA block of the main kernel walks: as many as
// leave four blocks for each SM, up to eight (fewer sums of dB and dC).
void split(const Problem &pr, BwdArgs &a) {
    a.gch = pr.nheads / pr.ngroups;
    a.tiles_per_group = (int)((a.gch + kCh - 1) / kCh);
    const int64_t rows = pr.batch * chunks(pr) * pr.ngroups;
    int k = 8;
    while (k > 1 && rows * ((a.tiles_per_group + k - 1) / k) < 4 * 148) --k;
    a.tiles_per_block = k;
    a.blocks_per_group = (a.tiles_per_group + k - 1) / k;
}

struct Carved {
    size_t S, R, steps, bc, dA, d, total;
};
Carved carve(const Problem &pr, const BwdArgs &a) {
    Carved c;
    const size_t lanes = (size_t)(pr.batch * chunks(pr) * pr.nheads), N = (size_t)pr.dstate;
    size_t at = 0;
    auto take = [&](size_t floats) {
        const size_t here = at;
        at += align256(floats * 4);
        return here;
    };
    c.S = take(lanes * N);
    c.R = take(lanes * N);
    c.steps = take(lanes);
    c.bc = take((size_t)a.blocks_per_group * (size_t)(pr.batch * pr.seqlen * pr.ngroups) * N * 2);
    c.dA = take(lanes * N);
    c.d = take(lanes * 2);
    c.total = at;
    return c;
}

template <typename T, int N, bool ZOH>
cudaError_t launch(const Problem &pr, BwdArgs a, const float *h0, const float *dh_final,
                   float *dA, float *dD, float *ddt_bias, float *dh0, cudaStream_t st) {
    cudaError_t e;
    const unsigned grid = (unsigned)(a.batch * a.nc * a.G * a.blocks_per_group);
    const int sums_smem = (int)sizeof(Tile<N>), main_smem = (int)sizeof(MainTile<N>);
    if ((e = cudaFuncSetAttribute(scan_bwd_sums<T, N, ZOH>,
                                  cudaFuncAttributeMaxDynamicSharedMemorySize, sums_smem)) !=
            cudaSuccess ||
        (e = cudaFuncSetAttribute(scan_bwd_main<T, N, ZOH>,
                                  cudaFuncAttributeMaxDynamicSharedMemorySize, main_smem)) !=
            cudaSuccess)
        return e;
    launch_begin("scan_bwd_sums", st);
    scan_bwd_sums<T, N, ZOH><<<grid, kCh * N / kQ, sums_smem, st>>>(a);
    launch_end(st);
    const int64_t lanes = a.batch * a.D * N;
    launch_begin("scan_bwd_chain", st);
    scan_bwd_chain<N, ZOH><<<dim3((unsigned)((lanes + 127) / 128), 2), 128, 0, st>>>(a, h0, dh_final,
                                                                                    dh0);
    launch_end(st);
    launch_begin("scan_bwd_main", st);
    scan_bwd_main<T, N, ZOH><<<grid, kMainThreads, main_smem, st>>>(a);
    launch_end(st);
    const int64_t n = a.batch * a.L * a.G * N;
    launch_begin("scan_bwd_rows", st);
    scan_bwd_rows<<<(unsigned)((n + 127) / 128), 128, 0, st>>>(
        reinterpret_cast<const float2 *>(a.bc_part), a.dB, a.dC, a.blocks_per_group, n);
    launch_end(st);
    launch_begin("scan_bwd_params", st);
    scan_bwd_params<<<(unsigned)((a.D * N + 31) / 32), dim3(32, 8), 0, st>>>(
        a.dA_part, dA, nullptr, false, a.batch * a.nc, a.D * N);
    launch_end(st);
    launch_begin("scan_bwd_params", st);
    scan_bwd_params<<<(unsigned)((2 * a.D + 31) / 32), dim3(32, 8), 0, st>>>(
        a.d_part, dD, ddt_bias, true, a.batch * a.nc, 2 * a.D);
    launch_end(st);
    return cudaGetLastError();
}

template <typename T, int N>
cudaError_t launch_n(const Problem &pr, const BwdArgs &a, bool zoh, const float *h0,
                     const float *dh_final, float *dA, float *dD, float *ddt_bias, float *dh0,
                     cudaStream_t st) {
    return zoh ? launch<T, N, true>(pr, a, h0, dh_final, dA, dD, ddt_bias, dh0, st)
               : launch<T, N, false>(pr, a, h0, dh_final, dA, dD, ddt_bias, dh0, st);
}

template <typename T>
cudaError_t launch_t(const Problem &pr, const BwdArgs &a, bool zoh, const float *h0,
                     const float *dh_final, float *dA, float *dD, float *ddt_bias, float *dh0,
                     cudaStream_t st) {
    switch (pr.dstate) {
        case 4: return launch_n<T, 4>(pr, a, zoh, h0, dh_final, dA, dD, ddt_bias, dh0, st);
        case 8: return launch_n<T, 8>(pr, a, zoh, h0, dh_final, dA, dD, ddt_bias, dh0, st);
        default: return launch_n<T, 16>(pr, a, zoh, h0, dh_final, dA, dD, ddt_bias, dh0, st);
    }
}

// The value that softplus takes to v (minus infinity for v = 0), as two floats.
void softplus_preimage(double v, float (&out)[2]) {
    const double u = v > 30.0 ? v + log1p(-exp(-v)) : log(expm1(v));
    out[0] = (float)u;
    out[1] = isinf(out[0]) ? 0.f : (float)(u - (double)out[0]);
}

}  // namespace

size_t scan_backward_workspace_bytes(const Problem &pr) {
    BwdArgs a;
    split(pr, a);
    return carve(pr, a).total;
}

ssd_status scan_backward_launch(const Problem &pr, const void *x, const void *dt, const float *A,
                                const void *B, const void *C, const float *Dskip, const float *h0,
                                const void *dy, const float *dh_final, float *dx, float *ddt,
                                float *dA, float *dB, float *dC, float *dD, float *ddt_bias,
                                float *dh0, void *ws, const DtPre &pre, cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    if (pr.seqlen == 0) {
        const size_t lanes = (size_t)(pr.batch * pr.nheads * pr.dstate) * 4;
        e = cudaMemsetAsync(dA, 0, (size_t)(pr.nheads * pr.dstate) * 4, st);
        if (e == cudaSuccess && dD) e = cudaMemsetAsync(dD, 0, (size_t)pr.nheads * 4, st);
        if (e == cudaSuccess && ddt_bias)
            e = cudaMemsetAsync(ddt_bias, 0, (size_t)pr.nheads * 4, st);
        if (e == cudaSuccess && dh0 && dh_final && dh0 != dh_final)
            e = cudaMemcpyAsync(dh0, dh_final, lanes, cudaMemcpyDeviceToDevice, st);
        else if (e == cudaSuccess && dh0 && !dh_final)
            e = cudaMemsetAsync(dh0, 0, lanes, st);
        return e == cudaSuccess ? SSD_OK : cuda_fail(e, "selective scan backward");
    }
    BwdArgs a;
    split(pr, a);
    const Carved c = carve(pr, a);
    char *w = static_cast<char *>(ws);
    a.x = x;
    a.dt = dt;
    a.B = B;
    a.C = C;
    a.dy = dy;
    a.A = A;
    a.Dskip = Dskip;
    a.dx = dx;
    a.ddt = ddt;
    a.dB = dB;
    a.dC = dC;
    a.S = reinterpret_cast<float *>(w + c.S);
    a.R = reinterpret_cast<float *>(w + c.R);
    a.steps = reinterpret_cast<float *>(w + c.steps);
    a.bc_part = reinterpret_cast<float *>(w + c.bc);
    a.dA_part = reinterpret_cast<float *>(w + c.dA);
    a.d_part = reinterpret_cast<float *>(w + c.d);
    a.batch = pr.batch;
    a.L = pr.seqlen;
    a.D = pr.nheads;
    a.G = pr.ngroups;
    a.nc = chunks(pr);
    a.step.pre = DtPreArgs{pre.bias, pre.softplus, pre.zoh, pre.dt_min, pre.dt_max};
    a.step.on = pre.bias || pre.softplus || pre.dt_max > 0.f;
    for (int k = 0; k < 2; ++k) a.step.lo[k] = a.step.hi[k] = 0.f;
    if (pre.dt_max > 0.f) {
        a.step.lo[0] = pre.dt_min;
        a.step.hi[0] = pre.dt_max;
        if (pre.softplus) {
            softplus_preimage(pre.dt_min, a.step.lo);
            softplus_preimage(pre.dt_max, a.step.hi);
        }
    }
    const bool zoh = pre.zoh != 0;
    e = pr.dtype == SSD_F32
            ? launch_t<float>(pr, a, zoh, h0, dh_final, dA, dD, ddt_bias, dh0, st)
            : launch_t<__nv_bfloat16>(pr, a, zoh, h0, dh_final, dA, dD, ddt_bias, dh0, st);
    return e == cudaSuccess ? SSD_OK : cuda_fail(e, "selective scan backward launch");
}

}  // namespace ssd
