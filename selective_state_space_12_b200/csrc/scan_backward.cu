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
// softplus. Every state entry takes an exponential a token and about a dozen
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

// exp(z), the input weight and (SLOPE) dw/dA of one state entry, z = dt A.
// The hold takes e^z - 1 and what follows from it by their series where
// |z| < 1/4: phi2 = (phi1 - 1) / z to z^4 (remainder below z^5/5040 < 2e-7),
// phi1 = (e^z - 1) / z = 1 + z phi2, w = dt phi1, dw/dA = dt^2 (phi1 - phi2),
// none of which cancels. A = 0 comes as -1e-30 (read_A).
template <bool ZOH, bool SLOPE>
__device__ __forceinline__ void entry(float dt, float A, float invA, float &a, float &w,
                                      float &slope) {
    if (!ZOH) {
        a = tc::fast_exp2(dt * A);  // A holds A log2 e
        w = dt;
        return;
    }
    const float z = dt * A;
    const float e = tc::fast_exp2(z * kLog2eB), em = e - 1.f;
    float phi2 = 1.f / 720.f;
    phi2 = fmaf(phi2, z, 1.f / 120.f);
    phi2 = fmaf(phi2, z, 1.f / 24.f);
    phi2 = fmaf(phi2, z, 1.f / 6.f);
    phi2 = fmaf(phi2, z, 0.5f);
    const float phi1 = fmaf(z, phi2, 1.f);
    const bool small = fabsf(z) < 0.25f;
    a = small ? fmaf(z, phi1, 1.f) : e;
    w = small ? dt * phi1 : em * invA;
    if (SLOPE) slope = small ? dt * dt * (phi1 - phi2) : (dt * e - w) * invA;
}

__device__ __forceinline__ float read_A(float A, bool zoh) {
    return zoh ? (A == 0.f ? -1e-30f : A) : A * kLog2eB;
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
struct Tile {
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

// The map of a run of tokens for one thread's states: end state S from zero,
// gradient R handed to the left when none comes from the right, product P.
template <int N, bool ZOH, int TOKENS>
__device__ __forceinline__ void run_sums(const Tile<N> &s, int c, int t0, int n0,
                                         const float (&A)[kQ], const float (&invA)[kQ],
                                         float (&S)[kQ], float (&R)[kQ], float (&P)[kQ]) {
#pragma unroll
    for (int k = 0; k < kQ; ++k) S[k] = R[k] = 0.f, P[k] = 1.f;
#pragma unroll 4
    for (int t = t0; t < t0 + TOKENS; ++t) {
        const float xv = s.x[c][t], dtv = s.dt[c][t], yv = s.dy[c][t];
#pragma unroll
        for (int k = 0; k < kQ; ++k) {
            float av, w, unused;
            entry<ZOH, false>(dtv, A[k], invA[k], av, w, unused);
            S[k] = fmaf(av, S[k], w * xv * s.B[t][n0 + k]);
            P[k] *= av;
            R[k] = fmaf(P[k], yv * s.C[t][n0 + k], R[k]);
        }
    }
}

template <int N>
__device__ __forceinline__ void load_A(const BwdArgs &a, int64_t d, int n0, bool zoh,
                                       float (&A)[kQ], float (&invA)[kQ]) {
#pragma unroll
    for (int k = 0; k < kQ; ++k) {
        A[k] = read_A(a.A[d * N + n0 + k], zoh);
        invA[k] = zoh ? 1.f / A[k] : 0.f;
    }
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
        float A[kQ], invA[kQ], S[kQ], R[kQ], P[kQ];
        load_A<N>(a, d, n0, ZOH, A, invA);
        run_sums<N, ZOH, kChunk>(s, c, 0, n0, A, invA, S, R, P);
        if (has) {
            const int64_t at = (p.b * a.nc + p.chunk) * a.D + d;
#pragma unroll
            for (int j = 0; j < kQ; ++j) {
                a.S[at * N + n0 + j] = S[j];
                a.R[at * N + n0 + j] = R[j];
            }
            if (n0 == 0) {
                float sum = 0.f;
                for (int t = 0; t < kChunk; ++t) sum += s.dt[c][t];
                a.steps[at] = sum;
            }
        }
    }
}

// The chains over chunks: blockIdx.y 0 the states, 1 the gradients.
__global__ void scan_bwd_chain(const BwdArgs a, int N, const float *h0, const float *dh_final,
                               float *dh0) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t lane_len = a.D * N;
    if (i >= a.batch * lane_len) return;
    const int64_t b = i / lane_len, dn = i % lane_len;
    const bool back = blockIdx.y == 1;
    const float A = a.A[dn] * kLog2eB;
    const float *first = back ? dh_final : h0;
    float *S = back ? a.R : a.S;
    float h = first ? first[i] : 0.f;
    for (int64_t j = 0; j < a.nc; ++j) {
        const int64_t c = b * a.nc + (back ? a.nc - 1 - j : j);
        const float v = S[c * lane_len + dn];
        S[c * lane_len + dn] = h;
        h = fmaf(tc::fast_exp2(a.steps[c * a.D + dn / N] * A), h, v);
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

template <typename T, int N, bool ZOH>
__global__ void __launch_bounds__(kMainThreads, 1) scan_bwd_main(const BwdArgs a) {
    constexpr int kLanes = N / kQ, kPerWarp = 32 / kLanes, kState = kCh * N;
    extern __shared__ __align__(16) unsigned char raw[];
    MainTile<N> &s = *reinterpret_cast<MainTile<N> *>(raw);
    const Place p = place(a);
    const int64_t dend = (p.g + 1) * a.gch;
    const int tid = threadIdx.x, lane = tid & 31, piece = tid >> 5;
    const int n0 = (lane % kLanes) * kQ, t0 = piece * kPiece;
    float accB[kPiece][kQ], accC[kPiece][kQ];
#pragma unroll
    for (int t = 0; t < kPiece; ++t)
#pragma unroll
        for (int k = 0; k < kQ; ++k) accB[t][k] = accC[t][k] = 0.f;
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
        for (int c = lane / kLanes; c < kCh; c += kPerWarp) {
            float A[kQ], invA[kQ], S[kQ], R[kQ], P[kQ];
            load_A<N>(a, d0 + c < dend ? d0 + c : dend - 1, n0, ZOH, A, invA);
            run_sums<N, ZOH, kPiece>(s, c, t0, n0, A, invA, S, R, P);
#pragma unroll
            for (int k = 0; k < kQ; ++k) {
                s.S[piece][c * N + n0 + k] = S[k];
                s.R[piece][c * N + n0 + k] = R[k];
                s.P[piece][c * N + n0 + k] = P[k];
            }
        }
        __syncthreads();
        if (tid < kState) {
            for (int j = 0; j < kPieces; ++j) {
                const float v = s.S[j][tid];
                s.S[j][tid] = h;
                h = fmaf(s.P[j][tid], h, v);
            }
            for (int j = kPieces - 1; j >= 0; --j) {
                const float v = s.R[j][tid];
                s.R[j][tid] = r;
                r = fmaf(s.P[j][tid], r, v);
            }
        }
        __syncthreads();
        for (int c = lane / kLanes; c < kCh; c += kPerWarp) {
            const int64_t d = d0 + c < dend ? d0 + c : dend - 1;
            float A[kQ], invA[kQ], An[kQ], dA[kQ], hp[kPiece][kQ], av[kPiece][kQ],
                sl[kPiece][kQ], hc[kQ], rc[kQ];
            load_A<N>(a, d, n0, ZOH, A, invA);
            const float Ds = a.Dskip ? a.Dskip[d] : 0.f;
#pragma unroll
            for (int k = 0; k < kQ; ++k) {
                An[k] = ZOH ? A[k] : a.A[d * N + n0 + k];
                dA[k] = 0.f;
                hc[k] = s.S[piece][c * N + n0 + k];
                rc[k] = s.R[piece][c * N + n0 + k];
            }
#pragma unroll
            for (int t = 0; t < kPiece; ++t) {
                const float xv = s.x[c][t0 + t], dtv = s.dt[c][t0 + t], yv = s.dy[c][t0 + t];
#pragma unroll
                for (int k = 0; k < kQ; ++k) {
                    float w;
                    entry<ZOH, true>(dtv, A[k], invA[k], av[t][k], w, sl[t][k]);
                    hp[t][k] = hc[k];
                    hc[k] = fmaf(av[t][k], hc[k], w * xv * s.B[t0 + t][n0 + k]);
                    accC[t][k] = fmaf(yv, hc[k], accC[t][k]);
                }
            }
            float vB[kPiece], vA[kPiece];
#pragma unroll
            for (int t = kPiece - 1; t >= 0; --t) {
                const float xv = s.x[c][t0 + t], dtv = s.dt[c][t0 + t], yv = s.dy[c][t0 + t];
                vB[t] = vA[t] = 0.f;
#pragma unroll
                for (int k = 0; k < kQ; ++k) {
                    const float Bv = s.B[t0 + t][n0 + k];
                    const float rv = fmaf(yv, s.C[t0 + t][n0 + k], rc[k]);
                    const float ra = rv * av[t][k];
                    if (ZOH) {
                        const float w = fmaf(dtv, av[t][k], -An[k] * sl[t][k]);
                        const float rw = rv * w, xB = xv * Bv;
                        vB[t] = fmaf(rw, Bv, vB[t]);
                        accB[t][k] = fmaf(rw, xv, accB[t][k]);
                        vA[t] = fmaf(ra, fmaf(An[k], hp[t][k], xB), vA[t]);
                        dA[k] = fmaf(ra * dtv, hp[t][k], fmaf(rv * sl[t][k], xB, dA[k]));
                    } else {
                        vB[t] = fmaf(rv, Bv, vB[t]);
                        accB[t][k] = fmaf(rv, dtv * xv, accB[t][k]);
                        const float t1 = ra * hp[t][k];
                        vA[t] = fmaf(An[k], t1, vA[t]);
                        dA[k] = fmaf(dtv, t1, dA[k]);
                    }
                    rc[k] = ra;
                }
            }
#pragma unroll
            for (int t = 0; t < kPiece; ++t) {
                const float sB = lanes_sum<kLanes>(vB[t]), sA = lanes_sum<kLanes>(vA[t]);
                if (lane % kLanes == 0) {
                    const float xv = s.x[c][t0 + t], yv = s.dy[c][t0 + t];
                    s.dx[c][t0 + t] = fmaf(Ds, yv, ZOH ? sB : sB * s.dt[c][t0 + t]);
                    s.fac[c][t0 + t] *= ZOH ? sA : fmaf(xv, sB, sA);  // ddt
                }
            }
#pragma unroll
            for (int k = 0; k < kQ; ++k) s.P[piece][c * N + n0 + k] = dA[k];
        }
        __syncthreads();
        if (chain) {
            float v = 0.f;
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
            float vb = accB[t][k], vc = accC[t][k];
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
    scan_bwd_chain<<<dim3((unsigned)((lanes + 127) / 128), 2), 128, 0, st>>>(a, N, h0, dh_final,
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
