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
//   g <- g + E (g + x B)   w = E / A   ddt = sum_n a r (g + x B) = sum_n r (g' + x B)
//
// where g' is the state after the token. dA = sum_t r [dt a h + (dw/dA) x B] by these is
//
//   dA = (1/A) sum_t r [dt g' - (w - dt) x B]
//
// w - dt is about z dt / 2, z = dt A; from w it keeps 1 / z of its bits, so for small E it
// is dt E (1/2 - z/12) (w - dt = dt E (1/z - 1/E), and 1/z - 1/E = 1/2 - z/12 + z^3/720 -
// ...). For large -z both forms lose: g' + x B is a (g + x B), a difference of a's size,
// and dt g' nearly cancels dt x B. Channels that come to such steps are done by
// far_channel, from a itself.
// Every state entry takes an exponential a token and about a dozen fp32
// operations, 16 or so times what a token's bytes need: the pass is bound by the
// arithmetic, and by keeping sums over states (dx, ddt), over channels
// (dB, dC) and over tokens (dA) all in registers.
//
// Time is cut into chunks of 32 tokens that run side by side:
//   1. scan_bwd_sums: each chunk's end state from a zero state, and the
//      gradient it hands to its left when none comes from its right;
//   2. scan_bwd_chain: the chains over chunks, forward and backward, leaving
//      the state entering each chunk and the gradient entering it from its right;
//   3. scan_bwd_main: the same again inside a chunk over its eight pieces of four
//      tokens (a warp each), then each piece's states forward and gradients
//      back, from registers;
//   4. scan_bwd_finish: sums of dB and dC over blocks of channels, and of dA, dDskip
//      and the bias's gradient over batch and chunks. No atomics: every sum has
//      one order.
//
// Measured, B200, bf16, b8 L2048 D5120 N16 with softplus: hold 4080 us (0.33 T state
// entries a second), of which the sums take 802 us, the chain 168, the main kernel
// 3071 and the last sums 54; Euler 2860 us (617, 166, 2035, 54). The main kernel with
// the hold issues about 103 instructions for each pair of entries and token in 58 % of
// its issue slots: 16 warps an SM at 128 registers a thread, whose latencies (exp2,
// shared memory, the packed arithmetic) they do not quite hide. (18 of the 103 are what
// dA takes to keep its bits at small steps: 85 and 2730 us with the two terms that
// cancel.)
#include <cudaTypedefs.h>
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace ssd {
namespace {

constexpr float kLog2eB = 1.4426950408889634f;
constexpr int kChunk = 32;               // tokens of a chunk
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

// log(1 + e), e in [0, 1], as 2 atanh(z), z = e / (2 + e) <= 1/3: the series to
// z^13, whose remainder is below 1.6e-8 of the result (at e = 1; 2 z^15 (1/15 +
// z^2/17 + ...) of 2 z (1 + z^2/3 + ...)).
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
// E = exp(dt A) - 1 (hold). With y = dt A log2 e both start from exp2(y); the hold
// takes E by its series in y where |y| < 1/8 (the term (y ln 2)^4 / 4! ends it:
// the next is below 5e-7 relative), else from exp2, whose error of 2^-22 is then
// below 3e-6 of it.
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
    f2 Al;  // A log2 e (hold: A kept off zero)
    __device__ __forceinline__ f2 at(f2 dt) const {
        f2 a;
        return at(dt, a);
    }
    __device__ __forceinline__ f2 at(f2 dt, f2 &e) const {  // e: exp(dt A) in both cases
        const f2 y = f2_mul(dt, Al);
        float y0, y1;
        f2_unpack(y, y0, y1);
        e = f2_pack(tc::fast_exp2(y0), tc::fast_exp2(y1));
        if (!ZOH) return e;
        constexpr double k = 0.693147180559945309;  // ln 2
        f2 p = f2_fma(f2_both((float)(k * k * k * k / 24)), y, f2_both((float)(k * k * k / 6)));
        p = f2_fma(p, y, f2_both((float)(k * k / 2)));
        p = f2_fma(p, y, f2_both((float)k));
        float s0, s1, e0, e1;
        f2_unpack(f2_mul(y, p), s0, s1);
        f2_unpack(f2_add(e, f2_both(-1.f)), e0, e1);
        return f2_pack(fabsf(y0) < 0.125f ? s0 : e0, fabsf(y1) < 0.125f ? s1 : e1);
    }
};

// A as the hold uses it: |A| >= 2^-40, which changes no result by more than
// 2^-40 a token and lets g = A h carry the state of A = 0 too.
__device__ __forceinline__ float off_zero(float A) {
    return fabsf(A) < 0x1p-40f ? (A > 0.f ? 0x1p-40f : -0x1p-40f) : A;
}

// Steps at which the hold's forms in the main loop lose bits: -z above kFar for one state
// (they lose z 2^-24 a rounding, 2e-5 in all at kFar), or above kFast for all of a channel's
// (ddt is then of a's size, and loses 2^-24 / a). Such a channel's dA and ddt are computed a
// second time: where all are such, b8 L2048 D5120 takes 5680 us for 4080.
constexpr float kFar = 96.f, kFast = 4.f;
// For a step dt of a channel with -A in [least, most].
__device__ __forceinline__ bool far_step(float dt, float least, float most) {
    const float lo = dt < 0.f ? dt * most : dt * least, hi = dt < 0.f ? dt * least : dt * most;
    return hi > kFar || lo > kFast;
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
    bool words;          // x, dt and dy start on 4 bytes
    unsigned *err;
    long long wait;
};

// Shared memory of the staged tile. Channels' rows of tokens, as stored, arrive
// in `words` a tile ahead and are spread from there as floats, tokens along a
// row. Where rows start on 16 bytes (ALIGNED) they come by one TMA load a tensor,
// elsewhere by asynchronous copies of the 4-byte words that cover them.
struct Maps {
    CUtensorMap m[3];
};
constexpr long long kDrain = 1ll << 24;  // cycles: a wait for loads in flight at an early end
template <typename T, int N, int CH, bool ALIGNED>
struct __align__(128) Tile {
    static constexpr int kState = CH * N;
    static constexpr int kPitch = CH * (int)sizeof(T) + (ALIGNED ? 0 : 16);
    __align__(128) unsigned char words[3][kChunk][kPitch];
    float x[CH][kRow], dt[CH][kRow], dy[CH][kRow];
    float B[kChunk][N], C[kChunk][N];
    float A[kState], Al[kState], invA[kState];  // A, A log2 e, -1 / A (hold)
    float next_A[kState], next_bias[CH], next_Ds[CH];  // as they arrive
    uint64_t bar;
};
template <typename T, int N, int CH, bool ALIGNED>
struct MainTile : Tile<T, N, CH, ALIGNED> {
    float fac[CH][kRow];
    float S[kPieces][CH * N], R[kPieces][CH * N], P[kPieces][CH * N];
    float dd[kPieces][CH], db[kPieces][CH];
    float Ds[CH];
    unsigned far;  // channels with steps that far_channel is for
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

__device__ __forceinline__ void copy4(void *to, const void *from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(tc::smem_u32(to)), "l"(from)
                 : "memory");
}

// Requests the rows of x, dt and dy of the tile at d0. Words that might leave
// the tensor (its last tile; a bf16 tensor that starts inside a word) are not
// requested: spread() then reads the tensors themselves.
template <typename T, int CH>
__device__ __forceinline__ bool by_words(const BwdArgs &a, const Place &p, int64_t d0) {
    return sizeof(T) == 4 || (a.words && !(p.b == a.batch - 1 && p.chunk == a.nc - 1 &&
                                           d0 + CH >= a.D));
}
template <typename T, int N, int CH, bool ALIGNED, int THREADS>
__device__ __forceinline__ void request(const BwdArgs &a, const Maps &maps, const Place &p, int64_t d0,
                                        int64_t dend, Tile<T, N, CH, ALIGNED> &s) {
    constexpr int kE = (int)sizeof(T), kWords = CH * kE / 4;  // of a row that starts on one
    if constexpr (ALIGNED) {
        if (threadIdx.x == 0) {
            tc::mbar_arrive_expect_tx(&s.bar, sizeof(s.words));
#pragma unroll
            for (int w = 0; w < 3; ++w)
                tc::tma_load_4d(s.words[w], &maps.m[w], &s.bar, (int)d0, (int)p.t0, (int)p.b, 0);
        }
    } else if (by_words<T, CH>(a, p, d0)) {
        const void *const src[3] = {a.x, a.dt, a.dy};
        const int len = (int)(dend - d0 < CH ? dend - d0 : CH);
        const int i = threadIdx.x % kWords, t0 = threadIdx.x / kWords;
#pragma unroll
        for (int w = 0; w < 3; ++w) {
            const uintptr_t row = reinterpret_cast<uintptr_t>(src[w]) +
                                  kE * ((p.b * a.L + p.t0) * a.D + d0);
            for (int t = t0; t < p.n; t += THREADS / kWords) {
                const uintptr_t r = row + kE * (uintptr_t)(t * a.D);
                const int words = ((int)(r & 3) + kE * len + 3) / 4;
                if (i < words)
                    copy4(&s.words[w][t][4 * i], reinterpret_cast<const void *>((r & ~uintptr_t(3)) + 4 * i));
                if (kE == 2 && i == 0 && words > kWords)
                    copy4(&s.words[w][t][4 * kWords],
                          reinterpret_cast<const void *>((r & ~uintptr_t(3)) + 4 * kWords));
            }
        }
    }
    const int has = (int)(dend - d0 < CH ? dend - d0 : CH);
    for (int i = threadIdx.x; i < has * N; i += THREADS) copy4(&s.next_A[i], a.A + d0 * N + i);
    for (int i = threadIdx.x; i < has; i += THREADS) {
        if (a.step.pre.bias) copy4(&s.next_bias[i], a.step.pre.bias + d0 + i);
        if (a.Dskip) copy4(&s.next_Ds[i], a.Dskip + d0 + i);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}

// Waits for the requested tile, all threads; false when the wait ran out.
template <typename T, int N, int CH, bool ALIGNED>
__device__ __forceinline__ bool arrived(const BwdArgs &a, Tile<T, N, CH, ALIGNED> &s, uint32_t &parity) {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if constexpr (!ALIGNED) {
        __syncthreads();
        return true;
    }
    if (__syncthreads_and(tc::mbar_wait(&s.bar, parity, a.wait))) {
        parity ^= 1;
        return true;
    }
    if (threadIdx.x == 0) atomicExch(a.err, 0x5bacd001u);
    tc::mbar_wait(&s.bar, parity, kDrain);
    return false;
}

// The requested tile as floats, dt prepared; channels and tokens past the end
// are zeros (dt = 0: a = 1, w = 0). Also A and what follows from it.
// GRAD: fac, and with the hold the channels of `far` are for the main kernel.
template <typename T, int N, int CH, bool ALIGNED, bool ZOH, bool GRAD, int THREADS>
__device__ __forceinline__ void spread(const BwdArgs &a, const Place &p, int64_t d0, int64_t dend,
                                       Tile<T, N, CH, ALIGNED> &s, float (*fac)[kRow],
                                       unsigned *far) {
    const void *const src[3] = {a.x, a.dt, a.dy};
    const bool words = ALIGNED || by_words<T, CH>(a, p, d0);
    // eight channels by four runs of four tokens a warp: rows are written 16 bytes at a time
    const int64_t base = (p.b * a.L + p.t0) * a.D + d0;
    for (int i = threadIdx.x; i < CH * (kChunk / 4); i += THREADS) {
        const int c = (i / 8 / (kChunk / 4)) * 8 + i % 8, t0 = (i / 8) % (kChunk / 4) * 4;
        const bool has = d0 + c < dend;
        const float bias = (has && a.step.pre.bias) ? s.next_bias[c] : 0.f;
        float v[3][4], f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[j] = v[0][j] = v[1][j] = v[2][j] = 0.f;
            if (has && t0 + j < p.n) {
#pragma unroll
                for (int w = 0; w < 3; ++w) {
                    if constexpr (ALIGNED) {
                        v[w][j] = to_f(reinterpret_cast<const T *>(s.words[w][t0 + j])[c]);
                    } else {
                        const T *row = static_cast<const T *>(src[w]) + base + (t0 + j) * a.D;
                        const uintptr_t in_word = reinterpret_cast<uintptr_t>(row) & 3;
                        v[w][j] = words ? to_f(reinterpret_cast<const T *>(
                                              &s.words[w][t0 + j][in_word])[c])
                                        : to_f(row[c]);
                    }
                }
                v[1][j] = prepare_step<GRAD>(v[1][j], bias, a.step, f[j]);
            }
        }
        *reinterpret_cast<float4 *>(&s.x[c][t0]) = make_float4(v[0][0], v[0][1], v[0][2], v[0][3]);
        *reinterpret_cast<float4 *>(&s.dt[c][t0]) = make_float4(v[1][0], v[1][1], v[1][2], v[1][3]);
        *reinterpret_cast<float4 *>(&s.dy[c][t0]) = make_float4(v[2][0], v[2][1], v[2][2], v[2][3]);
        if (GRAD) *reinterpret_cast<float4 *>(&fac[c][t0]) = make_float4(f[0], f[1], f[2], f[3]);
        if (GRAD && ZOH) {
            // the four lanes of a channel look at a quarter of its A each
            const float *mine = &s.next_A[c * N + (i / 8) % 4 * (N / 4)];
            float least = -mine[0], most = least;
#pragma unroll
            for (int n = 1; n < N / 4; ++n) {
                least = fminf(least, -mine[n]);
                most = fmaxf(most, -mine[n]);
            }
#pragma unroll
            for (int o = 8; o < 32; o <<= 1) {
                least = fminf(least, __shfl_xor_sync(0xffffffffu, least, o));
                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
            }
            if (has &&
                (far_step(fmaxf(fmaxf(v[1][0], v[1][1]), fmaxf(v[1][2], v[1][3])), least, most) ||
                 far_step(fminf(fminf(v[1][0], v[1][1]), fminf(v[1][2], v[1][3])), least, most)))
                atomicOr(far, 1u << c);
        }
    }
    for (int i = threadIdx.x; i < CH * N; i += THREADS) {
        float v = d0 + i / N < dend ? s.next_A[i] : -1.f;
        if (ZOH) v = off_zero(v);
        s.A[i] = v;
        s.Al[i] = v * kLog2eB;
        if (ZOH) s.invA[i] = -1.f / v;
    }
}
template <typename T, int N, int CH, bool ALIGNED, int THREADS>
__device__ __forceinline__ void stage_rows(const BwdArgs &a, const Place &p, Tile<T, N, CH, ALIGNED> &s) {
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
// zero, gradient R handed to the left when none comes from the right, product P
// (EXACT: of the decays themselves, not of 1 + E: dh0 is of their size).
template <typename T, int N, int CH, bool ALIGNED, bool ZOH, int TOKENS, bool EXACT>
__device__ __forceinline__ void run_sums(const Tile<T, N, CH, ALIGNED> &s, int c, int t0, int n0,
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
                f2 e;
                const f2 F = A[k].at(dt, e);
                S[k] = move<ZOH>(F, S[k], f2_mul(in, B[k]));
                P[k] = EXACT ? f2_mul(P[k], e) : times_decay<ZOH>(P[k], F);
                R[k] = f2_fma(P[k], f2_mul(dy, C[k]), R[k]);
            }
        }
    }
}

template <typename T, int N, int CH, bool ALIGNED, bool ZOH>
__device__ __forceinline__ void load_A(const Tile<T, N, CH, ALIGNED> &s, int at, Decay<ZOH> (&A)[2]) {
    f2 l[2];
    load4x(&s.Al[at], l);
    A[0].Al = l[0];
    A[1].Al = l[1];
}

// A thread walks a chunk's 32 tokens for four states of a channel; one exponential and
// five packed operations a pair of entries.
template <typename T, int N, bool ZOH, bool ALIGNED>
__global__ void __launch_bounds__(kCh *N / kQ, 640 / (kCh * N / kQ))
scan_bwd_sums(const BwdArgs a, const __grid_constant__ Maps maps) {
    constexpr int CH = kCh, kThreads = CH * N / kQ, kLanes = N / kQ;
    extern __shared__ __align__(128) unsigned char raw[];
    using S_ = Tile<T, N, CH, ALIGNED>;
    S_ &s = *reinterpret_cast<S_ *>(raw);
    const Place p = place(a);
    const int64_t dend = (p.g + 1) * a.gch, dstart = p.g * a.gch + (int64_t)p.tile0 * CH;
    uint32_t parity = 0;
    if (threadIdx.x == 0) {
        tc::mbar_init(&s.bar, 1);
        tc::fence_mbar_init();
    }
    __syncthreads();
    request<T, N, CH, ALIGNED, kThreads>(a, maps, p, dstart, dend, s);
    stage_rows<T, N, CH, ALIGNED, kThreads>(a, p, s);
    const int c = threadIdx.x / kLanes, n0 = (threadIdx.x % kLanes) * kQ;
    for (int k = 0; k < p.tiles; ++k) {
        const int64_t d0 = dstart + (int64_t)k * CH;
        if (!arrived(a, s, parity)) return;
        spread<T, N, CH, ALIGNED, ZOH, false, kThreads>(a, p, d0, dend, s, nullptr, nullptr);
        __syncthreads();
        if (k + 1 < p.tiles) request<T, N, CH, ALIGNED, kThreads>(a, maps, p, d0 + CH, dend, s);
        const bool has = d0 + c < dend;
        Decay<ZOH> A[2];
        f2 S[2], R[2], P[2];
        load_A<T, N, CH, ALIGNED, ZOH>(s, c * N + n0, A);
        run_sums<T, N, CH, ALIGNED, ZOH, kChunk, true>(s, c, 0, n0, A, S, R, P);
        if (has) {
            const int64_t at = (p.b * a.nc + p.chunk) * a.D + d0 + c;
            store4x(&a.S[at * N + n0], S);
            store4x(&a.R[at * N + n0], R);
            if (n0 == 0) {
                float sum = 0.f;
#pragma unroll
                for (int t = 0; t < kChunk; t += 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(&s.dt[c][t]);
                    sum += (v.x + v.y) + (v.z + v.w);
                }
                a.steps[at] = sum;
            }
        }
        __syncthreads();  // the tile has been read
    }
}

// The chains over chunks, bound by their bytes (read and written: 671 MB of S and R at
// b8 L2048 D5120 N16, 167 us, 4 TB/s): blockIdx.y 0 the states (with the hold g = A h), 1
// the gradients. Eight chunks' words are loaded at a time.
template <int N, bool ZOH>
__global__ void __launch_bounds__(128)
scan_bwd_chain(const BwdArgs a, const float *h0, const float *dh_final, float *dh0) {
    after_previous();
    let_next();
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
    float v[kBatch], t[kBatch];
    auto load = [&](int64_t j0) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const bool has = j0 + j < a.nc;
            v[j] = has ? __ldcg(S + way * (j0 + j) * lane_len) : 0.f;
            t[j] = has ? __ldcg(steps + way * (j0 + j) * a.D) : 0.f;
        }
    };
    load(0);
    for (int64_t j0 = 0; j0 < a.nc; j0 += kBatch) {
        float e[kBatch], u[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            e[j] = t[j];
            u[j] = v[j];
        }
        if (j0 + kBatch < a.nc) load(j0 + kBatch);  // the next batch is on its way
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            if (j0 + j >= a.nc) break;
            S[way * (j0 + j) * lane_len] = h;
            h = fmaf(tc::fast_exp2(e[j] * Al), h, u[j]);
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

// -(w - dt) and its bits, by the size of E: kNear is where what the one form leaves out
// (z^3/360 of it: 2e-5) is as much as the other loses (an error of E of 2^-22).
constexpr float kNear = 1.f / 6.f;
__device__ __forceinline__ f2 dt_less_w(f2 dt, f2 E, f2 wn, f2 A12) {
    const f2 near = f2_mul(f2_mul(dt, E), f2_fma(dt, A12, f2_both(-0.5f)));
    float e0, e1, n0, n1, f0, f1;
    f2_unpack(E, e0, e1);
    f2_unpack(near, n0, n1);
    f2_unpack(f2_add(dt, wn), f0, f1);
    return f2_pack(fabsf(e0) < kNear ? n0 : f0, fabsf(e1) < kNear ? n1 : f1);
}

// The hold for one lane's states of a channel with such steps: dA (its sign turned, as
// from the main loop) to s.P, and the lane's sums for ddt, a r (g + x B) with a from exp2.
template <typename T, int N, int CH, bool ALIGNED>
__device__ __noinline__ float4 far_channel(MainTile<T, N, CH, ALIGNED> &s, int piece, int c, int n0) {
    float v[kPiece] = {};
    for (int k = 0; k < kQ; ++k) {
        const int n = n0 + k, at = c * N + n;
        const float Al = s.Al[at], invA = s.invA[at];
        float E[kPiece], decay[kPiece], after[kPiece], decayed[kPiece];
        float st = s.S[piece][at], carry = s.R[piece][at], dA = 0.f, unused;
#pragma unroll
        for (int t = 0; t < kPiece; ++t) {
            const int tok = piece * kPiece + t;
            const float dt = s.dt[c][tok], before = fmaf(s.x[c][tok], s.B[tok][n], st);
            f2 e;
            f2_unpack(Decay<true>{f2_both(Al)}.at(f2_both(dt), e), E[t], unused);
            f2_unpack(e, decay[t], unused);
            decayed[t] = decay[t] * before;
            after[t] = st = fmaf(E[t], before, st);
        }
#pragma unroll
        for (int t = kPiece - 1; t >= 0; --t) {
            const int tok = piece * kPiece + t;
            const float dt = s.dt[c][tok], in = s.x[c][tok] * s.B[tok][n];
            const float r = fmaf(s.dy[c][tok], s.C[tok][n], carry), wn = E[t] * invA;
            const float near = dt * E[t] * fmaf(dt, s.A[at] * (1.f / 12.f), -0.5f);
            const bool is_near = fabsf(E[t]) < kNear;
            dA = fmaf(r, fmaf(dt, is_near ? after[t] : decayed[t], in * (is_near ? near : wn)), dA);
            v[t] = fmaf(r, decayed[t], v[t]);
            carry = r * decay[t];
        }
        s.P[piece][at] = invA * dA;
    }
    return make_float4(v[0], v[1], v[2], v[3]);
}

// A warp has a piece of four tokens, a lane four states of one channel at a time: sums
// over channels (dB, dC) stay in the lane over all its channels, sums over states (dx,
// ddt) are shared out over a channel's lanes, sums over tokens (dA) are the lane's own.
// Four tokens are what two thread blocks an SM have registers for: the exponentials
// and states of a piece are computed again rather than kept (kept in shared memory,
// with half the channels a tile, was slower).
template <typename T, int N, bool ZOH, bool ALIGNED>
__global__ void __launch_bounds__(kMainThreads, 2)
scan_bwd_main(const BwdArgs a, const __grid_constant__ Maps maps) {
    after_previous();
    let_next();
    constexpr int CH = kCh, kLanes = N / kQ, kPerWarp = 32 / kLanes, kState = CH * N;
    constexpr int kShare = kPiece / kLanes;  // tokens of a piece whose dx and ddt a lane ends with
    extern __shared__ __align__(128) unsigned char raw[];
    using S_ = MainTile<T, N, CH, ALIGNED>;
    S_ &s = *reinterpret_cast<S_ *>(raw);
    const Place p = place(a);
    const int64_t dend = (p.g + 1) * a.gch, dstart = p.g * a.gch + (int64_t)p.tile0 * CH;
    const int tid = threadIdx.x, lane = tid & 31, piece = tid >> 5;
    const int n0 = (lane % kLanes) * kQ, t0 = piece * kPiece, cl = lane / kLanes;
    const int share0 = t0 + (lane % kLanes) * kShare;  // the first of this lane's tokens
    const f2 none = f2_both(0.f);
    uint32_t parity = 0;
    f2 accB[kPiece][2], accC[kPiece][2];
#pragma unroll
    for (int t = 0; t < kPiece; ++t)
#pragma unroll
        for (int k = 0; k < 2; ++k) accB[t][k] = accC[t][k] = none;
    if (tid == 0) {
        tc::mbar_init(&s.bar, 1);
        tc::fence_mbar_init();
    }
    __syncthreads();
    request<T, N, CH, ALIGNED, kMainThreads>(a, maps, p, dstart, dend, s);
    stage_rows<T, N, CH, ALIGNED, kMainThreads>(a, p, s);
    const int64_t row = (p.b * a.nc + p.chunk) * a.D;
    for (int tile = 0; tile < p.tiles; ++tile) {
        const int64_t d0 = dstart + (int64_t)tile * CH;
        const int here = (int)(dend - d0 < CH ? dend - d0 : CH);  // channels
        if (tid == 0) s.far = 0;
        if (!arrived(a, s, parity)) return;
        spread<T, N, CH, ALIGNED, ZOH, true, kMainThreads>(a, p, d0, dend, s, s.fac, &s.far);
        if (tid < CH) s.Ds[tid] = (a.Dskip && tid < here) ? s.next_Ds[tid] : 0.f;
        // this thread's pair of links of the chains over pieces
        float2 link_h = make_float2(0.f, 0.f), link_r = link_h;
        if (2 * tid < here * N) {
            link_h = *reinterpret_cast<const float2 *>(&a.S[(row + d0) * N + 2 * tid]);
            link_r = *reinterpret_cast<const float2 *>(&a.R[(row + d0) * N + 2 * tid]);
        }
        __syncthreads();
        if (tile + 1 < p.tiles) request<T, N, CH, ALIGNED, kMainThreads>(a, maps, p, d0 + CH, dend, s);
#pragma unroll 1
        for (int c = cl; c < CH; c += kPerWarp) {
            Decay<ZOH> A[2];
            f2 S[2], R[2], P[2];
            load_A<T, N, CH, ALIGNED, ZOH>(s, c * N + n0, A);
            run_sums<T, N, CH, ALIGNED, ZOH, kPiece, false>(s, c, t0, n0, A, S, R, P);
            store4x(&s.S[piece][c * N + n0], S);
            store4x(&s.R[piece][c * N + n0], R);
            store4x(&s.P[piece][c * N + n0], P);
        }
        __syncthreads();
        if (2 * tid < kState) {
            f2 P[kPieces], S[kPieces], R[kPieces];
#pragma unroll
            for (int j = 0; j < kPieces; ++j) {
                P[j] = *reinterpret_cast<const f2 *>(&s.P[j][2 * tid]);
                S[j] = *reinterpret_cast<const f2 *>(&s.S[j][2 * tid]);
                R[j] = *reinterpret_cast<const f2 *>(&s.R[j][2 * tid]);
            }
            f2 h = f2_pack(link_h.x, link_h.y), r = f2_pack(link_r.x, link_r.y);
#pragma unroll
            for (int j = 0; j < kPieces; ++j) {
                const int k = kPieces - 1 - j;
                *reinterpret_cast<f2 *>(&s.S[j][2 * tid]) = h;
                *reinterpret_cast<f2 *>(&s.R[k][2 * tid]) = r;
                h = f2_fma(P[j], h, S[j]);
                r = f2_fma(P[k], r, R[k]);
            }
        }
        __syncthreads();
        const unsigned far = ZOH ? s.far : 0;
        float *dx = a.dx + (p.b * a.L + p.t0 + share0) * a.D + d0 + cl;
        float *ddt = a.ddt + (dx - a.dx);
#pragma unroll 1
        for (int c = cl; c < CH; c += kPerWarp, dx += kPerWarp, ddt += kPerWarp) {
            Decay<ZOH> A[2];
            // the hold's 1 / A enters with its sign turned, so that dA's difference is a sum:
            // accB, accC, sB and dA come out turned too
            f2 invA[2], An[2], st[2], carry[2], dA[2], F[kPiece][2];
            f2 state[kPiece][2];  // the state before each token; with the hold g after it
            load_A<T, N, CH, ALIGNED, ZOH>(s, c * N + n0, A);
            load4x(&s.invA[c * N + n0], invA);
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
                    if (ZOH) {
                        st[k] = f2_fma(F[t][k], f2_fma(in, B[k], st[k]), st[k]);
                        state[t][k] = st[k];
                        accC[t][k] = f2_fma(dy, f2_mul(st[k], invA[k]), accC[t][k]);
                    } else {
                        state[t][k] = st[k];
                        st[k] = f2_fma(F[t][k], st[k], f2_mul(in, B[k]));
                        accC[t][k] = f2_fma(dy, st[k], accC[t][k]);
                    }
                }
            }
            load4x(&s.A[c * N + n0], An);
            if (ZOH)
#pragma unroll
                for (int k = 0; k < 2; ++k) An[k] = f2_mul(An[k], f2_both(1.f / 12.f));
            float vB[kPiece], vA[kPiece];
#pragma unroll
            for (int k = 0; k < 2; ++k) dA[k] = none;
#pragma unroll
            for (int t = kPiece - 1; t >= 0; --t) {
                const f2 dt = f2_both(ds[t]), dy = f2_both(ys[t]);
                const f2 u = f2_both(ZOH ? xs[t] : xs[t] * ds[t]);
                f2 B[2], C[2], sB = none, sA = none, sAB = none;
                load4x(&s.B[t0 + t][n0], B);
                load4x(&s.C[t0 + t][n0], C);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const f2 rv = f2_fma(dy, C[k], carry[k]);
                    const f2 ra = times_decay<ZOH>(rv, F[t][k]);
                    if (ZOH) {
                        const f2 wn = f2_mul(F[t][k], invA[k]), ru = f2_mul(rv, u);
                        const f2 rg = f2_mul(rv, state[t][k]), rB = f2_mul(rv, B[k]);
                        sB = k == 0 ? f2_mul(rB, wn) : f2_fma(rB, wn, sB);
                        accB[t][k] = f2_fma(ru, wn, accB[t][k]);
                        sA = k == 0 ? rg : f2_add(sA, rg);
                        sAB = k == 0 ? rB : f2_add(sAB, rB);
                        dA[k] = f2_fma(dt, rg, f2_fma(f2_mul(ru, B[k]),
                                                      dt_less_w(dt, F[t][k], wn, An[k]), dA[k]));
                    } else {
                        const f2 t1 = f2_mul(ra, state[t][k]);
                        sB = k == 0 ? f2_mul(rv, B[k]) : f2_fma(rv, B[k], sB);
                        accB[t][k] = f2_fma(rv, u, accB[t][k]);
                        sA = k == 0 ? f2_mul(An[k], t1) : f2_fma(An[k], t1, sA);
                        dA[k] = f2_fma(dt, t1, dA[k]);
                    }
                    carry[k] = ra;
                }
                float lo, hi;
                f2_unpack(sB, lo, hi);
                vB[t] = lo + hi;
                f2_unpack(ZOH ? f2_fma(u, sAB, sA) : sA, lo, hi);
                vA[t] = lo + hi;
            }
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (ZOH) dA[k] = f2_mul(invA[k], dA[k]);
            store4x(&s.P[piece][c * N + n0], dA);
            if (ZOH && (far >> c & 1)) {
                const float4 v = far_channel<T, N, CH, ALIGNED>(s, piece, c, n0);
                vA[0] = v.x, vA[1] = v.y, vA[2] = v.z, vA[3] = v.w;
            }
            // dx and ddt: each lane of the channel ends with the sums of its share of the tokens
            share_sums<kLanes>(vB, vA, lane);
            float db = 0.f, dd = 0.f;
            const float Ds = s.Ds[c];
#pragma unroll
            for (int j = 0; j < kShare; ++j) {
                const float sB = vB[j], x = s.x[c][share0 + j], y = s.dy[c][share0 + j];
                const float g = s.fac[c][share0 + j] * (ZOH ? vA[j] : fmaf(x, sB, vA[j]));
                if (share0 + j < p.n && c < here) {
                    dx[j * a.D] = fmaf(Ds, y, ZOH ? -sB : sB * s.dt[c][share0 + j]);
                    ddt[j * a.D] = g;
                    db += g;
                }
                dd = fmaf(x, y, dd);
            }
            db = lanes_sum<kLanes>(db);
            dd = lanes_sum<kLanes>(dd);
            if (lane % kLanes == 0) {
                s.db[piece][c] = db;
                s.dd[piece][c] = dd;
            }
        }
        __syncthreads();
        if (2 * tid < here * N) {
            float2 v = make_float2(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < kPieces; ++j) {
                const float2 q = *reinterpret_cast<const float2 *>(&s.P[j][2 * tid]);
                v.x += q.x;
                v.y += q.y;
            }
            if (ZOH) v = make_float2(-v.x, -v.y);
            *reinterpret_cast<float2 *>(&a.dA_part[(row + d0) * N + 2 * tid]) = v;
        }
        if (tid < here) {
            float2 v = make_float2(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < kPieces; ++j) {
                v.x += s.dd[j][tid];
                v.y += s.db[j][tid];
            }
            *reinterpret_cast<float2 *>(&a.d_part[(row + d0 + tid) * 2]) = v;
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
                *reinterpret_cast<float2 *>(&a.bc_part[(at * N + n0 + k) * 2]) =
                    ZOH ? make_float2(-vb, -vc) : make_float2(vb, vc);
            }
        }
}

// The last sums, a kernel: dB and dC over blocks of channels (blocks of threads
// [0, row_blocks)), then dA, and dDskip and the bias's gradient (the even and odd
// columns of d_part), over batch and chunks.
struct Sums {
    const float2 *rows;
    float *dB, *dC;
    int parts;
    int64_t n;  // b L G N
    const float *dA_part, *d_part;
    float *dA, *dD, *ddt_bias;
    int64_t chunks, wide_A, wide_d;
    unsigned row_blocks, A_blocks;
};
__global__ void __launch_bounds__(512) scan_bwd_finish(const Sums q) {
    after_previous();
    const int x = threadIdx.x, y = threadIdx.y, tid = y * 32 + x;
    if (blockIdx.x < q.row_blocks) {
        const int64_t i = (int64_t)blockIdx.x * 512 + tid;
        if (i >= q.n) return;
        float b = 0.f, c = 0.f;
#pragma unroll 4
        for (int j = 0; j < q.parts; ++j) {
            const float2 v = q.rows[j * q.n + i];
            b += v.x;
            c += v.y;
        }
        q.dB[i] = b;
        q.dC[i] = c;
        return;
    }
    const unsigned block = blockIdx.x - q.row_blocks;
    const bool is_A = block < q.A_blocks;
    const int64_t i = (int64_t)(is_A ? block : block - q.A_blocks) * 32 + x;
    const int64_t wide = is_A ? q.wide_A : q.wide_d;
    __shared__ float red[16][33];
    red[y][x] = column_sum(is_A ? q.dA_part : q.d_part, q.chunks, wide, i, y, 16);
    __syncthreads();
    if (y != 0 || i >= wide) return;
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) s += red[j][x];
    if (is_A) {
        q.dA[i] = s;
    } else {
        float *to = (i & 1) ? q.ddt_bias : q.dD;
        if (to) to[i / 2] = s;
    }
}

int64_t chunks(const Problem &pr) { return (pr.seqlen + kChunk - 1) / kChunk; }

// Tiles of channels that one thread block walks, up to eight (fewer sums of dB and dC,
// inputs a tile ahead): those that take the fewest rounds of `resident` thread blocks,
// each as long as its tiles and half a tile to begin and end.
void split(const Problem &pr, BwdArgs &a, int resident) {
    a.gch = pr.nheads / pr.ngroups;
    a.tiles_per_group = (int)((a.gch + kCh - 1) / kCh);
    const int64_t rows = pr.batch * chunks(pr) * pr.ngroups;
    int64_t least = INT64_MAX;
    for (int k = 8; k >= 1; --k) {
        const int64_t blocks = (a.tiles_per_group + k - 1) / k;
        const int64_t cost = (rows * blocks + resident - 1) / resident * (2 * k + 1);
        if (cost >= least) continue;
        least = cost;
        a.tiles_per_block = k;
        a.blocks_per_group = (int)blocks;
    }
}
constexpr int kSms = 148;  // the B200's: the workspace's size must not hang on a device
void split_main(const Problem &pr, BwdArgs &a) { split(pr, a, 2 * kSms); }

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

template <typename T, int N, bool ZOH, bool ALIGNED>
cudaError_t launch_first(const BwdArgs &first, const Maps &maps, cudaStream_t st) {
    constexpr auto *sums = scan_bwd_sums<T, N, ZOH, ALIGNED>;
    const int smem = (int)sizeof(Tile<T, N, kCh, ALIGNED>);
    const cudaError_t e =
        cudaFuncSetAttribute(sums, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    launch_begin("scan_bwd_sums", st);
    sums<<<(unsigned)(first.batch * first.nc * first.G * first.blocks_per_group), kCh * N / kQ, smem,
           st>>>(first, maps);
    launch_end(st);
    return cudaGetLastError();
}
template <typename T, int N, bool ZOH, bool ALIGNED>
cudaError_t launch_main(const BwdArgs &a, const Maps &maps, cudaStream_t st) {
    constexpr auto *main = scan_bwd_main<T, N, ZOH, ALIGNED>;
    const int smem = (int)sizeof(MainTile<T, N, kCh, ALIGNED>);
    const cudaError_t e =
        cudaFuncSetAttribute(main, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    launch_begin("scan_bwd_main", st);
    const cudaError_t l = launch_after(
        main, (unsigned)(a.batch * a.nc * a.G * a.blocks_per_group), kMainThreads, smem, st, a, maps);
    launch_end(st);
    return l;
}

// A map over a (b, L, D) tensor whose box is a tile of 32 channels by 32 tokens.
// False where rows, or groups of channels, do not start on 16 bytes.
template <typename T>
bool tile_map(CUtensorMap *m, const void *base, const BwdArgs &a) {
    const uint64_t row = (uint64_t)a.D * sizeof(T);
    if (!tensor_map_encoder() || reinterpret_cast<uintptr_t>(base) % 16 != 0 || row % 16 != 0 ||
        (a.G > 1 && a.gch * (int64_t)sizeof(T) % 16 != 0) || row * (uint64_t)a.L >= 1ull << 40)
        return false;
    const cuuint64_t dims[4] = {(cuuint64_t)a.D, (cuuint64_t)a.L, (cuuint64_t)a.batch, 1};
    const cuuint64_t strides[3] = {row, row * (uint64_t)a.L, row * (uint64_t)a.L};
    const cuuint32_t box[4] = {kCh, kChunk, 1, 1}, estr[4] = {1, 1, 1, 1};
    return tensor_map_encoder()(m,
                                sizeof(T) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                               : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                                4, const_cast<void *>(base), dims, strides, box, estr,
                                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                                CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int N, bool ZOH>
cudaError_t launch(const Problem &pr, BwdArgs a, const float *h0, const float *dh_final,
                   float *dA, float *dD, float *ddt_bias, float *dh0, cudaStream_t st) {
    BwdArgs first = a;
    split(pr, first, kSms * (640 / (kCh * N / kQ)));
    Maps maps;
    const bool aligned = tile_map<T>(&maps.m[0], a.x, a) && tile_map<T>(&maps.m[1], a.dt, a) &&
                         tile_map<T>(&maps.m[2], a.dy, a);
    cudaError_t e = aligned ? launch_first<T, N, ZOH, true>(first, maps, st)
                            : launch_first<T, N, ZOH, false>(first, maps, st);
    if (e != cudaSuccess) return e;
    const int64_t lanes = a.batch * a.D * N;
    launch_begin("scan_bwd_chain", st);
    e = launch_after(scan_bwd_chain<N, ZOH>, dim3((unsigned)((lanes + 127) / 128), 2), 128, 0, st, a,
                     h0, dh_final, dh0);
    launch_end(st);
    if (e != cudaSuccess) return e;
    e = aligned ? launch_main<T, N, ZOH, true>(a, maps, st) : launch_main<T, N, ZOH, false>(a, maps, st);
    if (e != cudaSuccess) return e;
    Sums q;
    q.rows = reinterpret_cast<const float2 *>(a.bc_part);
    q.dB = a.dB;
    q.dC = a.dC;
    q.parts = a.blocks_per_group;
    q.n = a.batch * a.L * a.G * N;
    q.dA_part = a.dA_part;
    q.d_part = a.d_part;
    q.dA = dA;
    q.dD = dD;
    q.ddt_bias = ddt_bias;
    q.chunks = a.batch * a.nc;
    q.wide_A = a.D * N;
    q.wide_d = 2 * a.D;
    q.row_blocks = (unsigned)((q.n + 511) / 512);
    q.A_blocks = (unsigned)((q.wide_A + 31) / 32);
    launch_begin("scan_bwd_finish", st);
    e = launch_after(scan_bwd_finish, q.row_blocks + q.A_blocks + (unsigned)((q.wide_d + 31) / 32),
                     dim3(32, 16), 0, st, q);
    launch_end(st);
    return e;
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
    split_main(pr, a);
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
    split_main(pr, a);
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
    a.words = ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(dt) |
                reinterpret_cast<uintptr_t>(dy)) & 3) == 0;
    a.err = device_error_word();
    a.wait = wait_limit_cycles();
    if (!a.err) return fail(SSD_ERR_CUDA, "cannot locate the device error word");
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
