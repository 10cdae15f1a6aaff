// The gated linear recurrence h <- a h + m sigmoid(i) x, one state per
// channel (arithmetic in gated.cuh), its backward pass and its one-token step.
//
// The sequence is cut into blocks of 64 tokens. A block maps the state that
// enters it to the one that leaves it by h -> P h + H, so the forward runs as
// three passes: every block's (P, H); the chain over blocks, which leaves the
// state entering each block; every block's outputs from that state. The
// backward pass is the same in reverse for the gradient G of each state,
//
//   G_t = dy_t + a_{t+1} G_{t+1}
//
// with what a block receives from its right, a_{t+1} G_{t+1}, as the chained
// quantity; its last pass recomputes the block's states from the saved one.
#include "gated.cuh"
#include "internal.h"

namespace ssd {
namespace {

using namespace gated;

constexpr int kThreads = 64;  // channels of a CUDA block

// The inputs of one (batch, block, channel): the I/O tensors, or with CK their
// 8-bit copies, int8 steps of 2^(code - 127) (code 255: the block held an
// infinity or a NaN and reads as NaN, 0 x inf).
template <typename T, bool CK>
struct Inputs {
    const T *v[3];
    const int8_t *q[3];
    float step[3];
    __device__ __forceinline__ float get(int w, int64_t off) const {
        return CK ? (float)q[w][off] * step[w] : to_f(v[w][off]);
    }
};

struct Where {
    int64_t b, blk, d, t0, row0;  // row0: offset of (b, t0, d) in a (b, L, D) tensor
    int n;                        // tokens
    bool ok;
};
__device__ __forceinline__ Where locate(int64_t L, int64_t D, int64_t nb, int64_t dblocks) {
    Where w;
    int64_t i = blockIdx.x;
    const int64_t db = i % dblocks;
    i /= dblocks;
    w.blk = i % nb;
    w.b = i / nb;
    w.d = db * kThreads + threadIdx.x;
    w.ok = w.d < D;
    if (!w.ok) w.d = D - 1;
    w.t0 = w.blk * kBlock;
    w.n = (int)(L - w.t0 < kBlock ? L - w.t0 : kBlock);
    w.row0 = (w.b * L + w.t0) * D + w.d;
    return w;
}

template <typename T, bool CK>
__device__ __forceinline__ Inputs<T, CK> inputs(const GatedArgs &a, const Where &w) {
    Inputs<T, CK> in;
    const void *v[3] = {a.x, a.r, a.i};
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        in.v[k] = static_cast<const T *>(v[k]);
        in.q[k] = CK ? a.q + k * a.batch * a.L * a.D : nullptr;
        in.step[k] = CK ? __uint_as_float((uint32_t)a.e[((k * a.batch + w.b) * a.nb + w.blk) * a.D +
                                                       w.d] << 23)
                        : 0.f;
    }
    return in;
}

__device__ __forceinline__ bool is_reset(const GatedArgs &a, const Where &w, int t) {
    return a.reset && a.reset[w.b * a.L + w.t0 + t];
}

template <typename T, bool CK>
__device__ __forceinline__ Gate token_gate(const GatedArgs &a, const Where &w,
                                           const Inputs<T, CK> &in, int t, float k) {
    const int64_t off = w.row0 + t * a.D;
    Gate g = gate<false>(in.get(1, off), in.get(2, off), k);
    if (is_reset(a, w, t)) {
        g.a = reset_decay();
        g.m2 = g.rm = 1.f;
    }
    return g;
}

// (P, H) of each block: forward h -> P h + H, or (BACK) the gradient received
// from the right -> the one handed to the left.
template <typename T, bool CK, bool BACK>
__global__ void __launch_bounds__(kThreads) gated_sums_kernel(const GatedArgs a) {
    const Where w = locate(a.L, a.D, a.nb, a.dblocks);
    const Inputs<T, CK> in = inputs<T, CK>(a, w);
    const float k = -a.c * softplus_full(a.lam[w.d]);
    float P = 1.f, H = 0.f;
    for (int j = 0; j < w.n; ++j) {
        const int t = BACK ? w.n - 1 - j : j;
        const int64_t off = w.row0 + t * a.D;
        const Gate g = token_gate<T, CK>(a, w, in, t, k);
        P *= g.a;
        H = BACK ? carry_on(g.a, to_f(static_cast<const T *>(a.dy)[off]) + H, 0.f)
                 : carry_on(g.a, H, g.m() * g.si * in.get(0, off));
    }
    if (w.ok) a.sums[(w.b * a.nb + w.blk) * a.D + w.d] = make_float2(P, H);
}

// The chain over blocks: what enters each one, and what leaves the last.
template <bool BACK>
__global__ void __launch_bounds__(kThreads)
gated_chain_kernel(const float2 *__restrict__ sums, const float *first, float *entering,
                   float *last, int64_t nb, int64_t D, int64_t lanes) {
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= lanes) return;
    const int64_t b = i / D, d = i % D;
    float h = first ? first[i] : 0.f;
    for (int64_t j = 0; j < nb; ++j) {
        const int64_t at = (b * nb + (BACK ? nb - 1 - j : j)) * D + d;
        entering[at] = h;
        const float2 s = sums[at];
        h = carry_on(s.x, h, s.y);
    }
    if (last) last[i] = h;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) gated_output_kernel(const GatedArgs a) {
    const Where w = locate(a.L, a.D, a.nb, a.dblocks);
    const Inputs<T, false> in = inputs<T, false>(a, w);
    const float k = -a.c * softplus_full(a.lam[w.d]);
    float h = a.states[(w.b * a.nb + w.blk) * a.D + w.d];
    for (int t = 0; t < w.n; ++t) {
        const int64_t off = w.row0 + t * a.D;
        const Gate g = token_gate<T, false>(a, w, in, t, k);
        h = carry_on(g.a, h, g.m() * g.si * in.get(0, off));
        if (w.ok) static_cast<T *>(a.y)[off] = from_f<T>(h);
    }
}

// The largest magnitude of a block as float bits -> the code of the least
// power of two whose 127-fold reaches it (255 for an infinity or a NaN).
__device__ __forceinline__ uint32_t step_code(uint32_t bits) {
    const uint32_t E = bits >> 23;
    if (E == 255) return 255;
    const int code = (int)E - 6 + ((bits & 0x7fffffu) > 0x7e0000u ? 1 : 0);
    return code < 1 ? 1u : (uint32_t)code;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) gated_pack_kernel(const GatedArgs a) {
    const Where w = locate(a.L, a.D, a.nb, a.dblocks);
    const Inputs<T, false> in = inputs<T, false>(a, w);
    for (int k = 0; k < 3; ++k) {
        uint32_t top = 0;
        for (int t = 0; t < w.n; ++t)
            top = max(top, __float_as_uint(in.get(k, w.row0 + t * a.D)) & 0x7fffffffu);
        const uint32_t code = step_code(top);
        const float inv = code == 255 ? 0.f : __uint_as_float((254u - code) << 23);
        if (!w.ok) continue;
        a.e[((k * a.batch + w.b) * a.nb + w.blk) * a.D + w.d] = (uint8_t)code;
        int8_t *q = a.q + k * a.batch * a.L * a.D;
        for (int t = 0; t < w.n; ++t) {
            const int64_t off = w.row0 + t * a.D;
            q[off] = code == 255 ? 0 : (int8_t)__float2int_rn(in.get(k, off) * inv);
        }
    }
}

template <typename T, bool CK>
__global__ void __launch_bounds__(kThreads) gated_gradient_kernel(const GatedArgs a) {
    __shared__ float before[kBlock][kThreads];
    const Where w = locate(a.L, a.D, a.nb, a.dblocks);
    const Inputs<T, CK> in = inputs<T, CK>(a, w);
    const float lam = a.lam[w.d], k = -a.c * softplus_full(lam);
    const int64_t at = (w.b * a.nb + w.blk) * a.D + w.d;
    float h = a.states[at];
    for (int t = 0; t < w.n; ++t) {
        const Gate g = token_gate<T, CK>(a, w, in, t, k);
        before[t][threadIdx.x] = h;
        h = carry_on(g.a, h, g.m() * g.si * in.get(0, w.row0 + t * a.D));
    }
    float carry = a.grads[at], dl = 0.f;
    for (int t = w.n - 1; t >= 0; --t) {
        const int64_t off = w.row0 + t * a.D;
        const Gate g = token_gate<T, CK>(a, w, in, t, k);
        const float x = in.get(0, off), G = to_f(static_cast<const T *>(a.dy)[off]) + carry;
        const float m = g.m(), v = g.si * x;
        // dlog a scaled by s: finite where s -> 0, though dm/ds is not
        const float e = is_reset(a, w, t)
                            ? 0.f
                            : G * (g.s * (g.a * before[t][threadIdx.x] - g.a * g.a * g.rm * v));
        carry = carry_on(g.a, G, 0.f);
        dl += e;
        if (w.ok) {
            static_cast<T *>(a.dx)[off] = from_f<T>(G * m * g.si);
            static_cast<T *>(a.dr)[off] = from_f<T>(e * (1.f - g.sr));
            static_cast<T *>(a.di)[off] = from_f<T>(G * m * v * (1.f - g.si));
        }
    }
    if (w.ok) a.dlam_part[at] = dl;
}

// dlam: the blocks' sums over batch and blocks, times the channel's factor.
__global__ void gated_dlam_kernel(const float *__restrict__ part, const float *__restrict__ lam,
                                  float *__restrict__ dlam, int64_t rows, int64_t D) {
    __shared__ float red[8][33];
    const int64_t d = (int64_t)blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    if (d < D)
        for (int64_t i = threadIdx.y; i < rows; i += 8) s += part[i * D + d];
    red[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && d < D) {
        for (int j = 1; j < 8; ++j) s += red[j][threadIdx.x];
        dlam[d] = s * lam_ratio(lam[d]);
    }
}

template <typename T>
__global__ void gated_step_kernel(float *__restrict__ h, const T *__restrict__ x,
                                  const T *__restrict__ r, const T *__restrict__ i,
                                  const float *__restrict__ lam, float c, T *__restrict__ y,
                                  int64_t D, int64_t n) {
    const int64_t at = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (at >= n) return;
    const Gate g = gate<false>(to_f(r[at]), to_f(i[at]), -c * softplus_full(lam[at % D]));
    const float v = fmaf(g.a, h[at], g.m() * g.si * to_f(x[at]));
    h[at] = v;
    y[at] = from_f<T>(v);
}

template <typename T>
cudaError_t forward_t(GatedArgs a, const float *h0, float *h_final, cudaStream_t st) {
    const unsigned grid = (unsigned)(a.dblocks * a.nb * a.batch);
    const int64_t lanes = a.batch * a.D;
    launch_begin("gated_sums", st);
    gated_sums_kernel<T, false, false><<<grid, kThreads, 0, st>>>(a);
    launch_end(st);
    launch_begin("gated_chain", st);
    gated_chain_kernel<false><<<(unsigned)((lanes + kThreads - 1) / kThreads), kThreads, 0, st>>>(
        a.sums, h0, a.states, h_final, a.nb, a.D, lanes);
    launch_end(st);
    launch_begin("gated_output", st);
    gated_output_kernel<T><<<grid, kThreads, 0, st>>>(a);
    launch_end(st);
    if (a.q) {
        launch_begin("gated_pack", st);
        gated_pack_kernel<T><<<grid, kThreads, 0, st>>>(a);
        launch_end(st);
    }
    return cudaGetLastError();
}

template <typename T, bool CK>
cudaError_t backward_t(GatedArgs a, const float *dh_final, float *dlam, float *dh0,
                       cudaStream_t st) {
    const unsigned grid = (unsigned)(a.dblocks * a.nb * a.batch);
    const int64_t lanes = a.batch * a.D;
    launch_begin("gated_sums_back", st);
    gated_sums_kernel<T, CK, true><<<grid, kThreads, 0, st>>>(a);
    launch_end(st);
    launch_begin("gated_chain_back", st);
    gated_chain_kernel<true><<<(unsigned)((lanes + kThreads - 1) / kThreads), kThreads, 0, st>>>(
        a.sums, dh_final, a.grads, dh0, a.nb, a.D, lanes);
    launch_end(st);
    launch_begin("gated_gradient", st);
    gated_gradient_kernel<T, CK><<<grid, kThreads, 0, st>>>(a);
    launch_end(st);
    launch_begin("gated_dlam", st);
    gated_dlam_kernel<<<(unsigned)((a.D + 31) / 32), dim3(32, 8), 0, st>>>(
        a.dlam_part, a.lam, dlam, a.batch * a.nb, a.D);
    launch_end(st);
    return cudaGetLastError();
}

}  // namespace

int64_t gated_blocks(const Problem &pr) { return (pr.seqlen + kBlock - 1) / kBlock; }

// (P, H) and the entering state (or gradient) of every block, and in the
// backward pass its sum of dlam.
size_t gated_workspace_bytes(const Problem &pr, bool back) {
    const size_t n = (size_t)(pr.batch * gated_blocks(pr) * pr.nheads);
    return align256(n * sizeof(float2)) + (back ? 2 : 1) * align256(n * sizeof(float));
}

static void carve(const Problem &pr, GatedArgs &a, void *ws, bool back) {
    a.batch = pr.batch;
    a.L = pr.seqlen;
    a.D = pr.nheads;
    a.nb = gated_blocks(pr);
    a.dblocks = (a.D + kThreads - 1) / kThreads;
    const size_t n = (size_t)(a.batch * a.nb * a.D);
    char *p = static_cast<char *>(ws);
    a.sums = reinterpret_cast<float2 *>(p);
    p += align256(n * sizeof(float2));
    if (back) {
        a.grads = reinterpret_cast<float *>(p);
        a.dlam_part = reinterpret_cast<float *>(p + align256(n * sizeof(float)));
    } else if (!a.states) {
        a.states = reinterpret_cast<float *>(p);
    }
}

ssd_status gated_forward_launch(const Problem &pr, GatedArgs a, const float *h0, float *h_final,
                                void *ws, cudaStream_t st) {
    const int64_t lanes = pr.batch * pr.nheads;
    cudaError_t e = cudaSuccess;
    if (pr.seqlen == 0) {
        if (h_final && h0 && h0 != h_final)
            e = cudaMemcpyAsync(h_final, h0, (size_t)lanes * 4, cudaMemcpyDeviceToDevice, st);
        else if (h_final && !h0)
            e = cudaMemsetAsync(h_final, 0, (size_t)lanes * 4, st);
    } else {
        carve(pr, a, ws, false);
        e = pr.dtype == SSD_F32 ? forward_t<float>(a, h0, h_final, st)
                                : forward_t<__nv_bfloat16>(a, h0, h_final, st);
    }
    return e == cudaSuccess ? SSD_OK : cuda_fail(e, "gated scan launch");
}

ssd_status gated_backward_launch(const Problem &pr, GatedArgs a, const float *dh_final,
                                 float *dlam, float *dh0, void *ws, cudaStream_t st) {
    const int64_t lanes = pr.batch * pr.nheads;
    cudaError_t e = cudaSuccess;
    if (pr.seqlen == 0) {
        e = cudaMemsetAsync(dlam, 0, (size_t)pr.nheads * 4, st);
        if (e == cudaSuccess && dh0 && dh_final && dh0 != dh_final)
            e = cudaMemcpyAsync(dh0, dh_final, (size_t)lanes * 4, cudaMemcpyDeviceToDevice, st);
        else if (e == cudaSuccess && dh0 && !dh_final)
            e = cudaMemsetAsync(dh0, 0, (size_t)lanes * 4, st);
    } else {
        carve(pr, a, ws, true);
        if (pr.dtype == SSD_F32)
            e = a.q ? backward_t<float, true>(a, dh_final, dlam, dh0, st)
                    : backward_t<float, false>(a, dh_final, dlam, dh0, st);
        else
            e = a.q ? backward_t<__nv_bfloat16, true>(a, dh_final, dlam, dh0, st)
                    : backward_t<__nv_bfloat16, false>(a, dh_final, dlam, dh0, st);
    }
    return e == cudaSuccess ? SSD_OK : cuda_fail(e, "gated scan backward launch");
}

ssd_status gated_step_launch(const Problem &pr, float *h, const void *x, const void *r,
                             const void *i, const float *lam, float c, void *y, cudaStream_t st) {
    const int64_t n = pr.batch * pr.nheads;
    const unsigned grid = (unsigned)((n + 127) / 128);
    using bf = __nv_bfloat16;
    launch_begin("gated_step", st);
    if (pr.dtype == SSD_F32)
        gated_step_kernel<float><<<grid, 128, 0, st>>>(h, (const float *)x, (const float *)r,
                                                       (const float *)i, lam, c, (float *)y,
                                                       pr.nheads, n);
    else
        gated_step_kernel<bf><<<grid, 128, 0, st>>>(h, (const bf *)x, (const bf *)r, (const bf *)i,
                                                    lam, c, (bf *)y, pr.nheads, n);
    launch_end(st);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SSD_OK : cuda_fail(e, "gated step launch");
}

}  // namespace ssd
