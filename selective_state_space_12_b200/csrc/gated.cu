// The gated linear recurrence h <- a h + m sigmoid(i) x, one state per
// channel (arithmetic in gated.cuh), its backward pass and its one-token step.
//
// A tile is one block of 64 tokens by 64 channels: eight warps of eight tokens,
// two channels a lane. It maps the state that enters it to the one that leaves
// it by h -> P h + H, so all tiles work at once, in one pass over the data:
// a tile computes its gates, folds its (P, H), finds the state that enters it
// by looking back over the tiles before it (below), and then writes its
// outputs from values it still holds. The backward pass is the same in reverse
// for the gradient G of each state,
//
//   G_t = dy_t + a_{t+1} G_{t+1}
//
// with a_{t+1} G_{t+1} as what a tile receives from its right; the states
// before its tokens it recomputes from the saved one, at the tile's start.
//
// Looking back. Tiles are handed out by a counter, all channels of a block of
// tokens before the next block, so that whoever holds a tile knows that the
// tiles before it are done or held by a running thread block. A ninth warp
// folds the maps of a tile's eight runs. If the tile before has published what
// leaves it, that is what enters; if not, the warp publishes its own (P, H),
// and waits for some tile among the kWindow before it that has published its
// end, all between them their (P, H), and folds these in order. What enters a
// tile is the same fold whichever tile it starts from: results do not depend on
// the timing. A published word is 64 bits, cleared to all ones before the
// kernel, and is complete once it differs from that: readers poll the data
// itself, one trip to L2, and no fence stands between data and flag. Waits are
// bounded; one that runs out tells the others and all return.
#include <type_traits>

#include "gated.cuh"
#include "internal.h"

namespace ssd {
namespace {

using namespace gated;

constexpr int kWarps = 8;                  // warps that compute
constexpr int kCompute = 32 * kWarps;
constexpr int kThreads = kCompute + 32;    // and the one that folds and looks back
constexpr int kRun = kBlock / kWarps;  // tokens of a warp
constexpr int kTileCh = 64;            // channels of a tile, two a lane
constexpr int kWindow = 8;             // tiles that a look reaches back

// Barriers of the compute warps and the chain warp.
enum { kMapsReady = 1, kEntryReady = 2 };
__device__ __forceinline__ void bar_sync(int id) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(kThreads) : "memory");
}
__device__ __forceinline__ void bar_arrive(int id) {
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "n"(kThreads) : "memory");
}

// ------------------------------------------------------------ global words

using word = unsigned long long;
constexpr word kEmpty = ~0ull;

__device__ __forceinline__ word load_word(const word *p) {
    word v;
    asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void store_word(word *p, float lo, float hi) {
    word v = f2_pack(lo, hi);
    if (v == kEmpty) v = 0x7fffffff7fffffffull;  // two NaNs all the same
    asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p), "l"(v) : "memory");
}
__device__ __forceinline__ unsigned load_relaxed(const unsigned *p) {
    unsigned v;
    asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

struct Tile {
    int64_t b, blk, row0;  // row0: offset of (b, first token, 0) in a (b, L, D) tensor
    int64_t id;            // index of its record
    int d0, n;             // first channel, tokens
};
template <bool BACK>
__device__ __forceinline__ Tile tile_of(const GatedArgs &a, unsigned ticket) {
    Tile t;
    const unsigned lanes = (unsigned)(a.batch * a.dblocks);
    const unsigned step = ticket / lanes, lane = ticket % lanes;
    t.b = lane / (unsigned)a.dblocks;
    t.d0 = (int)(lane % (unsigned)a.dblocks) * kTileCh;
    t.blk = BACK ? a.nb - 1 - step : step;
    t.row0 = (t.b * a.L + t.blk * kBlock) * a.D;
    const int64_t left = a.L - t.blk * kBlock;
    t.n = (int)(left < kBlock ? left : kBlock);
    t.id = ticket;
    return t;
}

// ------------------------------------------------------------ two channels

// A lane's two channels: adjacent with VEC (one load; D even, aligned), else
// 32 apart (two loads that neighbouring lanes continue).
template <bool VEC>
__device__ __forceinline__ int channel(int j) {
    const int lane = threadIdx.x & 31;
    return VEC ? 2 * lane + j : lane + 32 * j;
}

template <typename T>
struct Pair;  // storage of two adjacent elements
template <>
struct Pair<float> {
    using type = float2;
};
template <>
struct Pair<__nv_bfloat16> {
    using type = uint32_t;
};
__device__ __forceinline__ f2 widen(float2 v) { return f2_pack(v.x, v.y); }
__device__ __forceinline__ f2 widen(uint32_t v) {
    return f2_pack(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

template <typename T>
__device__ __forceinline__ typename Pair<T>::type raw_pair(const void *p, int64_t row,
                                                           const GatedArgs &a, int d0) {
    const T *v = static_cast<const T *>(p) + row;
    const int c0 = d0 + channel<false>(0), c1 = d0 + channel<false>(1);
    const T lo = c0 < a.D ? v[c0] : from_f<T>(0.f), hi = c1 < a.D ? v[c1] : from_f<T>(0.f);
    if constexpr (sizeof(T) == 4)
        return make_float2(lo, hi);
    else
        return (uint32_t)__bfloat16_as_ushort(lo) | (uint32_t)__bfloat16_as_ushort(hi) << 16;
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_pair(void *p, int64_t row, const GatedArgs &a, int d0,
                                           f2 val) {
    T *v = static_cast<T *>(p) + row;
    float lo, hi;
    f2_unpack(val, lo, hi);
    const int c0 = d0 + channel<VEC>(0), c1 = d0 + channel<VEC>(1);
    if constexpr (VEC) {
        if (c0 >= a.D) return;
        if constexpr (sizeof(T) == 4)
            *reinterpret_cast<float2 *>(v + c0) = make_float2(lo, hi);
        else
            *reinterpret_cast<uint32_t *>(v + c0) = tc::pack_bf16(lo, hi);
    } else {
        if (c0 < a.D) v[c0] = from_f<T>(lo);
        if (c1 < a.D) v[c1] = from_f<T>(hi);
    }
}

// ------------------------------------------------------------ staged inputs

// With VEC, each thread copies the pairs it will read itself, a tile ahead
// and asynchronously, to its own words of shared memory: no registers and no
// barriers are spent on them.
template <typename T, bool VEC, int TENSORS>
struct Stage {
    using P = typename Pair<T>::type;
    static constexpr size_t kBytes = VEC ? sizeof(P) * TENSORS * kRun * kCompute : 16;

    static __device__ __forceinline__ P *own(unsigned char *s, int w, int t) {
        return reinterpret_cast<P *>(s) + (w * kRun + t) * kCompute + threadIdx.x;
    }
    static __device__ __forceinline__ void request(unsigned char *s, const GatedArgs &a,
                                                   const Tile &t, const void *const (&src)[TENSORS]) {
        if constexpr (VEC) {
            const int tok0 = (threadIdx.x >> 5) * kRun, c = t.d0 + channel<true>(0);
#pragma unroll
            for (int w = 0; w < TENSORS; ++w)
#pragma unroll
                for (int j = 0; j < kRun; ++j) {
                    const bool ok = tok0 + j < t.n && c < a.D;
                    const T *from = static_cast<const T *>(src[w]) +
                                    (ok ? t.row0 + (tok0 + j) * a.D + c : 0);
                    const uint32_t to = (uint32_t)__cvta_generic_to_shared(own(s, w, j));
                    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(to), "l"(from),
                                 "n"((int)sizeof(P)), "r"(ok ? (int)sizeof(P) : 0)
                                 : "memory");
                }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    }
    static __device__ __forceinline__ void wait() {
        if constexpr (VEC) asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    static __device__ __forceinline__ P raw(unsigned char *s, const GatedArgs &a, const Tile &t,
                                            const void *src, int w, int j) {
        if constexpr (VEC) {
            return *own(s, w, j);
        } else {
            const int tok = (threadIdx.x >> 5) * kRun + j;
            return tok < t.n ? raw_pair<T>(src, t.row0 + tok * a.D, a, t.d0) : P{};
        }
    }
};

// Reset marks of the warp's tokens, one bit each.
__device__ __forceinline__ unsigned reset_byte(const GatedArgs &a, const Tile &t) {
    const int lane = threadIdx.x & 31, tok = (threadIdx.x >> 5) * kRun + lane;
    if (!a.reset || lane >= kRun || tok >= t.n) return 0;
    return a.reset[t.b * a.L + t.blk * kBlock + tok];
}

// ------------------------------------------------------------ folding

// (P, H) of the lane's two channels: {P0, H0, P1, H1}.
__device__ __forceinline__ f2 apply(float4 m, f2 h) {
    float h0, h1;
    f2_unpack(h, h0, h1);
    return f2_pack(carry_on(m.x, h0, m.y), carry_on(m.z, h1, m.w));
}
__device__ __forceinline__ float4 as_map(f2 P, f2 H) {
    float4 m;
    f2_unpack(P, m.x, m.z);
    f2_unpack(H, m.y, m.w);
    return m;
}
__device__ __forceinline__ float4 then(float4 first, float4 next) {
    return make_float4(chain_decay(first.x, next.x), carry_on(next.x, first.y, next.y),
                       chain_decay(first.z, next.z), carry_on(next.z, first.w, next.w));
}

// What enters tile `id`, the step-th of its lane (step > 0), for this lane's
// channels, `before` the word of the tile before as read earlier. False when a
// wait ran out (here or elsewhere).
__device__ __forceinline__ bool look_back(const GatedArgs &a, int64_t id, unsigned step,
                                          int64_t lanes, float4 map, word before, f2 &in) {
    const int lane = threadIdx.x & 31;
    bool done = before != kEmpty;
    in = before;
    if (__all_sync(0xffffffffu, done)) return true;
    store_word(&a.maps[(id * 32 + lane) * 2], map.x, map.y);
    store_word(&a.maps[(id * 32 + lane) * 2 + 1], map.z, map.w);
    const long long began = clock64();
    while (true) {
        word e[kWindow], m0[kWindow - 1], m1[kWindow - 1];
#pragma unroll
        for (int j = 0; j < kWindow; ++j) {
            const int64_t at = (id - (j + 1) * lanes) * 32 + lane;
            e[j] = (unsigned)j < step ? load_word(&a.ends[at]) : kEmpty;
            if (j + 1 < kWindow) {
                m0[j] = (unsigned)j < step ? load_word(&a.maps[at * 2]) : kEmpty;
                m1[j] = (unsigned)j < step ? load_word(&a.maps[at * 2 + 1]) : kEmpty;
            }
        }
        if (!done) {
            int from = kWindow;  // the nearest tile with an end, and maps up to it
#pragma unroll
            for (int j = kWindow - 1; j >= 0; --j) {
                if (e[j] != kEmpty) from = j;
                else if (j + 1 < kWindow && (m0[j] == kEmpty || m1[j] == kEmpty)) from = kWindow;
            }
            if (from < kWindow) {
                done = true;
#pragma unroll
                for (int j = kWindow - 1; j >= 0; --j) {
                    if (j == from) in = e[j];
                    if (j + 1 < kWindow && j < from) {
                        float4 m;
                        f2_unpack(m0[j], m.x, m.y);
                        f2_unpack(m1[j], m.z, m.w);
                        in = apply(m, in);
                    }
                }
            }
        }
        if (__all_sync(0xffffffffu, done)) return true;
        bool stop = false;
        if (lane == 0) {
            stop = clock64() - began > a.wait || load_relaxed(a.abort) != 0;
            if (stop) {
                atomicExch(a.err, 0x6a7ed001u);
                atomicExch(a.abort, 1u);
            }
        }
        if (__shfl_sync(0xffffffffu, stop, 0)) return false;
    }
}

template <bool VEC>
__device__ __forceinline__ f2 read_state(const float *p, int64_t row, int d0, int64_t D) {
    const int c0 = d0 + channel<VEC>(0), c1 = d0 + channel<VEC>(1);
    return f2_pack(p && c0 < D ? p[row + c0] : 0.f, p && c1 < D ? p[row + c1] : 0.f);
}
template <bool VEC>
__device__ __forceinline__ void write_state(float *p, int64_t row, int d0, int64_t D, f2 v) {
    const int c0 = d0 + channel<VEC>(0), c1 = d0 + channel<VEC>(1);
    float lo, hi;
    f2_unpack(v, lo, hi);
    if (c0 < D) p[row + c0] = lo;
    if (c1 < D) p[row + c1] = hi;
}

struct Shared {
    float4 maps[kWarps][32];   // (P, H) of each run: {P0, H0, P1, H1}
    float2 right[kWarps][32];  // backward: R of each run
    f2 entry[kWarps][32];      // the state entering each run
    f2 grad[kWarps][32];       // backward: the gradient entering it from its right
    float k[2][kTileCh];       // -c softplus(lam), of this and the next tile
    float dlam[2][kWarps][kTileCh];
    unsigned top[2][3][kTileCh];  // 8-bit copies: largest magnitudes
    unsigned code[3][kTileCh];
    unsigned ticket[2];        // of this and the next tile
    int stop;
};

template <bool VEC>
__device__ __forceinline__ void gate_scales(const GatedArgs &a, int d0, float *k) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int c = channel<VEC>(j);
        k[c] = d0 + c < a.D ? -a.c * softplus_full(a.lam[d0 + c]) : 0.f;
    }
}
__device__ __forceinline__ bool all_fast(f2 k) {
    float lo, hi;
    f2_unpack(k, lo, hi);
    return __all_sync(0xffffffffu, lo >= kSeries && hi >= kSeries);
}

// ------------------------------------------------------------ 8-bit copies

// The largest magnitude of a block as float bits -> the code of the least
// power of two whose 127-fold reaches it (255 for an infinity or a NaN).
__device__ __forceinline__ uint32_t step_code(uint32_t bits) {
    const uint32_t E = bits >> 23;
    if (E == 255) return 255;
    const int code = (int)E - 6 + ((bits & 0x7fffffu) > 0x7e0000u ? 1 : 0);
    return code < 1 ? 1u : (uint32_t)code;
}
__device__ __forceinline__ int8_t in_steps(float v, uint32_t code) {
    return code == 255 ? 0 : (int8_t)__float2int_rn(v * __uint_as_float((254u - code) << 23));
}

// ------------------------------------------------------------ chain warp

// The ninth warp: for each tile of this thread block, folds its runs' maps,
// finds what enters it, hands every run what enters that, and publishes what
// leaves. While the others compute a tile it fetches the next ticket and
// prepares the next tile's gate scales.
template <bool VEC, bool CK, bool BACK>
__device__ __forceinline__ void chain_warp(const GatedArgs &a, Shared &s, unsigned tiles,
                                           int64_t lanes) {
    const int lane = threadIdx.x & 31;
    const bool chained = a.nb > 1;
    unsigned now = s.ticket[0], next = s.ticket[1];
    int64_t last_row = -1;  // dlam of the tile before: its row and channels
    int last_d0 = 0;
    auto flush = [&](int slot) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int c = channel<VEC>(j);
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) sum += s.dlam[slot][w][c];
            if (last_d0 + c < a.D) a.dlam_part[last_row + last_d0 + c] = sum;
        }
    };
    for (int n = 0; now < tiles; ++n) {
        const Tile t = tile_of<BACK>(a, now);
        const unsigned step = (unsigned)(BACK ? a.nb - 1 - t.blk : t.blk);
        unsigned after = tiles;
        if (next < tiles) {
            if (lane == 0) after = atomicAdd(a.counter, 1u);
            gate_scales<VEC>(a, tile_of<BACK>(a, next).d0, s.k[(n + 1) & 1]);
            after = __shfl_sync(0xffffffffu, after, 0);
        }
        f2 in = 0, h = 0;
        word before = kEmpty;
        if (step == 0) in = read_state<VEC>(a.first, t.b * a.D, t.d0, a.D);
        else before = load_word(&a.ends[(t.id - lanes) * 32 + lane]);
        if (BACK) h = read_state<VEC>(a.states, (t.b * a.nb + t.blk) * a.D, t.d0, a.D);
        bar_sync(kMapsReady);
        if (BACK && last_row >= 0) flush((n + 1) & 1);
        float4 m[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            m[w] = s.maps[w][lane];
            if (BACK) {
                s.entry[w][lane] = h;
                h = apply(m[w], h);
                const float2 r = s.right[w][lane];
                m[w].y = r.x;
                m[w].w = r.y;
            }
        }
        float4 all = m[BACK ? kWarps - 1 : 0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) all = then(all, m[BACK ? kWarps - 1 - w : w]);
        if (step > 0 && !look_back(a, t.id, step, lanes, all, before, in)) {
            if (lane == 0) s.stop = 1;
            __syncwarp();
            bar_arrive(kEntryReady);
            return;
        }
        const f2 out = apply(all, in);
        if (chained && step + 1 < a.nb) {
            float2 e;
            f2_unpack(out, e.x, e.y);
            store_word(&a.ends[t.id * 32 + lane], e.x, e.y);
        }
        f2 run = in;
#pragma unroll
        for (int j = 0; j < kWarps; ++j) {
            const int w = BACK ? kWarps - 1 - j : j;
            (BACK ? s.grad : s.entry)[w][lane] = run;
            run = apply(m[w], run);
        }
        if (CK && !BACK) {
#pragma unroll
            for (int w = 0; w < 3; ++w)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int c = channel<VEC>(j);
                    const uint32_t code = step_code(s.top[n & 1][w][c]);
                    s.code[w][c] = code;
                    s.top[n & 1][w][c] = 0;
                    if (t.d0 + c < a.D)
                        a.e[((w * a.batch + t.b) * a.nb + t.blk) * a.D + t.d0 + c] = (uint8_t)code;
                }
        }
        if (lane == 0) s.ticket[n & 1] = after;
        __syncwarp();
        bar_arrive(kEntryReady);
        if (!BACK && a.states)
            write_state<VEC>(a.states, (t.b * a.nb + t.blk) * a.D, t.d0, a.D, in);
        if (a.last && step + 1 == a.nb) write_state<VEC>(a.last, t.b * a.D, t.d0, a.D, out);
        last_row = (t.b * a.nb + t.blk) * a.D;
        last_d0 = t.d0;
        now = next;
        next = after;
        if (BACK && now >= tiles) {
            bar_sync(kMapsReady);
            flush(n & 1);
        }
    }
}

// The first two tickets of this thread block, and its first gate scales.
template <bool VEC, bool BACK>
__device__ __forceinline__ void open_block(const GatedArgs &a, Shared &s, unsigned tiles) {
    if (threadIdx.x == 0) {
        s.stop = 0;
        if (a.nb > 1) {
            s.ticket[0] = atomicAdd(a.counter, 1u);
            s.ticket[1] = atomicAdd(a.counter, 1u);
        } else {  // one block of tokens: a tile a thread block
            s.ticket[0] = blockIdx.x;
            s.ticket[1] = tiles;
        }
    }
    for (int i = threadIdx.x; i < 2 * 3 * kTileCh; i += kThreads) (&s.top[0][0][0])[i] = 0;
    __syncthreads();
    if (threadIdx.x >= kCompute && s.ticket[0] < tiles)
        gate_scales<VEC>(a, tile_of<BACK>(a, s.ticket[0]).d0, s.k[0]);
    __syncthreads();
}

// ------------------------------------------------------------ forward

template <typename T, bool VEC, bool CK>
__global__ void __launch_bounds__(kThreads, CK ? 2 : 3) gated_forward_kernel(const GatedArgs a) {
    extern __shared__ __align__(16) unsigned char staged[];
    __shared__ Shared s;
    using In = Stage<T, VEC, 3>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t lanes = a.batch * a.dblocks;
    const unsigned tiles = (unsigned)(lanes * a.nb);
    open_block<VEC, false>(a, s, tiles);
    if (warp == kWarps) {
        chain_warp<VEC, CK, false>(a, s, tiles, lanes);
        return;
    }
    const void *const src[3] = {a.x, a.r, a.i};
    unsigned now = s.ticket[0], next = s.ticket[1];
    if (now >= tiles) return;
    Tile t = tile_of<false>(a, now);
    In::request(staged, a, t, src);
    unsigned mark = reset_byte(a, t);
    const int tok0 = warp * kRun;
    for (int n = 0;; ++n) {
        const f2 k = f2_pack(s.k[n & 1][channel<VEC>(0)], s.k[n & 1][channel<VEC>(1)]);
        const bool fast = all_fast(k);
        const unsigned marks = __ballot_sync(0xffffffffu, mark != 0);
        const int left = t.n - tok0;
        In::wait();
        typename Pair<T>::type v[3][kRun];
        f2 av[kRun], u[kRun];
        f2 P = f2_both(1.f), H = f2_both(0.f);
        auto gates = [&](auto is_fast) {
#pragma unroll
            for (int j = 0; j < kRun; ++j) {
#pragma unroll
                for (int w = 0; w < 3; ++w) v[w][j] = In::raw(staged, a, t, src[w], w, j);
                const Gate2 g = gate2<decltype(is_fast)::value>(widen(v[1][j]), widen(v[2][j]), k);
                const f2 ix = f2_mul(g.si, widen(v[0][j]));
                if (marks >> j & 1) {
                    av[j] = P = f2_both(reset_decay());
                    H = u[j] = ix;
                } else if (j < left) {
                    av[j] = g.a;
                    u[j] = f2_mul(g.m, ix);
                    H = f2_fma(g.a, H, u[j]);
                    P = f2_mul(P, g.a);
                } else {
                    av[j] = f2_both(1.f);
                    u[j] = f2_both(0.f);
                }
            }
        };
        if (fast) gates(std::true_type{});
        else gates(std::false_type{});
        if (CK) {
#pragma unroll
            for (int w = 0; w < 3; ++w) {
                uint32_t m0 = 0, m1 = 0;
#pragma unroll
                for (int j = 0; j < kRun; ++j) {
                    const f2 f = widen(v[w][j]);
                    m0 = max(m0, (uint32_t)f & 0x7fffffffu);
                    m1 = max(m1, (uint32_t)(f >> 32) & 0x7fffffffu);
                }
                atomicMax(&s.top[n & 1][w][channel<VEC>(0)], m0);
                atomicMax(&s.top[n & 1][w][channel<VEC>(1)], m1);
            }
        }
        s.maps[warp][lane] = as_map(P, H);
        bar_arrive(kMapsReady);
        Tile tn = t;
        if (next < tiles) {  // the next tile's inputs are on their way while this one waits
            tn = tile_of<false>(a, next);
            In::request(staged, a, tn, src);
            mark = reset_byte(a, tn);
        }
        bar_sync(kEntryReady);
        if (s.stop) break;
        const unsigned after = s.ticket[n & 1];
        f2 h = s.entry[warp][lane];
#pragma unroll
        for (int j = 0; j < kRun; ++j) {
            h = (marks >> j & 1) ? u[j] : f2_fma(av[j], h, u[j]);
            if (j < left) store_pair<T, VEC>(a.y, t.row0 + (tok0 + j) * a.D, a, t.d0, h);
        }
        if (CK) {
#pragma unroll
            for (int w = 0; w < 3; ++w) {
                const int c0 = channel<VEC>(0), c1 = channel<VEC>(1);
                const uint32_t k0 = s.code[w][c0], k1 = s.code[w][c1];
                int8_t *q = a.q + w * a.batch * a.L * a.D + t.row0 + t.d0;
#pragma unroll
                for (int j = 0; j < kRun; ++j) {
                    float lo, hi;
                    f2_unpack(widen(v[w][j]), lo, hi);
                    const int8_t q0 = in_steps(lo, k0), q1 = in_steps(hi, k1);
                    int8_t *to = q + (tok0 + j) * a.D;
                    if (j >= left) continue;
                    if (VEC && t.d0 + c0 < a.D) {
                        *reinterpret_cast<char2 *>(to + c0) = make_char2(q0, q1);
                    } else if (!VEC) {
                        if (t.d0 + c0 < a.D) to[c0] = q0;
                        if (t.d0 + c1 < a.D) to[c1] = q1;
                    }
                }
            }
        }
        if (next >= tiles) break;
        t = tn;
        next = after;
    }
    In::wait();  // nothing may be in flight to shared memory at the end
}

// ------------------------------------------------------------ backward

// A pair of an 8-bit copy: int8 steps.
template <bool VEC>
__device__ __forceinline__ char2 copy_pair(const GatedArgs &a, const Tile &t, int w, int tok) {
    if (tok >= t.n) return make_char2(0, 0);
    const int8_t *q = a.q + w * a.batch * a.L * a.D + t.row0 + tok * a.D + t.d0;
    const int c0 = channel<VEC>(0), c1 = channel<VEC>(1);
    if (VEC)
        return t.d0 + c0 < a.D ? *reinterpret_cast<const char2 *>(q + c0) : make_char2(0, 0);
    return make_char2(t.d0 + c0 < a.D ? q[c0] : 0, t.d0 + c1 < a.D ? q[c1] : 0);
}
template <bool VEC>
__device__ __forceinline__ f2 copy_step(const GatedArgs &a, const Tile &t, int w) {
    const uint8_t *e = a.e + ((w * a.batch + t.b) * a.nb + t.blk) * a.D + t.d0;
    const int c0 = channel<VEC>(0), c1 = channel<VEC>(1);
    return f2_pack(t.d0 + c0 < a.D ? __uint_as_float((uint32_t)e[c0] << 23) : 0.f,
                   t.d0 + c1 < a.D ? __uint_as_float((uint32_t)e[c1] << 23) : 0.f);
}
__device__ __forceinline__ f2 widen(char2 v) { return f2_pack((float)v.x, (float)v.y); }

template <typename T, bool VEC, bool CK>
__global__ void __launch_bounds__(kThreads, 2) gated_backward_kernel(const GatedArgs a) {
    extern __shared__ __align__(16) unsigned char staged[];
    __shared__ Shared s;
    constexpr int kIn = CK ? 1 : 4;
    using In = Stage<T, VEC, kIn>;
    using P2 = typename Pair<T>::type;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t lanes = a.batch * a.dblocks;
    const unsigned tiles = (unsigned)(lanes * a.nb);
    open_block<VEC, true>(a, s, tiles);
    if (warp == kWarps) {
        chain_warp<VEC, CK, true>(a, s, tiles, lanes);
        return;
    }
    const void *src[kIn];
    src[0] = a.dy;
    if constexpr (!CK) {
        src[1] = a.r;
        src[2] = a.i;
        src[3] = a.x;
    }
    unsigned now = s.ticket[0], next = s.ticket[1];
    if (now >= tiles) return;
    Tile t = tile_of<true>(a, now);
    In::request(staged, a, t, src);
    unsigned mark = reset_byte(a, t);
    const int tok0 = warp * kRun;
    const f2 one = f2_both(1.f), none = f2_both(0.f);
    for (int n = 0;; ++n) {
        const f2 k = f2_pack(s.k[n & 1][channel<VEC>(0)], s.k[n & 1][channel<VEC>(1)]);
        const bool fast = all_fast(k);
        const unsigned marks = __ballot_sync(0xffffffffu, mark != 0);
        const int left = t.n - tok0;
        // kept until the gradients: dy, x (as stored) and the two sigmoids
        std::conditional_t<CK, char2, P2> xr[kRun];
        P2 dyr[kRun];
        f2 sr[kRun], si[kRun], steps[3];
        if (CK) {
#pragma unroll
            for (int w = 0; w < 3; ++w) steps[w] = copy_step<VEC>(a, t, w);
        }
        auto xv = [&](int j) { return CK ? f2_mul(widen(xr[j]), steps[0]) : widen(xr[j]); };
        In::wait();
        f2 P = f2_both(1.f), H = none, R = none;
        auto gates = [&](auto is_fast) {
#pragma unroll
            for (int j = 0; j < kRun; ++j) {
                f2 rv, iv;
                dyr[j] = In::raw(staged, a, t, src[0], 0, j);
                if constexpr (CK) {
                    xr[j] = copy_pair<VEC>(a, t, 0, tok0 + j);
                    rv = f2_mul(widen(copy_pair<VEC>(a, t, 1, tok0 + j)), steps[1]);
                    iv = f2_mul(widen(copy_pair<VEC>(a, t, 2, tok0 + j)), steps[2]);
                } else {
                    rv = widen(In::raw(staged, a, t, src[1], 1, j));
                    iv = widen(In::raw(staged, a, t, src[2], 2, j));
                    xr[j] = In::raw(staged, a, t, src[3], 3, j);
                }
                const Gate2 g = gate2<decltype(is_fast)::value>(rv, iv, k);
                sr[j] = g.sr;
                si[j] = g.si;
                const f2 vx = f2_mul(g.si, xv(j));
                if (marks >> j & 1) {
                    P = f2_both(reset_decay());
                    H = vx;
                } else if (j < left) {
                    H = f2_fma(g.a, H, f2_mul(g.m, vx));
                    P = f2_mul(P, g.a);
                    // R: dy times the decays up to and with its own, before any reset
                    if ((marks & ((1u << j) - 1)) == 0) R = f2_fma(P, widen(dyr[j]), R);
                }
            }
        };
        if (fast) gates(std::true_type{});
        else gates(std::false_type{});
        s.maps[warp][lane] = as_map(P, H);
        float2 Rw;
        f2_unpack(R, Rw.x, Rw.y);
        s.right[warp][lane] = Rw;
        bar_arrive(kMapsReady);
        Tile tn = t;
        if (next < tiles) {
            tn = tile_of<true>(a, next);
            In::request(staged, a, tn, src);
            mark = reset_byte(a, tn);
        }
        bar_sync(kEntryReady);
        if (s.stop) break;
        const unsigned after = s.ticket[n & 1];
        f2 dl = none;
        auto grads = [&](auto is_fast) {
            constexpr bool kFast = decltype(is_fast)::value;
            f2 E[kRun], G[kRun];
            f2 c = s.grad[warp][lane];
#pragma unroll
            for (int j = kRun - 1; j >= 0; --j) {
                E[j] = j < left ? expm1_neg2<kFast>(f2_mul(k, sr[j])) : none;  // a = 1 + E
                G[j] = f2_add(j < left ? widen(dyr[j]) : none, c);
                c = (marks >> j & 1) ? none : f2_fma(E[j], G[j], G[j]);
            }
            f2 h = s.entry[warp][lane];
#pragma unroll
            for (int j = 0; j < kRun; ++j) {
                const bool cut = marks >> j & 1;
                Gate2 g;
                decay_from2(E[j], g);
                const f2 vx = f2_mul(si[j], xv(j));  // sigmoid(i) x
                const f2 gm = cut ? G[j] : f2_mul(G[j], g.m);
                // s dm/ds = -s a^2 / m: finite where s -> 0
                const f2 sa = f2_mul(f2_mul(k, sr[j]), g.a);
                const f2 e = cut ? none
                                 : f2_mul(f2_mul(G[j], sa),
                                          f2_fma(f2_neg(f2_mul(g.a, g.rm)), vx, h));
                if (j < left) {
                    dl = f2_add(dl, e);
                    const int64_t row = t.row0 + (tok0 + j) * a.D;
                    store_pair<T, VEC>(a.dx, row, a, t.d0, f2_mul(gm, si[j]));
                    store_pair<T, VEC>(a.dr, row, a, t.d0, f2_fma(f2_neg(e), sr[j], e));
                    const f2 gv = f2_mul(gm, vx);
                    store_pair<T, VEC>(a.di, row, a, t.d0, f2_fma(f2_neg(gv), si[j], gv));
                }
                h = cut ? vx : f2_fma(g.a, h, f2_mul(g.m, vx));
            }
        };
        if (fast) grads(std::true_type{});
        else grads(std::false_type{});
        float2 dw;
        f2_unpack(dl, dw.x, dw.y);
        s.dlam[n & 1][warp][channel<VEC>(0)] = dw.x;
        s.dlam[n & 1][warp][channel<VEC>(1)] = dw.y;
        if (next >= tiles) {
            bar_arrive(kMapsReady);  // the chain warp takes the last tile's dlam
            break;
        }
        t = tn;
        next = after;
    }
    In::wait();
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
    const Gate g = gate(to_f(r[at]), to_f(i[at]), -c * softplus_full(lam[at % D]));
    const float v = fmaf(g.a, h[at], g.m * g.si * to_f(x[at]));
    h[at] = v;
    y[at] = from_f<T>(v);
}

// ------------------------------------------------------------ host

// Thread blocks of a persistent kernel: as many as fit, fewer where there are
// fewer tiles; without a chain one per tile.
template <typename F>
cudaError_t start(const char *name, F *kernel, size_t smem, const GatedArgs &a, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    int per_sm = 1, dev = 0, sms = 0;
    const int64_t tiles = a.batch * a.dblocks * a.nb;
    int64_t grid = tiles;
    if (e == cudaSuccess && a.nb > 1) {
        if ((e = cudaGetDevice(&dev)) == cudaSuccess &&
            (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) == cudaSuccess)
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kThreads, smem);
        if (e == cudaSuccess && (int64_t)per_sm * sms < grid) grid = (int64_t)per_sm * sms;
        if (e == cudaSuccess) e = cudaMemsetAsync(a.counter, 0, 256, st);
        if (e == cudaSuccess) e = cudaMemsetAsync(a.ends, 0xff, (size_t)tiles * 32 * 24, st);
    }
    if (e != cudaSuccess) return e;
    launch_begin(name, st);
    kernel<<<(unsigned)grid, kThreads, smem, st>>>(a);
    launch_end(st);
    return cudaGetLastError();
}

bool even(const void *p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

template <typename T, bool VEC>
cudaError_t forward_t(const GatedArgs &a, cudaStream_t st) {
    const size_t smem = Stage<T, VEC, 3>::kBytes;
    return a.q ? start("gated_forward", gated_forward_kernel<T, VEC, true>, smem, a, st)
               : start("gated_forward", gated_forward_kernel<T, VEC, false>, smem, a, st);
}
template <typename T>
cudaError_t forward_v(const GatedArgs &a, cudaStream_t st) {
    const size_t two = 2 * sizeof(T);
    const bool vec = a.D % 2 == 0 && even(a.x, two) && even(a.r, two) && even(a.i, two) &&
                     even(a.y, two) && even(a.q, 2);
    return vec ? forward_t<T, true>(a, st) : forward_t<T, false>(a, st);
}

template <typename T, bool VEC>
cudaError_t backward_t(const GatedArgs &a, cudaStream_t st) {
    return a.q ? start("gated_backward", gated_backward_kernel<T, VEC, true>,
                       Stage<T, VEC, 1>::kBytes, a, st)
               : start("gated_backward", gated_backward_kernel<T, VEC, false>,
                       Stage<T, VEC, 4>::kBytes, a, st);
}
template <typename T>
cudaError_t backward_v(const GatedArgs &a, float *dlam, cudaStream_t st) {
    const size_t two = 2 * sizeof(T);
    const bool vec = a.D % 2 == 0 && even(a.x, two) && even(a.r, two) && even(a.i, two) &&
                     even(a.dy, two) && even(a.dx, two) && even(a.dr, two) && even(a.di, two) &&
                     even(a.q, 2);
    cudaError_t e = vec ? backward_t<T, true>(a, st) : backward_t<T, false>(a, st);
    if (e != cudaSuccess) return e;
    launch_begin("gated_dlam", st);
    gated_dlam_kernel<<<(unsigned)((a.D + 31) / 32), dim3(32, 8), 0, st>>>(
        a.dlam_part, a.lam, dlam, a.batch * a.nb, a.D);
    launch_end(st);
    return cudaGetLastError();
}

// The workspace: the tile counter and the abort word, the tiles' ends and
// maps, and in the backward pass the blocks' sums of dlam.
size_t carve(const Problem &pr, GatedArgs &a, void *ws, bool back) {
    a.batch = pr.batch;
    a.L = pr.seqlen;
    a.D = pr.nheads;
    a.nb = gated_blocks(pr);
    a.dblocks = (a.D + kTileCh - 1) / kTileCh;
    const size_t tiles = (size_t)(a.batch * a.dblocks * a.nb);
    char *p = static_cast<char *>(ws);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char *here = p + at;
        at += align256(bytes);
        return here;
    };
    if (a.nb > 1) {
        a.counter = reinterpret_cast<unsigned *>(take(256));
        a.abort = a.counter + 32;
        a.ends = reinterpret_cast<unsigned long long *>(take(tiles * 32 * 8));
        a.maps = reinterpret_cast<unsigned long long *>(take(tiles * 32 * 16));
    }
    if (back)
        a.dlam_part = reinterpret_cast<float *>(take((size_t)(a.batch * a.nb * a.D) * sizeof(float)));
    return at;
}

}  // namespace

int64_t gated_blocks(const Problem &pr) { return (pr.seqlen + kBlock - 1) / kBlock; }

size_t gated_workspace_bytes(const Problem &pr, bool back) {
    GatedArgs a;
    return carve(pr, a, nullptr, back);
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
        a.first = h0;
        a.last = h_final;
        a.err = device_error_word();
        a.wait = wait_limit_cycles();
        if (!a.err) return fail(SSD_ERR_CUDA, "cannot locate the device error word");
        e = pr.dtype == SSD_F32 ? forward_v<float>(a, st) : forward_v<__nv_bfloat16>(a, st);
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
        a.first = dh_final;
        a.last = dh0;
        a.err = device_error_word();
        a.wait = wait_limit_cycles();
        if (!a.err) return fail(SSD_ERR_CUDA, "cannot locate the device error word");
        e = pr.dtype == SSD_F32 ? backward_v<float>(a, dlam, st)
                                : backward_v<__nv_bfloat16>(a, dlam, st);
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
