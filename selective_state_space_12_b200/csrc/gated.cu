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
// Tiles are handed out by a counter, all channels of a block of tokens before
// the next block, so that whoever holds a tile knows that the tiles before it
// are done or held by a running thread block; a ninth warp folds the maps of a
// tile's eight runs and finds what enters the tile. There are two ways, by the
// number of lanes (batch times tiles of channels), each with one fixed order of
// sums:
//
//  - many lanes (one for every other SM or more): a tile waits for what leaves the
//    tile before, which was handed out a round of the lanes earlier. Thread blocks
//    hold a ticket ahead, so that the next tile's inputs arrive meanwhile.
//  - few lanes: thread blocks work on many consecutive tiles of a lane at once,
//    and a chain of waits from tile to tile would be the whole time (1 us a step).
//    Tiles form groups of four or eight (start()); each publishes its (P, H), folds those
//    before it in its group, and waits only for what leaves the group before, so
//    the chain has one step a group. A ticket held ahead would block the chain
//    behind its holder's wait (backward at 32 lanes 698 us for 578), so none is:
//    the inputs that the next round of tiles needs are brought to L2 instead.
//
// What bounds it: bytes (8 forward and 14 backward a token and channel in bf16, 0.67
// and 1.17 GB at b8 L2048 D5120) and, nearly as much, issue: about 80 instructions a
// pair of channels forward and 140 backward, at 45 to 60 % of the issue slots with 18
// to 36 warps an SM. Measured there, B200, bf16: forward 141 us (4.8 TB/s), backward
// 282 us (4.2 TB/s), forward with 8-bit copies 230 us and backward from them 334 us.
// One row of 65536 tokens by 2048 channels, few lanes: 364 and 565 us. Rows that
// start anywhere (D5121): 179 and 371 us.
//
// A published word is 64 bits, cleared to all ones before the kernel, and is
// complete once it differs from that: readers poll the data itself, and no
// fence stands between data and flag. Waits are bounded; one that runs out
// tells the others and all return.
#include <cudaTypedefs.h>

#include <atomic>
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
constexpr int kStepThreads = 128;

// Barriers of the compute warps and the chain warp.
enum { kMapsReady = 1, kEntryReady = 2, kTicketReady = 3 };
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

// Where a lane's two words of tile `id`'s map are: past 2^32 from 2^26 tiles on (5 rows
// of 2^30 tokens).
constexpr int64_t map_word(int64_t id, int lane) { return (id * 32 + lane) * 2; }
static_assert(map_word(1u << 26, 3) == (int64_t{1} << 32) + 6, "in 64 bits");

struct __align__(16) Tile {
    int64_t row0;     // offset of (b, first token, 0) in a (b, L, D) tensor
    int64_t flat;     // its first token's row in a (b L, D) tensor
    int64_t blocks0;  // and of (b, blk, 0) in a (b, nb, D) one
    int b, blk, d0, n;  // batch, block of tokens, first channel, tokens
    unsigned id;      // its ticket, and the index of its record
};
template <bool BACK>
__device__ __forceinline__ Tile tile_of(const GatedArgs &a, unsigned ticket) {
    Tile t;
    const unsigned lanes = (unsigned)(a.batch * a.dblocks);
    const unsigned step = ticket / lanes, lane = ticket % lanes;
    t.b = (int)(lane / (unsigned)a.dblocks);
    t.d0 = (int)(lane % (unsigned)a.dblocks) * kTileCh;
    t.blk = (int)(BACK ? a.nb - 1 - step : step);
    t.flat = t.b * a.L + (int64_t)t.blk * kBlock;
    t.row0 = t.flat * a.D;
    t.blocks0 = (t.b * a.nb + t.blk) * a.D;
    const int64_t left = a.L - (int64_t)t.blk * kBlock;
    t.n = (int)(left < kBlock ? left : kBlock);
    t.id = ticket;
    return t;
}

// ------------------------------------------------------------ two channels

// A lane's two channels: adjacent where rows are 16-byte aligned (ALIGNED: one
// load of shared memory, one store of global memory), else 32 apart (two, which
// neighbouring lanes continue).
template <bool ALIGNED>
__device__ __forceinline__ int channel(int j) {
    const int lane = threadIdx.x & 31;
    return ALIGNED ? 2 * lane + j : lane + 32 * j;
}

template <typename T>
struct Pair;  // two elements as stored
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
template <>
struct Pair<int8_t> {
    using type = uint16_t;
};
// int8 -> float without the (special-function unit's) conversion: the byte
// plus 128 in the low bits of 2^23.
__device__ __forceinline__ f2 widen(uint16_t v) {
    const uint32_t u = v ^ 0x8080u;
    return f2_sub(f2_pack(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440)),
                          __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7441))),
                  f2_both(8388736.f));
}

// An output's rows for this lane: stores its two channels of one token after
// the other. FULL: the tile's channels are all there.
template <typename T, bool ALIGNED>
struct Rows {
    T *p;
    int64_t step;
    bool has0, has1;
    __device__ __forceinline__ Rows(void *base, int64_t row, int d0, int64_t D)
        : p(static_cast<T *>(base) + row + d0 + channel<ALIGNED>(0)),
          step(D),
          has0(d0 + channel<ALIGNED>(0) < D),
          has1(d0 + channel<ALIGNED>(1) < D) {}
    template <bool FULL>
    __device__ __forceinline__ void put(f2 val) {
        float lo, hi;
        f2_unpack(val, lo, hi);
        if constexpr (ALIGNED) {
            if (FULL || has0) {
                if constexpr (sizeof(T) == 4)
                    *reinterpret_cast<float2 *>(p) = make_float2(lo, hi);
                else
                    *reinterpret_cast<uint32_t *>(p) = tc::pack_bf16(lo, hi);
            }
        } else {
            if (FULL || has0) p[0] = from_f<T>(lo);
            if (FULL || has1) p[32] = from_f<T>(hi);
        }
        p += step;
    }
};

// ------------------------------------------------------------ staged inputs

// Rows of a tile come to shared memory by TMA, a tile ahead where tickets are.
// T is the I/O type, or int8 for 8-bit copies.
struct Maps {
    CUtensorMap m[4];
};
// A wait for copies in flight before a thread block ends (about 9 ms), whatever
// the limit on the waits before it.
constexpr long long kDrain = 1ll << 24;

// Rows that start on 16 bytes: each warp brings its own eight tokens' rows, one
// TMA load a tensor, counted by a barrier of its own, and waits for nobody
// else's; past the last token and channel the load fills zeros.
template <typename T, int TENSORS, int KEEP = 0>
struct WarpRows {
    using P = typename Pair<T>::type;
    static constexpr bool kAhead = true;  // may be requested before other warps have read theirs
    static constexpr int kPitch = kTileCh * (int)sizeof(T);
    static constexpr int kRowsBytes = TENSORS * kRun * kPitch;
    static constexpr int kWarpBytes = kRowsBytes > KEEP ? kRowsBytes : KEEP;
    static constexpr size_t kBytes = (size_t)kWarps * kWarpBytes;

    unsigned char *buf;  // this warp's rows
    uint64_t *bar;
    uint32_t parity;

    __device__ __forceinline__ WarpRows(unsigned char *all, uint64_t *bars)
        : buf(all + (threadIdx.x >> 5) * kWarpBytes), bar(bars + (threadIdx.x >> 5)), parity(0) {}

    __device__ __forceinline__ void request(const GatedArgs &a, const CUtensorMap *maps,
                                            const Tile &t, const void *const (&)[TENSORS]) {
        const int tok0 = (threadIdx.x >> 5) * kRun;
        __syncwarp();  // the rows have been read
        if (KEEP > 0) {  // what was kept there was written by ordinary stores
            tc::fence_proxy_async_smem();
            __syncwarp();
        }
        if ((threadIdx.x & 31) == 0) {
            const bool any = tok0 < t.n;
            tc::mbar_arrive_expect_tx(bar, any ? kRowsBytes : 0);
            if (any) {
#pragma unroll
                for (int w = 0; w < TENSORS; ++w)
                    tc::tma_load_4d(buf + w * kRun * kPitch, maps + w, bar, t.d0,
                                    t.blk * kBlock + tok0, t.b, 0);
            }
        }
    }
    // Brings the rows of a tile that another thread block will take to L2.
    __device__ __forceinline__ void prefetch(const GatedArgs &a, const CUtensorMap *maps,
                                             unsigned tiles, const Tile &t,
                                             const void *const (&)[TENSORS]) const {
        const int tok0 = (threadIdx.x >> 5) * kRun;
        if (t.id < tiles && (threadIdx.x & 31) == 0 && tok0 < t.n) {
#pragma unroll
            for (int w = 0; w < TENSORS; ++w)
                tc::tma_prefetch_l2_4d(maps + w, t.d0, t.blk * kBlock + tok0, t.b, 0);
        }
    }
    // False when the wait ran out.
    __device__ __forceinline__ bool wait(long long limit) {
        const bool ok = __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, limit));
        if (ok) parity ^= 1;
        return ok;
    }
    __device__ __forceinline__ P get(int w, int j) const {
        return reinterpret_cast<const P *>(buf + (w * kRun + j) * kPitch)[threadIdx.x & 31];
    }
};

// Rows that start anywhere. kSlots consecutive rows of a (b L, D) tensor make one
// of 16 k bytes, so the tensor is mapped as (b L / kSlots, kSlots D): a box of
// this map holds every kSlots-th row of a tile, all at the same place within 16
// bytes, from which it starts (up to 15 bytes before the row). Eight warps bring
// the boxes, one or two each a tensor, once all have read the rows before, and
// wait for all of them. Lanes read from the rows' places in their boxes. A tile
// with rows past the map's whole ones (at the tensor's end), or tensors that do
// not start on 16 bytes, are read by plain loads. STACKED: the tensors lie behind
// one another and share one map.
template <typename T, int TENSORS, bool STACKED = false>
struct FlatRows {
    using P = typename Pair<T>::type;
    static constexpr bool kAhead = false;
    static constexpr int kE = (int)sizeof(T), kUnit = 16 / kE;
    static constexpr int kSlots = kE == 1 ? 16 : 8, kSlotRows = kBlock / kSlots;
    static constexpr int kPitch = kTileCh * kE + 16;
    static constexpr int kSlotBytes = (kSlotRows * kPitch + 127) & ~127;
    static constexpr size_t kBytes = (size_t)TENSORS * kSlots * kSlotBytes;

    unsigned char *buf;  // all rows
    uint64_t *bar;
    uint32_t parity;
    uint32_t first, low;  // the tile's first row and D, modulo the slots and the unit
    uint32_t behind;      // STACKED: rows of a tensor, modulo the slots
    bool plain;

    __device__ __forceinline__ FlatRows(unsigned char *all, uint64_t *bars)
        : buf(all), bar(bars), parity(0) {}

    // token j of this warp: its box and its row there
    static __device__ __forceinline__ int slot(int j) {
        return kE == 1 ? ((threadIdx.x >> 5) & 1) * kRun + j : j;
    }
    static __device__ __forceinline__ int row() {
        return kE == 1 ? threadIdx.x >> 6 : threadIdx.x >> 5;
    }
    __device__ __forceinline__ T *place(int w, int j) const {
        const uint32_t r = first + slot(j) + (STACKED ? w * behind : 0);
        const uint32_t shift = ((r & (kSlots - 1)) * low) & (kUnit - 1);
        return reinterpret_cast<T *>(buf + (w * kSlots + slot(j)) * kSlotBytes + row() * kPitch) +
               shift + (threadIdx.x & 31);
    }
    __device__ __forceinline__ void request(const GatedArgs &a, const CUtensorMap *maps,
                                            const Tile &t, const void *const (&src)[TENSORS]) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        first = (uint32_t)t.flat & (kSlots - 1);
        low = (uint32_t)a.D & (kUnit - 1);
        const int64_t rows = a.batch * a.L, before = STACKED ? (TENSORS - 1) * rows : 0;
        behind = (uint32_t)rows & (kSlots - 1);
        plain = !a.flat || before + t.flat + t.n > (before + rows & ~(int64_t)(kSlots - 1));
        if (plain) {
            const int tok0 = warp * kRun;
            const bool has0 = t.d0 + lane < a.D, has1 = t.d0 + lane + 32 < a.D;
#pragma unroll
            for (int w = 0; w < TENSORS; ++w)
#pragma unroll
                for (int j = 0; j < kRun; ++j) {
                    if (tok0 + j >= t.n) break;
                    const T *from = static_cast<const T *>(src[w]) + t.row0 + (tok0 + j) * a.D +
                                    t.d0 + lane;
                    T *to = place(w, j);
                    if (has0) to[0] = from[0];
                    if (has1) to[32] = from[32];
                }
        } else if (lane == 0) {
            // ordinary writes of a plain tile before these
            tc::fence_proxy_async_smem();
            constexpr int kMine = kSlots / kWarps;
            tc::mbar_arrive_expect_tx(bar, kMine * TENSORS * kSlotRows * kPitch);
#pragma unroll
            for (int i = 0; i < kMine; ++i)
#pragma unroll
                for (int w = 0; w < TENSORS; ++w) {
                    const int64_t r = t.flat + warp * kMine + i + (STACKED ? w * rows : 0);
                    const int x = (int)((int)(r & (kSlots - 1)) * a.D + t.d0) & ~(kUnit - 1);
                    tc::tma_load_4d(buf + (w * kSlots + warp * kMine + i) * kSlotBytes,
                                    maps + (STACKED ? 0 : w), bar, x, (int)(r / kSlots), 0, 0);
                }
        }
    }
    __device__ __forceinline__ void prefetch(const GatedArgs &a, const CUtensorMap *, unsigned tiles,
                                             const Tile &t,
                                             const void *const (&src)[TENSORS]) const {
        const int lane = threadIdx.x & 31, tok0 = (threadIdx.x >> 5) * kRun;
        const int w = lane / kRun, j = lane % kRun;
        if (t.id < tiles && w < TENSORS && tok0 + j < t.n) {
            const T *from = nullptr;
#pragma unroll
            for (int v = 0; v < TENSORS; ++v)
                if (v == w) from = static_cast<const T *>(src[v]);
            from += t.row0 + (tok0 + j) * a.D + t.d0;
            const int len = (int)(a.D - t.d0 < kTileCh ? a.D - t.d0 : kTileCh);
            for (int c = 0; c < len; c += 64 / kE)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(from + c));
        }
    }
    __device__ __forceinline__ bool wait(long long limit) {
        if (plain) {
            __syncwarp();
            return true;
        }
        const bool ok = __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, limit));
        if (ok) parity ^= 1;
        return ok;
    }
    __device__ __forceinline__ P get(int w, int j) const {
        const T *v = place(w, j);
        if constexpr (kE == 4)
            return make_float2(v[0], v[32]);
        else if constexpr (kE == 2)
            return (uint32_t)__bfloat16_as_ushort(v[0]) | (uint32_t)__bfloat16_as_ushort(v[32]) << 16;
        else
            return (uint16_t)((uint8_t)v[0] | (uint16_t)(uint8_t)v[32] << 8);
    }
};

template <typename T, bool ALIGNED, int TENSORS, int KEEP = 0>
using Stage = std::conditional_t<ALIGNED, WarpRows<T, TENSORS, KEEP>,
                                 FlatRows<T, TENSORS, std::is_same_v<T, int8_t>>>;

// Reset marks of the warp's tokens, one bit each.
__device__ __forceinline__ unsigned reset_byte(const GatedArgs &a, const Tile &t) {
    const int lane = threadIdx.x & 31, tok = (threadIdx.x >> 5) * kRun + lane;
    if (!a.reset || lane >= kRun || tok >= t.n) return 0;
    return a.reset[(int64_t)t.b * a.L + (int64_t)t.blk * kBlock + tok];
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

// A bounded wait of the chain warp: false once it, or another thread block's,
// has run out.
struct Patience {
    long long began = 0;
    int polls = 0;
    __device__ __forceinline__ bool more(const GatedArgs &a) {
        if (polls == 0) began = clock64();
        bool stop = false;
        if ((threadIdx.x & 31) == 0) {
            stop = clock64() - began > a.wait || ((polls & 15) == 15 && load_relaxed(a.abort) != 0);
            if (stop) {
                atomicExch(a.err, 0x6a7ed001u);
                atomicExch(a.abort, 1u);
            }
        }
        ++polls;
        return !__shfl_sync(0xffffffffu, stop, 0);
    }
};

// The word of each lane once it is there; false when the wait ran out.
__device__ __forceinline__ bool await(const GatedArgs &a, const word *p, word &v) {
    if (__all_sync(0xffffffffu, v != kEmpty)) return true;
    Patience wait;
    while (true) {
        v = load_word(p);
        if (__all_sync(0xffffffffu, v != kEmpty)) return true;
        if (!wait.more(a)) return false;
    }
}

// The composed map of the `count` tiles before tile `id` in its group.
__device__ __forceinline__ bool group_map(const GatedArgs &a, int64_t id, int count, int64_t lanes,
                                          float4 &map) {
    const int lane = threadIdx.x & 31;
    map = make_float4(1.f, 0.f, 1.f, 0.f);
    Patience wait;
    constexpr int kBatch = 4;
    for (int first = 0; first < count; first += kBatch) {
        while (true) {
            word m0[kBatch], m1[kBatch];
            bool there = true;
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const bool has = first + j < count;
                const word *at = &a.maps[map_word(id - (count - first - j) * lanes, lane)];
                m0[j] = has ? load_word(at) : 0;
                m1[j] = has ? load_word(at + 1) : 0;
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j) there = there && m0[j] != kEmpty && m1[j] != kEmpty;
            if (__all_sync(0xffffffffu, there)) {
#pragma unroll
                for (int j = 0; j < kBatch; ++j)
                    if (first + j < count) {
                        float4 m;
                        f2_unpack(m0[j], m.x, m.y);
                        f2_unpack(m1[j], m.z, m.w);
                        map = then(map, m);
                    }
                break;
            }
            if (!wait.more(a)) return false;
        }
    }
    return true;
}

template <bool ALIGNED>
__device__ __forceinline__ f2 read_state(const float *p, int64_t row, int d0, int64_t D) {
    const int c0 = d0 + channel<ALIGNED>(0), c1 = d0 + channel<ALIGNED>(1);
    return f2_pack(p && c0 < D ? p[row + c0] : 0.f, p && c1 < D ? p[row + c1] : 0.f);
}
template <bool ALIGNED>
__device__ __forceinline__ void write_state(float *p, int64_t row, int d0, int64_t D, f2 v) {
    const int c0 = d0 + channel<ALIGNED>(0), c1 = d0 + channel<ALIGNED>(1);
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
    float dlam[2][kWarps][kTileCh];
    uint2 top[3][kWarps][32];  // 8-bit copies: largest magnitudes of each run
    unsigned code[3][kTileCh];
    uint64_t bars[2 * kWarps];
    Tile tile[2];              // this thread block's next tiles
    Tile later[2];             // without tickets ahead: one to bring to L2, by turns: nothing
                               // keeps a warp that reads one from the next being written
    int stop[2];
};

// k = c softplus(lam) of the lane's channels
template <bool ALIGNED>
__device__ __forceinline__ f2 gate_scales(const GatedArgs &a, int d0) {
    return read_state<ALIGNED>(a.scale, 0, d0, a.D);
}
// A wait of a compute warp ran out.
__device__ __forceinline__ void give_up(const GatedArgs &a, int *stop) {
    if ((threadIdx.x & 31) == 0) {
        atomicExch(a.err, 0x6a7ed002u);
        if (a.abort) atomicExch(a.abort, 1u);
        *stop = 1;
    }
}
__device__ __forceinline__ bool all_fast(f2 k) {
    float lo, hi;
    f2_unpack(k, lo, hi);
    return __all_sync(0xffffffffu, lo <= kSeries && hi <= kSeries);
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
// The largest magnitudes of a pair of channels, as bits.
template <typename T>
struct Largest;
template <>
struct Largest<float> {
    uint2 m = {0, 0};
    __device__ __forceinline__ void add(float2 v) {
        m.x = max(m.x, __float_as_uint(v.x) & 0x7fffffffu);
        m.y = max(m.y, __float_as_uint(v.y) & 0x7fffffffu);
    }
    __device__ __forceinline__ void join(const Largest &o) {
        m.x = max(m.x, o.m.x);
        m.y = max(m.y, o.m.y);
    }
    __device__ __forceinline__ uint32_t bits(int j) const { return j ? m.y : m.x; }
};
template <>
struct Largest<__nv_bfloat16> {
    uint32_t m = 0;
    __device__ __forceinline__ void add(uint32_t v) { m = __vmaxu2(m, v & 0x7fff7fffu); }
    __device__ __forceinline__ void join(const Largest &o) { m = __vmaxu2(m, o.m); }
    __device__ __forceinline__ uint32_t bits(int j) const { return j ? m & 0xffff0000u : m << 16; }
};

// Two values as int8 steps, in the low bytes: adding 1.5 2^23 rounds to the
// nearest step, ties to even, and leaves it in the low byte (the copy's one rounding).
__device__ __forceinline__ uint32_t in_steps(f2 v, f2 inv) {
    float lo, hi;
    f2_unpack(f2_fma(v, inv, f2_both(12582912.f)), lo, hi);
    return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x0040);
}

// ------------------------------------------------------------ chain warp

// The ticket one round of thread blocks on (or none).
__device__ __forceinline__ unsigned round_on(unsigned ticket) {
    return ticket + gridDim.x < ticket ? ~0u : ticket + gridDim.x;
}

// The ninth warp: for each tile of this thread block, folds its runs' maps,
// finds what enters it, hands every run what enters that, and publishes what
// leaves. While the others compute a tile it fetches the next ticket and
// prepares the next tile's gate scales.
template <typename T, bool ALIGNED, bool CK, bool BACK, bool EAGER>
__device__ __forceinline__ void chain_warp(const GatedArgs &a, Shared &s, unsigned tiles,
                                           int64_t lanes) {
    const int lane = threadIdx.x & 31;
    const bool chained = a.nb > 1;
    unsigned now = s.tile[0].id, next = s.tile[1].id;
    int64_t last_row = -1;  // dlam of the tile before: its row and channels
    int last_d0 = 0;
    auto flush = [&](int slot) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int c = channel<ALIGNED>(j);
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
        if (EAGER && next < tiles) {
            if (lane == 0) after = atomicAdd(a.counter, 1u);
            after = __shfl_sync(0xffffffffu, after, 0);
        }
        const int last_pos = (1 << a.group_bits) - 1, pos = (int)step & last_pos;
        const bool leaves = EAGER || pos == last_pos;  // publishes what leaves it
        const bool waits = EAGER ? step > 0 : (int)step > last_pos;
        const int64_t slot =
            EAGER ? t.id : (int64_t)(step >> a.group_bits) * lanes + t.id % (unsigned)lanes;
        f2 in = 0, h = 0;
        word before = kEmpty;
        if (waits) before = load_word(&a.ends[(slot - lanes) * 32 + lane]);
        else in = read_state<ALIGNED>(a.first, (int64_t)t.b * a.D, t.d0, a.D);
        if (BACK) h = read_state<ALIGNED>(a.states, t.blocks0, t.d0, a.D);
        bar_sync(kMapsReady);
        if (s.stop[n & 1]) {
            bar_arrive(kEntryReady);
            return;
        }
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
        bool ok = true;
        if (chained && !EAGER) {
            if (pos < last_pos && step + 1 < a.nb) {
                // who has read the maps may write a.last, which may be a.first: our read is done
                if (!waits) __threadfence();
                word *mine = &a.maps[map_word(t.id, lane)];
                store_word(mine, all.x, all.y);
                store_word(mine + 1, all.z, all.w);
            }
            float4 ahead;
            ok = group_map(a, t.id, pos, lanes, ahead);
            if (ok && waits) ok = await(a, &a.ends[(slot - lanes) * 32 + lane], before);
            in = apply(ahead, waits ? before : in);
        } else if (waits) {
            ok = await(a, &a.ends[(slot - lanes) * 32 + lane], before);
            in = before;
        }
        if (!ok) {
            if (lane == 0) s.stop[n & 1] = 1;
            __syncwarp();
            bar_arrive(kEntryReady);
            return;
        }
        const f2 out = apply(all, in);
        if (chained && leaves && step + 1 < a.nb) {
            float2 e;
            f2_unpack(out, e.x, e.y);
            store_word(&a.ends[slot * 32 + lane], e.x, e.y);
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
            for (int w = 0; w < 3; ++w) {
                Largest<T> top;
#pragma unroll
                for (int j = 0; j < kWarps; ++j)
                    top.join(reinterpret_cast<const Largest<T> *>(s.top[w][j])[lane]);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int c = channel<ALIGNED>(j);
                    const uint32_t code = step_code(top.bits(j));
                    s.code[w][c] = code;
                    if (t.d0 + c < a.D)
                        a.e[w * a.batch * a.nb * a.D + t.blocks0 + t.d0 + c] = (uint8_t)code;
                }
            }
        }
        if (EAGER && lane == 0) s.tile[n & 1] = tile_of<BACK>(a, after);
        __syncwarp();
        bar_arrive(kEntryReady);
        if (chained && !EAGER) {
            if (lane == 0) next = atomicAdd(a.counter, 1u);
            next = __shfl_sync(0xffffffffu, next, 0);
            if (lane < 2)
                (lane ? s.later[(n + 1) & 1] : s.tile[0]) =
                    tile_of<BACK>(a, lane ? round_on(next) : next);
            __syncwarp();
            bar_arrive(kTicketReady);
        }
        if (!BACK && a.states)
            write_state<ALIGNED>(a.states, t.blocks0, t.d0, a.D, in);
        if (a.last && step + 1 == a.nb) write_state<ALIGNED>(a.last, (int64_t)t.b * a.D, t.d0, a.D, out);
        last_row = t.blocks0;
        last_d0 = t.d0;
        now = next;
        next = after;
        if (BACK && now >= tiles) {
            bar_sync(kMapsReady);
            flush(n & 1);
        }
    }
}

// The first tickets of this thread block, and its barriers.
template <bool ALIGNED, bool BACK, bool EAGER>
__device__ __forceinline__ void open_block(const GatedArgs &a, Shared &s, unsigned tiles) {
    after_previous();
    if (BACK) let_next();
    if (threadIdx.x == 0) {
        s.stop[0] = s.stop[1] = 0;
        // one block of tokens: a tile a thread block
        const unsigned first = a.nb > 1 ? atomicAdd(a.counter, 1u) : blockIdx.x;
        s.tile[0] = tile_of<BACK>(a, first);
        s.tile[1] = tile_of<BACK>(a, EAGER ? atomicAdd(a.counter, 1u) : tiles);
        s.later[0] = tile_of<BACK>(a, round_on(first));
        // a barrier a warp and stage, or one a stage that every warp arrives at
        for (int w = 0; w < 2 * kWarps; ++w) tc::mbar_init(&s.bars[w], ALIGNED ? 1 : kWarps);
        tc::fence_mbar_init();
    }
    __syncthreads();
}

// The plain case of a warp's eight tokens (all there, with all the tile's
// channels, no reset, slow decays, and with a shared reciprocal no gate all but
// shut) is straight code; every other case runs a general copy with a branch a
// token.
struct PlainRun : std::true_type {};
struct AnyRun : std::false_type {};

// ------------------------------------------------------------ forward

// Bytes that a warp keeps in its rows' place while it waits: a and u. Few lanes wait
// longest, and need no room for rows ahead: four thread blocks an SM fit for three (b1
// L65536 D2048 366 us for 388 without).
template <bool ALIGNED, bool CK, bool EAGER>
constexpr int kForwardKeep = ALIGNED && !EAGER && !CK ? 2 * kRun * 32 * 8 : 0;

// x, r, i (and with CK their 8-bit copies, from the values as stored) to y, the end
// state and the states that enter the blocks.
template <typename T, bool ALIGNED, bool CK, bool EAGER>
__global__ void
__launch_bounds__(kThreads, CK ? 2 : kForwardKeep<ALIGNED, CK, EAGER> ? 4 : 3) gated_forward_kernel(
    const GatedArgs a, const __grid_constant__ Maps maps) {
    extern __shared__ __align__(128) unsigned char staged[];
    __shared__ Shared s;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t lanes = a.batch * a.dblocks;
    const unsigned tiles = (unsigned)(lanes * a.nb);
    open_block<ALIGNED, false, EAGER>(a, s, tiles);
    if (warp == kWarps) {
        chain_warp<T, ALIGNED, CK, false, EAGER>(a, s, tiles, lanes);
        return;
    }
    Stage<T, ALIGNED, 3, kForwardKeep<ALIGNED, CK, EAGER>> in(staged, s.bars);
    const void *const src[3] = {a.x, a.r, a.i};
    Tile t = s.tile[0];
    if (t.id >= tiles) return;
    in.request(a, maps.m, t, src);
    unsigned mark = reset_byte(a, t);
    f2 k = gate_scales<ALIGNED>(a, t.d0);
    const int tok0 = warp * kRun;
    const bool chained = a.nb > 1;
    constexpr bool kAhead = decltype(in)::kAhead;
    // one reciprocal for both gates, and the plain case done again where that is not right:
    // b8 L2048 D5120 138 us for 147. Rows that start anywhere take 181 us with it and 177
    // without, few lanes 379 for 366 (b1 L65536 D2048), and the backward kernel, whose
    // registers it costs, 286 for 285. With copies 228 us for 225, but the outputs are to be
    // those without copies to the bit.
    constexpr bool kShared = ALIGNED && EAGER;
    bool ahead = false;  // copies are on their way
    for (int n = 0;; ++n) {
        const unsigned marks = __ballot_sync(0xffffffffu, mark != 0);
        const int left = t.n - tok0;
        bool plain = all_fast(k) && marks == 0 && left >= kRun && t.d0 + kTileCh <= a.D;
        const bool here = in.wait(a.wait);
        if (!here) give_up(a, &s.stop[n & 1]);
        typename Pair<T>::type v[3][kRun];
        f2 av[kRun], u[kRun];
        f2 P, H, top = f2_both(0.f);
        auto gates = [&](auto run) {
            constexpr bool kPlain = decltype(run)::value;
            P = f2_both(1.f);
            H = f2_both(0.f);
#pragma unroll
            for (int j = 0; j < kRun; ++j) {
#pragma unroll
                for (int w = 0; w < 3; ++w) v[w][j] = in.get(w, j);
                const Gate2 g =
                    gate2<kPlain, kPlain && kShared>(widen(v[1][j]), widen(v[2][j]), k, top);
                const f2 ix = f2_mul(g.si, widen(v[0][j]));
                if (kPlain || (j < left && !(marks >> j & 1))) {
                    av[j] = g.a;
                    u[j] = f2_mul(g.m, ix);
                    H = j == 0 ? u[j] : f2_fma(g.a, H, u[j]);
                    P = j == 0 ? g.a : f2_mul(P, g.a);
                } else if (j < left) {
                    av[j] = P = f2_both(reset_decay());
                    H = u[j] = ix;
                } else {
                    av[j] = f2_both(1.f);
                    u[j] = f2_both(0.f);
#pragma unroll
                    for (int w = 0; w < 3; ++w) v[w][j] = {};
                }
            }
        };
        if (plain) {
            gates(PlainRun());
            if (kShared) plain = gates_open(top);
        }
        if (!plain) gates(AnyRun());
        if (CK) {
#pragma unroll
            for (int w = 0; w < 3; ++w) {
                Largest<T> top;
#pragma unroll
                for (int j = 0; j < kRun; ++j) top.add(v[w][j]);
                reinterpret_cast<Largest<T> *>(s.top[w][warp])[lane] = top;
            }
        }
        s.maps[warp][lane] = as_map(P, H);
        // without a ticket ahead the rows' place is free: a and u wait there, so that more
        // thread blocks fit
        f2 *const keep = reinterpret_cast<f2 *>(in.buf) + lane;
        constexpr bool kKeep = kForwardKeep<ALIGNED, CK, EAGER> > 0;
        if (kKeep) {
            __syncwarp();
#pragma unroll
            for (int j = 0; j < kRun; ++j) {
                keep[2 * j * 32] = av[j];
                keep[(2 * j + 1) * 32] = u[j];
            }
        }
        bar_arrive(kMapsReady);
        Tile tn;
        f2 kn = k;
        auto advance = [&] {  // the next tile's inputs are on their way while this one waits
            in.request(a, maps.m, tn, src);
            mark = reset_byte(a, tn);
            kn = gate_scales<ALIGNED>(a, tn.d0);
        };
        ahead = false;
        if (EAGER) {
            tn = s.tile[(n + 1) & 1];
            ahead = here && tn.id < tiles;
            if (ahead && kAhead) advance();
        } else if (chained) in.prefetch(a, maps.m, tiles, s.later[n & 1], src);
        bar_sync(kEntryReady);
        if (s.stop[n & 1]) {
            if (!here) in.wait(kDrain);
            ahead = ahead && kAhead;
            break;
        }
        if (EAGER && !kAhead && ahead) advance();  // all warps have read their rows
        f2 h = s.entry[warp][lane];
        Rows<T, ALIGNED> y(a.y, t.row0 + tok0 * a.D, t.d0, a.D);
        if (plain) {
#pragma unroll
            for (int j = 0; j < kRun; ++j) {
                h = f2_fma(kKeep ? keep[2 * j * 32] : av[j], h, kKeep ? keep[(2 * j + 1) * 32] : u[j]);
                y.template put<true>(h);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kRun; ++j) {
                const f2 uj = kKeep ? keep[(2 * j + 1) * 32] : u[j];
                h = (marks >> j & 1) ? uj : f2_fma(kKeep ? keep[2 * j * 32] : av[j], h, uj);
                if (j < left) y.template put<false>(h);
            }
        }
        if (CK) {
            const int c0 = channel<ALIGNED>(0), c1 = channel<ALIGNED>(1);
            auto copy = [&](auto run) {
                constexpr bool kPlain = decltype(run)::value;
#pragma unroll
                for (int w = 0; w < 3; ++w) {
                    const uint32_t k0 = s.code[w][c0], k1 = s.code[w][c1];
                    const f2 inv = f2_pack(!kPlain && k0 == 255 ? 0.f : __uint_as_float((254u - k0) << 23),
                                           !kPlain && k1 == 255 ? 0.f : __uint_as_float((254u - k1) << 23));
                    int8_t *q = a.q + w * a.batch * a.L * a.D + t.row0 + tok0 * a.D + t.d0 + c0;
#pragma unroll
                    for (int j = 0; j < kRun; ++j, q += a.D) {
                        if (!kPlain && j >= left) break;
                        uint32_t both = in_steps(widen(v[w][j]), inv);
                        if (!kPlain) both &= (k0 == 255 ? 0u : 0xffu) | (k1 == 255 ? 0u : 0xff00u);
                        if (kPlain && ALIGNED) {
                            *reinterpret_cast<uint16_t *>(q) = (uint16_t)both;
                        } else {
                            if (kPlain || y.has0) q[0] = (int8_t)(both & 0xff);
                            if (kPlain || y.has1) q[c1 - c0] = (int8_t)(both >> 8);
                        }
                    }
                }
            };
            bool number = true;  // no infinity or NaN in this lane's blocks
#pragma unroll
            for (int w = 0; w < 3; ++w) number = number && s.code[w][c0] != 255 && s.code[w][c1] != 255;
            if (__all_sync(0xffffffffu, number) && left >= kRun && t.d0 + kTileCh <= a.D) copy(PlainRun());
            else copy(AnyRun());
        }
        if (chained && !EAGER) {
            bar_sync(kTicketReady);
            tn = s.tile[0];
            ahead = tn.id < tiles;
            if (ahead) advance();
        }
        if (!ahead) break;
        t = tn;
        k = kn;
    }
    if (ahead) in.wait(kDrain);  // nothing may be in flight to shared memory at the end
}

// ------------------------------------------------------------ backward

// The steps of an 8-bit copy's block.
template <bool ALIGNED>
__device__ __forceinline__ f2 copy_step(const GatedArgs &a, const Tile &t, int w) {
    const uint8_t *e = a.e + w * a.batch * a.nb * a.D + t.blocks0 + t.d0;
    const int c0 = channel<ALIGNED>(0), c1 = channel<ALIGNED>(1);
    return f2_pack(t.d0 + c0 < a.D ? __uint_as_float((uint32_t)e[c0] << 23) : 0.f,
                   t.d0 + c1 < a.D ? __uint_as_float((uint32_t)e[c1] << 23) : 0.f);
}

// Bytes of shared memory in which sigmoid(i) waits for the gradients. Spilled registers
// would wait in L2, which these kernels load most: at b8 L2048, D5121 380 us for 459
// and from copies (D5120) 333 for 415; plain rows, where fewer registers are
// spilled, took 284 us with it and 271 without.
template <bool ALIGNED, bool CK>
constexpr int kBackwardKeep = ALIGNED && !CK ? 0 : kRun * kCompute * 8;

// dy, r, i, x (CK: the copies) and the blocks' states to dx, dr, di, dh0 and each
// block's sums of dlam. The gates are computed once: two sigmoids, dy and x stay in
// registers between the maps and the gradients (96 registers, two thread blocks an
// SM; three, with all of it in shared memory, was slower).
template <typename T, bool ALIGNED, bool CK, bool EAGER>
__global__ void __launch_bounds__(kThreads, 2) gated_backward_kernel(
    const GatedArgs a, const __grid_constant__ Maps maps) {
    extern __shared__ __align__(128) unsigned char staged[];
    __shared__ Shared s;
    constexpr int kIn = CK ? 1 : 4;
    using P2 = typename Pair<T>::type;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t lanes = a.batch * a.dblocks;
    const unsigned tiles = (unsigned)(lanes * a.nb);
    open_block<ALIGNED, true, EAGER>(a, s, tiles);
    if (warp == kWarps) {
        chain_warp<T, ALIGNED, CK, true, EAGER>(a, s, tiles, lanes);
        return;
    }
    using In = Stage<T, ALIGNED, kIn>;
    using Copies = Stage<int8_t, ALIGNED, 3>;
    In in(staged, s.bars);
    Copies copies(staged + In::kBytes, s.bars + kWarps);  // used with CK
    const void *src[kIn];
    const void *const csrc[3] = {a.q, a.q + a.batch * a.L * a.D, a.q + 2 * a.batch * a.L * a.D};
    src[0] = a.dy;
    if constexpr (!CK) {
        src[1] = a.r;
        src[2] = a.i;
        src[3] = a.x;
    }
    Tile t = s.tile[0];
    if (t.id >= tiles) return;
    in.request(a, maps.m, t, src);
    f2 steps[3], steps_next[3];
    if constexpr (CK) {
        copies.request(a, maps.m + 1, t, csrc);
#pragma unroll
        for (int w = 0; w < 3; ++w) steps[w] = copy_step<ALIGNED>(a, t, w);
    }
    unsigned mark = reset_byte(a, t);
    f2 k = gate_scales<ALIGNED>(a, t.d0);
    const int tok0 = warp * kRun;
    const f2 none = f2_both(0.f), one = f2_both(1.f);
    constexpr bool kKeep = kBackwardKeep<ALIGNED, CK> > 0;
    f2 *const kept = reinterpret_cast<f2 *>(staged + In::kBytes + (CK ? Copies::kBytes : 0)) +
                     warp * kRun * 32 + lane;
    const bool chained = a.nb > 1;
    constexpr bool kAhead = In::kAhead;
    bool ahead = false;
    for (int n = 0;; ++n) {
        const unsigned marks = __ballot_sync(0xffffffffu, mark != 0);
        const int left = t.n - tok0;
        const bool plain = all_fast(k) && marks == 0 && left >= kRun && t.d0 + kTileCh <= a.D;
        // kept until the gradients: dy, x (as stored) and the two sigmoids, some in shared memory
        std::conditional_t<CK, uint16_t, P2> xr[kRun];
        P2 dyr[kRun];
        f2 sr[kRun], si[kRun];
        auto sigmoid_i = [&](int j) -> f2 & { return kKeep ? kept[j * 32] : si[j]; };
        bool here = in.wait(a.wait);
        if constexpr (CK) here = copies.wait(a.wait) && here;
        if (!here) give_up(a, &s.stop[n & 1]);
        f2 P = f2_both(1.f), H = none, R = none;
        auto gates = [&](auto run) {
            constexpr bool kPlain = decltype(run)::value;
#pragma unroll
            for (int j = 0; j < kRun; ++j) {
                f2 rv, iv, x;
                dyr[j] = in.get(0, j);
                if constexpr (CK) {
                    xr[j] = copies.get(0, j);
                    x = f2_mul(widen(xr[j]), steps[0]);
                    rv = f2_mul(widen(copies.get(1, j)), steps[1]);
                    iv = f2_mul(widen(copies.get(2, j)), steps[2]);
                } else {
                    rv = widen(in.get(1, j));
                    iv = widen(in.get(2, j));
                    xr[j] = in.get(3, j);
                    x = widen(xr[j]);
                }
                const Gate2 g = gate2<kPlain>(rv, iv, k);
                sr[j] = g.sr;
                sigmoid_i(j) = g.si;
                const f2 vx = f2_mul(g.si, x);
                if (kPlain || (j < left && !(marks >> j & 1))) {
                    H = j == 0 ? f2_mul(g.m, vx) : f2_fma(g.a, H, f2_mul(g.m, vx));
                    P = j == 0 ? g.a : f2_mul(P, g.a);
                    // R: dy times the decays up to and with its own, before any reset
                    if (kPlain || (marks & ((1u << j) - 1)) == 0)
                        R = f2_fma(P, widen(dyr[j]), R);
                } else if (j < left) {
                    P = f2_both(reset_decay());
                    H = vx;
                }
            }
        };
        if (plain) gates(PlainRun());
        else gates(AnyRun());
        s.maps[warp][lane] = as_map(P, H);
        float2 Rw;
        f2_unpack(R, Rw.x, Rw.y);
        s.right[warp][lane] = Rw;
        bar_arrive(kMapsReady);
        Tile tn;
        f2 kn = k;
        auto advance = [&] {
            in.request(a, maps.m, tn, src);
            if constexpr (CK) {
                copies.request(a, maps.m + 1, tn, csrc);
#pragma unroll
                for (int w = 0; w < 3; ++w) steps_next[w] = copy_step<ALIGNED>(a, tn, w);
            }
            mark = reset_byte(a, tn);
            kn = gate_scales<ALIGNED>(a, tn.d0);
        };
        ahead = false;
        if (EAGER) {
            tn = s.tile[(n + 1) & 1];
            ahead = here && tn.id < tiles;
            if (ahead && kAhead) advance();
        } else if (chained) {
            in.prefetch(a, maps.m, tiles, s.later[n & 1], src);
            if constexpr (CK) copies.prefetch(a, maps.m + 1, tiles, s.later[n & 1], csrc);
        }
        bar_sync(kEntryReady);
        if (s.stop[n & 1]) {
            if (!here) {
                in.wait(kDrain);
                if constexpr (CK) copies.wait(kDrain);
            }
            ahead = ahead && kAhead;
            break;
        }
        if (EAGER && !kAhead && ahead) advance();  // all warps have read their rows
        f2 dl = none;
        auto grads = [&](auto run) {
            constexpr bool kPlain = decltype(run)::value;
            const int64_t row = t.row0 + tok0 * a.D;
            Rows<T, ALIGNED> dx(a.dx, row, t.d0, a.D), dr(a.dr, row, t.d0, a.D),
                di(a.di, row, t.d0, a.D);
            f2 decay[kRun], G[kRun];
            f2 c = s.grad[warp][lane];
#pragma unroll
            for (int j = kRun - 1; j >= 0; --j) {
                if (kPlain || j < left) {
                    decay[j] = decay2<kPlain>(f2_mul(k, sr[j]));
                    G[j] = f2_add(widen(dyr[j]), c);
                    c = (!kPlain && (marks >> j & 1)) ? none : f2_mul(decay_of<kPlain>(decay[j]), G[j]);
                } else {
                    decay[j] = G[j] = none;
                }
            }
            f2 h = s.entry[warp][lane];
#pragma unroll
            for (int j = 0; j < kRun; ++j) {
                if (!kPlain && j >= left) break;
                const bool cut = !kPlain && (marks >> j & 1);
                Gate2 g;
                decay_from2<kPlain>(decay[j], f2_mul(k, sr[j]), g);
                const f2 x = CK ? f2_mul(widen(xr[j]), steps[0]) : widen(xr[j]);
                const f2 srj = sr[j], sij = sigmoid_i(j);
                const f2 vx = f2_mul(sij, x);  // sigmoid(i) x
                const f2 gm = cut ? G[j] : f2_mul(G[j], g.m);
                // q dm/dq = q a^2 / m: finite where q -> 0
                const f2 qa = f2_mul(f2_mul(k, srj), g.a);
                const f2 e = cut ? none
                                 : f2_mul(f2_mul(G[j], qa),
                                          f2_sub(f2_mul(f2_mul(g.a, g.rm), vx), h));
                dl = f2_add(dl, e);
                const f2 gv = f2_mul(gm, vx);
                dx.template put<kPlain>(f2_mul(gm, sij));
                // a reset token's decay gate counts for nothing, whatever it holds
                dr.template put<kPlain>(cut ? none : f2_mul(e, f2_sub(one, srj)));
                di.template put<kPlain>(f2_mul(gv, f2_sub(one, sij)));
                h = cut ? vx : f2_fma(g.a, h, f2_mul(g.m, vx));
            }
        };
        if (plain) grads(PlainRun());
        else grads(AnyRun());
        float2 dw;
        f2_unpack(dl, dw.x, dw.y);
        s.dlam[n & 1][warp][channel<ALIGNED>(0)] = dw.x;
        s.dlam[n & 1][warp][channel<ALIGNED>(1)] = dw.y;
        if (chained && !EAGER) {
            bar_sync(kTicketReady);
            tn = s.tile[0];
            ahead = tn.id < tiles;
            if (ahead) advance();
        }
        if (!ahead) {
            bar_arrive(kMapsReady);  // the chain warp takes the last tile's dlam
            break;
        }
        t = tn;
        k = kn;
        if constexpr (CK) {
#pragma unroll
            for (int w = 0; w < 3; ++w) steps[w] = steps_next[w];
        }
    }
    if (ahead) {
        in.wait(kDrain);
        if constexpr (CK) copies.wait(kDrain);
    }
}

// dlam: the blocks' sums over batch and blocks, times the channel's factor. 1/64 of a
// tensor's fp32 bytes; about 5 us at b8 L2048 D5120, most of it latency.
__global__ void __launch_bounds__(1024)
gated_dlam_kernel(const float *__restrict__ part, const float *__restrict__ lam,
                  float *__restrict__ dlam, int64_t rows, int64_t D) {
    __shared__ float red[32][33];
    after_previous();
    const int64_t d = (int64_t)blockIdx.x * 32 + threadIdx.x;
    const float s = column_sum(part, rows, D, d, threadIdx.y, 32);
    red[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    const float v = warp_sum(red[threadIdx.x][threadIdx.y]);
    const int64_t mine = (int64_t)blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && mine < D) dlam[mine] = v * lam_ratio(lam[mine]);
}

// One token. Bytes: 16 a channel in bf16 (5 us at b256 D8192, measured 8.3; a state
// that the last step left in L2 comes from there); at one row the launch is all of it.
// V neighbouring channels a thread, of `rows` batch rows after one
// another (the scale c softplus(lam) once for all of them). A row of channels takes
// `row_blocks` thread blocks.
template <typename T, int V>
__global__ void __launch_bounds__(kStepThreads)
gated_step_kernel(float *__restrict__ h, const T *__restrict__ x, const T *__restrict__ r,
                  const T *__restrict__ i, const float *__restrict__ lam, float c,
                  T *__restrict__ y, int64_t D, int64_t batch, int rows, unsigned row_blocks) {
    const unsigned part = blockIdx.x / row_blocks;
    const int64_t d = ((int64_t)(blockIdx.x - part * row_blocks) * kStepThreads + threadIdx.x) * V;
    if (d >= D) return;
    struct __align__(sizeof(T) * V) In {
        T v[V];
    };
    struct __align__(4 * V) State {
        float v[V];
    };
    float k[V];
#pragma unroll
    for (int j = 0; j < V; ++j) k[j] = c * softplus_full(lam[d + j]);
    const int64_t first = (int64_t)part * rows;
    const int64_t end = first + rows < batch ? first + rows : batch;
#pragma unroll 2
    for (int64_t at = first * D + d; at < end * D; at += D) {
        const In xs = *reinterpret_cast<const In *>(x + at), rs = *reinterpret_cast<const In *>(r + at),
                 is = *reinterpret_cast<const In *>(i + at);
        State hs = *reinterpret_cast<const State *>(h + at);
        In ys;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const Gate g = gate(to_f(rs.v[j]), to_f(is.v[j]), k[j]);
            hs.v[j] = fmaf(g.a, hs.v[j], g.m * g.si * to_f(xs.v[j]));
            ys.v[j] = from_f<T>(hs.v[j]);
        }
        *reinterpret_cast<State *>(h + at) = hs;
        *reinterpret_cast<In *>(y + at) = ys;
    }
}

// ------------------------------------------------------------ host

// Clears the words that tiles publish and the counter, and prepares the gate
// scales k = c softplus(lam). 1/32 of a bf16 tensor's bytes; about 2 us, partly
// behind the launch of the kernel that follows.
__global__ void gated_open_kernel(const GatedArgs a, int64_t ends, int64_t maps) {
    let_next();
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i == 0) *a.counter = *a.abort = 0;
    if (i < a.D) a.scale[i] = a.c * softplus_full(a.lam[i]);
    const ulonglong2 empty = make_ulonglong2(kEmpty, kEmpty);
    if (2 * i < ends) reinterpret_cast<ulonglong2 *>(a.ends)[i] = empty;
    if (2 * i < maps) reinterpret_cast<ulonglong2 *>(a.maps)[i] = empty;
}

// Thread blocks of K that fit the current device (0: an error), found once for
// each device; the kernel's shared memory is allowed on the way.
template <auto K>
int resident_blocks(size_t smem, cudaError_t *err) {
    static std::atomic<int> known[64];
    int dev = 0, per_sm = 0, sms = 0;
    if ((*err = cudaGetDevice(&dev)) != cudaSuccess) return 0;
    if (dev < 64) {
        const int n = known[dev].load(std::memory_order_relaxed);
        if (n > 0) return n;
    }
    if ((*err = cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) !=
            cudaSuccess ||
        (*err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess ||
        (*err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, K, kThreads, smem)) !=
            cudaSuccess)
        return 0;
    if (per_sm < 1) per_sm = 1;
    if (dev < 64) known[dev].store(per_sm * sms, std::memory_order_relaxed);
    return per_sm * sms;
}

// A persistent kernel's launch: as many thread blocks as fit, fewer where there
// are fewer tiles; with one block of tokens one per tile.
template <auto K>
cudaError_t start(const char *name, size_t smem, bool back, bool eager, GatedArgs a,
                  const Maps &maps, cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    const int64_t lanes = a.batch * a.dblocks, tiles = lanes * a.nb;
    int64_t grid = tiles, ends = 0, words = 0;
    // few lanes: groups of four tiles cost less to fold, of eight make half the chain. One
    // row of 16384 tokens, bf16, fours / eights: forward at 16 lanes 82 / 60 us, 24 85 / 79,
    // 28 91 / 89, 32 98 / 99, 48 134 / 139; backward at 4 lanes 48 / 32, 8 53 / 52, 12 69 /
    // 70, 24 119 / 123, 48 215 / 223 (65536 tokens, 32 lanes: 573 / 601, sixteens 640).
    a.group_bits = lanes >= (back ? 9 : 32) ? 2 : 3;
    const int64_t fit = resident_blocks<K>(smem, &e);
    if (e != cudaSuccess) return e;
    if (a.nb > 1) {
        if (fit < grid) grid = fit;
        ends = (eager ? tiles : lanes * (a.nb >> a.group_bits)) * 32;
        words = eager ? 0 : tiles * 64;
    }
    int64_t n = ends > words ? ends / 2 : words / 2;
    if (n < a.D) n = a.D;
    launch_begin("gated_open", st);
    gated_open_kernel<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(a, ends, words);
    launch_end(st);
    launch_begin(name, st);
    e = launch_after(K, (unsigned)grid, kThreads, smem, st, a, maps);
    launch_end(st);
    return e;
}

bool on(const void *p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

template <typename T>
bool encode(CUtensorMap *m, const void *base, const cuuint64_t (&dims)[4],
            const cuuint64_t (&strides)[3], const cuuint32_t (&box)[4]) {
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return tensor_map_encoder()(m, sizeof(T) == 4   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                        : sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                         : CU_TENSOR_MAP_DATA_TYPE_UINT8,
                     4, const_cast<void *>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A map over a (b, L, D) tensor whose box is one warp's rows of a tile. False
// where rows do not start on 16 bytes.
template <typename T>
bool warp_map(CUtensorMap *m, const void *base, const GatedArgs &a) {
    const uint64_t row = (uint64_t)a.D * sizeof(T);
    if (!tensor_map_encoder() || !on(base, 16) || row % 16 != 0 || row * (uint64_t)a.L >= 1ull << 40)
        return false;
    return encode<T>(m, base, {(cuuint64_t)a.D, (cuuint64_t)a.L, (cuuint64_t)a.batch, 1},
                     {row, row * (uint64_t)a.L, row * (uint64_t)a.L}, {kTileCh, kRun, 1, 1});
}

// A map of FlatRows over the same tensor: its whole groups of kSlots rows.
// False where there is none.
template <typename T>
bool flat_map(CUtensorMap *m, const void *base, int64_t rows, const GatedArgs &a) {
    using F = FlatRows<T, 1>;
    const uint64_t groups = (uint64_t)rows / F::kSlots;
    const uint64_t row = (uint64_t)a.D * sizeof(T) * F::kSlots;
    if (!tensor_map_encoder() || !on(base, 16) || groups == 0 || groups >= 1ull << 31 ||
        row * groups >= 1ull << 40)
        return false;
    return encode<T>(m, base, {(cuuint64_t)a.D * F::kSlots, groups, 1, 1},
                     {row, row * groups, row * groups},
                     {kTileCh + F::kUnit, F::kSlotRows, 1, 1});
}

// The maps of `n` tensors, of warps' rows or flat ones; whether they are there.
template <typename T>
bool warp_maps(CUtensorMap *m, const void *const *base, int n, const GatedArgs &a) {
    for (int w = 0; w < n; ++w)
        if (!warp_map<T>(m + w, base[w], a)) return false;
    return true;
}
template <typename T>
bool flat_maps(CUtensorMap *m, const void *const *base, int n, const GatedArgs &a) {
    for (int w = 0; w < n; ++w)
        if (!flat_map<T>(m + w, base[w], a.batch * a.L, a)) return false;
    return true;
}

// Many lanes or few (see the top): the chain of waits takes 0.7 to 1.3 us a step (a tile
// of each lane), which a GPU full of thread blocks spends on other lanes' tiles from about
// lanes for half the SMs on. Groups of four / waiting, one row of 8192 tokens, us:
//   lanes            64          80          96          128
//   bf16 forward     89 / 101    107 / 112   125 / 123   157 / 145
//   bf16 backward    143 / 145   175 / 167   206 / 194   268 / 248
//   bf16 copies      121 / 140   146 / 146   173 / 161   228 / 198, backward 169 / 163 ... 322 / 284
//   fp32 forward     109 / 107   130 / 118   152 / 132   199 / 164
//   fp32 backward    202 / 196   248 / 246   295 / 292   394 / 378
// Rows that start anywhere: bf16 as these, but fp32's backward pass (262 / 282 at 80 lanes)
// and those from copies (249 / 264) lose 4 to 12 % by waiting at all counts. At 32 lanes
// and 65536 tokens waiting takes 1314 us and groups 365.
bool many_lanes(const GatedArgs &a, cudaError_t *e) {
    int dev = 0, sms = 0;
    if ((*e = cudaGetDevice(&dev)) != cudaSuccess ||
        (*e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
        return false;
    return a.nb > 1 && 2 * a.batch * a.dblocks >= sms;
}

template <typename T, bool ALIGNED, bool CK>
cudaError_t forward_t(const GatedArgs &a, const Maps &maps, cudaStream_t st) {
    constexpr size_t ahead = Stage<T, ALIGNED, 3, kForwardKeep<ALIGNED, CK, true>>::kBytes,
                     kept = Stage<T, ALIGNED, 3, kForwardKeep<ALIGNED, CK, false>>::kBytes;
    constexpr auto *many = gated_forward_kernel<T, ALIGNED, CK, true>;
    constexpr auto *few = gated_forward_kernel<T, ALIGNED, CK, false>;
    cudaError_t e = cudaSuccess;
    const bool eager = many_lanes(a, &e);
    if (e != cudaSuccess) return e;
    return eager ? start<many>("gated_forward", ahead, false, true, a, maps, st)
                 : start<few>("gated_forward", kept, false, false, a, maps, st);
}
template <typename T, bool ALIGNED>
cudaError_t forward_c(const GatedArgs &a, const Maps &maps, cudaStream_t st) {
    return a.q ? forward_t<T, ALIGNED, true>(a, maps, st) : forward_t<T, ALIGNED, false>(a, maps, st);
}
template <typename T>
cudaError_t forward_v(GatedArgs a, cudaStream_t st) {
    Maps maps;
    const void *const in[3] = {a.x, a.r, a.i};
    const bool aligned = on(a.y, 8) && on(a.q, 4) && warp_maps<T>(maps.m, in, 3, a);
    if (!aligned) a.flat = flat_maps<T>(maps.m, in, 3, a);
    return aligned ? forward_c<T, true>(a, maps, st) : forward_c<T, false>(a, maps, st);
}

template <typename T, bool ALIGNED, bool CK>
cudaError_t backward_t(const GatedArgs &a, const Maps &maps, cudaStream_t st) {
    constexpr size_t smem =
        Stage<T, ALIGNED, CK ? 1 : 4>::kBytes + (CK ? Stage<int8_t, ALIGNED, 3>::kBytes : 0) +
        kBackwardKeep<ALIGNED, CK>;
    constexpr auto *many = gated_backward_kernel<T, ALIGNED, CK, true>;
    constexpr auto *few = gated_backward_kernel<T, ALIGNED, CK, false>;
    cudaError_t e = cudaSuccess;
    const bool eager = many_lanes(a, &e);
    if (e != cudaSuccess) return e;
    return eager ? start<many>("gated_backward", smem, true, true, a, maps, st)
                 : start<few>("gated_backward", smem, true, false, a, maps, st);
}
template <typename T, bool ALIGNED>
cudaError_t backward_c(const GatedArgs &a, const Maps &maps, cudaStream_t st) {
    return a.q ? backward_t<T, ALIGNED, true>(a, maps, st)
               : backward_t<T, ALIGNED, false>(a, maps, st);
}
template <typename T>
cudaError_t backward_v(GatedArgs a, float *dlam, cudaStream_t st) {
    Maps maps;
    const int64_t n = a.batch * a.L * a.D;
    const void *const in[4] = {a.dy, a.r, a.i, a.x};
    const void *const copies[3] = {a.q, a.q + n, a.q + 2 * n};
    const int own = a.q ? 1 : 4;
    const bool aligned = on(a.dx, 8) && on(a.dr, 8) && on(a.di, 8) &&
                         warp_maps<T>(maps.m, in, own, a) &&
                         (!a.q || warp_maps<int8_t>(maps.m + 1, copies, 3, a));
    if (!aligned)
        a.flat = flat_maps<T>(maps.m, in, own, a) &&
                 (!a.q || flat_map<int8_t>(&maps.m[1], a.q, 3 * a.batch * a.L, a));
    cudaError_t e = aligned ? backward_c<T, true>(a, maps, st) : backward_c<T, false>(a, maps, st);
    if (e != cudaSuccess) return e;
    launch_begin("gated_dlam", st);
    e = launch_after(gated_dlam_kernel, (unsigned)((a.D + 31) / 32), dim3(32, 32), 0, st,
                     a.dlam_part, a.lam, dlam, a.batch * a.nb, a.D);
    launch_end(st);
    return e;
}

// Pairs of channels where rows allow them and there is work for every SM all the
// same (b256 D8192: 10.3 us for 12.3), and up to eight rows a thread while eight
// thread blocks an SM are left (8.3 us). 148 SMs: the B200's; asking the device would
// cost the host more than a call's kernel takes, and nothing but speed hangs on it.
template <typename T>
void step_v(const Problem &pr, float *h, const void *x, const void *r, const void *i,
            const float *lam, float c, void *y, cudaStream_t st) {
    const int64_t D = pr.nheads;
    const bool pairs = D % 2 == 0 && on(h, 8) && on(x, 2 * sizeof(T)) && on(r, 2 * sizeof(T)) &&
                       on(i, 2 * sizeof(T)) && on(y, 2 * sizeof(T)) &&
                       pr.batch * D >= 148 * 2 * kStepThreads;
    const int64_t block = kStepThreads * (pairs ? 2 : 1);
    const int64_t row_blocks = (D + block - 1) / block;
    const int64_t fill = pr.batch * row_blocks / (148 * 8);
    const int64_t rows = fill < 1 ? 1 : fill < 8 ? fill : 8;
    const unsigned grid = (unsigned)((pr.batch + rows - 1) / rows * row_blocks);
    auto *kernel = pairs ? gated_step_kernel<T, 2> : gated_step_kernel<T, 1>;
    kernel<<<grid, kStepThreads, 0, st>>>(h, static_cast<const T *>(x), static_cast<const T *>(r),
                                          static_cast<const T *>(i), lam, c, static_cast<T *>(y), D,
                                          pr.batch, (int)rows, (unsigned)row_blocks);
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
    a.counter = reinterpret_cast<unsigned *>(take(256));
    a.abort = a.counter + 32;
    a.scale = reinterpret_cast<float *>(take((size_t)a.D * sizeof(float)));
    if (a.nb > 1) {
        a.ends = reinterpret_cast<unsigned long long *>(take(tiles * 32 * 8));
        a.maps = reinterpret_cast<unsigned long long *>(take(tiles * 32 * 16));
    }
    if (back)
        a.dlam_part = reinterpret_cast<float *>(take((size_t)(a.batch * a.nb * a.D) * sizeof(float)));
    return at;
}

}  // namespace

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault,
                                                &q) == cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p) : nullptr;
    }();
    return fn;
}

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
    launch_begin("gated_step", st);
    if (pr.dtype == SSD_F32)
        step_v<float>(pr, h, x, r, i, lam, c, y, st);
    else
        step_v<__nv_bfloat16>(pr, h, x, r, i, lam, c, y, st);
    launch_end(st);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SSD_OK : cuda_fail(e, "gated step launch");
}

}  // namespace ssd
