// The gated linear recurrence: every channel c of a packed batch has a state of its own,
//     h_t = e^{g_t} h_{t-1} + w_t x_t,   w = 1 (add) or 1 - e^{g_t} (mix),
// from h0 at the start of its sequence.  Backward, from the last token to the first, with
// u_t = e^{g_t} dh_t the adjoint that a step hands to the one before it:
//     dh_t = d_t + u_{t+1},   dx_t = w_t dh_t,   dg_t = u_t (h_{t-1} [- x_t]),   dh0 = u_first.
//
// Both are scans of maps s -> A s + B (A the product of the factors e^g, B the result from a
// zero start), which compose: a tile of some tokens x 64 channels is one map per channel.
// Every element should be read and written once, so the scan takes one pass: the warps of a
// block each run some of a tile's tokens (a lane has two channels) and join their maps; the
// block publishes the tile's map, looks back along the chain for what enters it, and writes its
// tokens.  Tiles are handed out by a counter so that a tile follows those that it waits for,
// which are then already being worked on; of few sequences they take turns, so that they are
// done, too.
//
// Eight tiles along a chain are a group.  The last of them publishes the group's map and, once
// it knows it, the group's end: the state that leaves it.  A tile's state comes from the nearest
// end that is there, through the maps of the groups after it and of its own group's earlier
// tiles, one at a time and in this order whoever computes it, so the results do not depend on
// how far a look back went.
//
// Without its look back the pass takes the time of its bytes, so that is what the layout hides:
// maps and ends are words that a NaN of their own marks as absent (no flag beside the data, no
// fence between the two, one trip to L2 for both); the window is asked for while the tile's
// tokens come; the forward pass holds a tile in registers while the next one's tokens come
// (TMA); tiles are large and few are in flight.  Measured, in ms (forward 81,920 x 7,168 and
// gradient of 81,920 x 4,096, BF16, mix: their bytes take 0.69 and 0.79; forward 1,048,576 x
// 512, add, 0.63): flags, and maps read four at a time, 1.62, 2.36, 3.75; words that mark
// themselves 0.82, 1.06, 3.39; as it is now 0.84, 0.83, 1.19.
//
// Batches of few tokens have no look back: a block takes all tiles of a sequence's 64
// channels one after another.
#include <math.h>

#include "kda_f2.cuh"
#include "kda_internal.cuh"
#include "kda_sm100.cuh"

namespace kda {
namespace {

using namespace sm100;

constexpr int kChan = 64;
// A tile: so many warps and tokens of each, by how the tokens come (TMA, or lane by lane).
// With TMA one block of 256 tokens to an SM has all of its registers in use (a warp holds its
// 32 tokens' factors and terms), and a chain has few steps: 81,920 x 7,168 BF16 takes 823 us,
// two blocks of 128 810, three 950; 1,048,576 x 512 1.22, 1.76 and 2.51 ms; 81,920 x 2,048
// fp32, four sequences, 297 us, 311, 311 (one sequence takes 316).  Loads of single lanes want
// warps: 81,920 x 2,047 BF16 800 us with three blocks of eight warps, 1,414 as with TMA, although
// with 80 registers 390 to 480 bytes a thread of the held tile are in local memory (walking, 140
// to 160).  The backward pass holds nothing: with TMA
// 128 tokens 834 us (81,920 x 4,096), 64 872; lane by lane 147 and 116 (20,011 x 1,001 fp32).
constexpr int warps_of(bool bwd, bool tma) { return bwd && !tma ? 4 : 8; }
constexpr int tok_of(bool bwd, bool tma) { return !bwd && tma ? 32 : 16; }
constexpr int tile_of(bool bwd, bool tma) { return warps_of(bwd, tma) * tok_of(bwd, tma); }
constexpr long long kWaitLimit = 4000000000ll;  // ~2 s of SM clocks
// Up to so many tokens one block walks a sequence; beyond, a launch lays out the tiles of a
// batch first (BF16 forward, 512 channels: 257 tokens walking 9.2 us, so 7.4, 400 12.4 and 8.4;
// 7,168: 11.1 and 12.9, 15.6 and 14.1).
constexpr int kWalkTokens = 256;

struct RecArgs {
    const void *x;
    const float *g, *h0;
    const int32_t *cu;  // NULL: one sequence
    void *h;
    float *h_final;
    const void *d, *hs;  // backward: adjoint of h, and h
    const float *d_final;
    void *dx;
    float *dg, *d_h0;
    long long x_stride, g_stride;  // elements between tokens
    int N, T, C, groups;
    int32_t *status;
    // the look back
    int4 *tiles;         // [tiles] in the order of work: row of maps and ends, first token, 256
                         // sequence + tokens - 1, 2 (place in the chain) + last
    float2 *maps;        // [tiles][64 groups]
    float *ends;         // [tiles][64 groups], behind maps
    unsigned *control;   // next tile, tiles, a wait gave up
    int most_tiles, window;  // window: tiles that a look back reads
    long long wait_limit;    // of a look back, in SM clocks
};
enum { NEXT = 0, TILES = 1, ABORT = 2 };

__device__ __forceinline__ int begin_of(const RecArgs &p, int n) { return p.cu ? p.cu[n] : 0; }
__device__ __forceinline__ int end_of(const RecArgs &p, int n) { return p.cu ? p.cu[n + 1] : p.T; }

// a = e^g and w = 1 - e^g of two channels.  Slow decays are what a state keeps for thousands
// of steps, so a comes from the exact side: for |g| < 0.34 w is the series of 1 - e^g (seven
// terms, the next is below 2^-25 of w) and a = 1 - w is rounded once; ex2.approx alone is up
// to 2^-22 off, every step in the same direction for a constant gate.
__device__ __forceinline__ void decay2(f2 g, f2 &a, f2 &w) {
    const float2 t = un(mul2(g, both(1.4426950408889634f)));
    const float2 e = make_float2(ex2(t.x), ex2(t.y));
    f2 s = fma2(g, both(-1.f / 5040.f), both(-1.f / 720.f));
    s = fma2(g, s, both(-1.f / 120.f));
    s = fma2(g, s, both(-1.f / 24.f));
    s = fma2(g, s, both(-1.f / 6.f));
    s = fma2(g, s, both(-0.5f));
    const f2 ng = mul2(g, both(-1.f));
    const float2 series = un(fma2(mul2(g, g), s, ng)), v = un(g);
    const float2 far = un(fma2(pk(e.x, e.y), both(-1.f), both(1.f)));
    const bool near0 = fabsf(v.x) < 0.34f, near1 = fabsf(v.y) < 0.34f;
    w = pk(near0 ? series.x : far.x, near1 ? series.y : far.y);
    const float2 one = un(fma2(w, both(-1.f), both(1.f)));
    a = pk(near0 ? one.x : e.x, near1 ? one.y : e.y);
}

// A state through a map; a product of growing factors may be infinite where the state is zero.
__device__ __forceinline__ float through(float A, float B, float s) {
    return s == 0.f ? B : fmaf(A, s, B);
}
__device__ __forceinline__ float2 through(const float4 &m, float2 s) {  // two channels
    return make_float2(through(m.x, m.y, s.x), through(m.z, m.w, s.y));
}

// Two channels of one token.
__device__ __forceinline__ f2 get2(const float *p) {
    const float2 v = *(const float2 *)p;
    return pk(v.x, v.y);
}
__device__ __forceinline__ f2 get2(const __nv_bfloat16 *p) {
    const uint32_t v = *(const uint32_t *)p;
    return pk(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
// The same from global memory, `n` of them in the row; PAIRS: aligned to both.
template <bool PAIRS, typename T>
__device__ __forceinline__ f2 load2(const T *p, int n) {
    if (PAIRS) return n > 0 ? get2(p) : pk(0.f, 0.f);
    return pk(n > 0 ? act_ld(p, 0) : 0.f, n > 1 ? act_ld(p, 1) : 0.f);
}
template <bool PAIRS>
__device__ __forceinline__ void store2(float *p, int n, f2 v) {
    const float2 u = un(v);
    if (n <= 0) return;
    if (PAIRS) {
        __stcs((float2 *)p, u);
    } else {
        p[0] = u.x;
        if (n > 1) p[1] = u.y;
    }
}
template <bool PAIRS>
__device__ __forceinline__ void store2(__nv_bfloat16 *p, int n, f2 v) {
    const float2 u = un(v);
    if (n <= 0) return;
    if (PAIRS) {
        __stcs((uint32_t *)p, pack_bf16x2(u.x, u.y));
    } else {
        act_st(p, 0, u.x);
        if (n > 1) act_st(p, 1, u.y);
    }
}

// A word of maps or ends that nobody has written yet: a NaN that arithmetic does not make
// (its own is 0x7fffffff; were this one ever to come up, that is stored instead).  The copies
// that poll them promise no order and nothing wider than a word, so each word is looked at.
constexpr uint32_t kNone = 0xffffffffu;
__device__ __forceinline__ bool there(float v) { return __float_as_uint(v) != kNone; }
__device__ __forceinline__ float told(float v) { return there(v) ? v : __uint_as_float(0x7fffffffu); }
__device__ __forceinline__ void tell(void *p, float a, float b) {  // two words at once
    asm volatile("st.relaxed.gpu.b64 [%0], %1;" ::"l"(p), "l"(pk(told(a), told(b))) : "memory");
}

struct TileAt {
    int seq, t0, t1, place, group, index;
    bool last;
};

// A tile's entry in a look back's window: maps of 64 channels, then their ends.
constexpr int kEntry = kChan * 12;

// Tiles go in groups of eight along a chain.  A tile of a group publishes its map, the group's
// last one the group's map instead, and its end: with one step for eight tiles, a chain of
// few channels and many tokens is not bound by the look back's latency (1,048,576 x 512: 1.73
// ms where every tile was a step).
constexpr int kGroup = 8;
// A look back reads so many groups at first, and twice as many when all their maps are there
// and no end.
constexpr int kFirstRead = 2;
constexpr int kUsualWindow = 10;  // entries, of a batch of many channels

// 8-byte asynchronous copy global -> shared (zero fill when !pred).
__device__ __forceinline__ void cp_async8(uint32_t dst, const void *src, bool pred) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src),
                 "r"(pred ? 8 : 0)
                 : "memory");
}
// A lane's `n` channels of a token into shared memory.
template <bool PAIRS>
__device__ __forceinline__ void fetch(uint32_t dst, const float *src, const float *some, int n) {
    if (PAIRS) {
        cp_async8(dst, n > 0 ? src : some, n > 0);
    } else {
        cp_async4(dst, n > 0 ? src : some, n > 0);
        cp_async4(dst + 4, n > 1 ? src + 1 : some, n > 1);
    }
}
template <bool PAIRS>
__device__ __forceinline__ void fetch(uint32_t dst, const __nv_bfloat16 *src, const float *some, int n) {
    if (PAIRS) {
        cp_async4(dst, n > 0 ? (const void *)src : some, n > 0);
    } else {
        const unsigned short *q = (const unsigned short *)src;
        const uint32_t v = (n > 0 ? q[0] : 0u) | (n > 1 ? (uint32_t)q[1] << 16 : 0u);
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst), "r"(v) : "memory");
    }
}

struct Yes {
    static constexpr bool value = true;
};
struct No {
    static constexpr bool value = false;
};

// How a tile's tokens come: by TMA, or lane by lane, pairs of channels or single ones.
enum { BY_TMA = 0, BY_PAIRS = 1, BY_ONE = 2 };

template <typename T, bool BWD, bool MIX, bool TMA>
struct Stage {  // a warp's part of a tile in shared memory
    static constexpr int tok = tok_of(BWD, TMA), warps = warps_of(BWD, TMA);
    static constexpr int g = 0, v = tok * kChan * 4, one = tok * kChan * (int)sizeof(T);
    static constexpr int h = v + one, x = h + (BWD ? one : 0), bytes = x + (BWD && MIX ? one : 0);
    static constexpr int block = warps * bytes;
    // blocks to an SM, with a window of so many entries
    static constexpr int most = BWD ? 6 : TMA ? 1 : 3;
    static constexpr int fit(int window) {
        const int n = 227 * 1024 / (block + (BWD ? 1 : 2) * window * kEntry + 10 * 1024);
        return n < 1 ? 1 : n < most ? n : most;
    }
};

template <typename T, bool BWD, bool MIX, int BY, bool SPLIT>
__global__ void __launch_bounds__(32 * warps_of(BWD, BY == BY_TMA),
                                  Stage<T, BWD, MIX, BY == BY_TMA>::fit(kUsualWindow))
    recurrence_kernel(const __grid_constant__ RecArgs p, const __grid_constant__ CUtensorMap tm_g,
                      const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ CUtensorMap tm_h,
                      const __grid_constant__ CUtensorMap tm_x) {
    using S = Stage<T, BWD, MIX, BY == BY_TMA>;
    constexpr int TOK = S::tok, kWarps = S::warps, kTile = TOK * kWarps;
    constexpr bool PAIRS = BY != BY_ONE;
    extern __shared__ __align__(128) uint8_t sm_raw[];
    __shared__ float4 maps[2][kWarps][32];  // (A, B) of two channels
    __shared__ float2 carry[2][32];         // without a look back
    __shared__ uint2 seen[2][kWarps];       // a warp's entries of the window: maps, ends
    __shared__ int4 tile_at[2];             // this block's tiles, in turn
    __shared__ int ticket_at[2];
    __shared__ __align__(8) uint64_t bars[kWarps];
    __shared__ int abort_flag;
    // Whether a wait gave up, told and read with `seen` (one thread's view at some moment could
    // be another's at the next, and a warp would leave a loop whose barriers others still enter).
    __shared__ bool gave_up[2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const T *x = (const T *)p.x, *d = (const T *)p.d, *hs = (const T *)p.hs;
    const float *first = BWD ? p.d_final : p.h0;
    float *final_out = BWD ? p.d_h0 : p.h_final;
    uint8_t *sm = sm_raw + ((128u - (smem_addr(sm_raw) & 127u)) & 127u);
    uint8_t *windows = sm + S::block;
    if (threadIdx.x == 0) {
        abort_flag = 0;
        gave_up[0] = gave_up[1] = false;
        if (BY == BY_TMA) {
            for (int w = 0; w < kWarps; ++w) mbar_init(smem_addr(&bars[w]), 1);
            mbar_fence_init();
        }
    }
    griddep_wait();
    griddep_launch_dependents();

    int total = 0, begin = 0, end = 0, walk_seq = 0, walk_group = 0;
    auto take = [&](int &ticket, int4 &tile) {  // one thread
        ticket = (int)atomicAdd(p.control + NEXT, 1u);
        const int k = ticket / p.groups;
        tile = make_int4(0, 0, 0, 0);
        if (k < total) tile = p.tiles[k];
    };
    if (SPLIT) {
        total = (int)p.control[TILES];
        if (threadIdx.x == 0) take(ticket_at[0], tile_at[0]);
    } else {
        walk_seq = blockIdx.x / p.groups;
        walk_group = blockIdx.x - walk_seq * p.groups;
        begin = begin_of(p, walk_seq);
        end = end_of(p, walk_seq);
        const bool good = !p.cu || (begin >= 0 && begin <= end && end <= p.T && p.cu[0] == 0 &&
                                    p.cu[p.N] == p.T);
        if (!good) {
            if (threadIdx.x == 0) dev_fail(p.status, KDA_ERR_INVALID_ARG);
            return;
        }
        if (warp == 0) {
            const int c = walk_group * kChan + 2 * lane;
            const f2 s = first ? load2<false>(first + (size_t)walk_seq * p.C + c, p.C - c) : pk(0.f, 0.f);
            carry[0][lane] = un(s);
            if (begin == end && final_out)
                store2<false>(final_out + (size_t)walk_seq * p.C + c, p.C - c, s);
        }
    }
    __syncthreads();

    // This block's k-th tile; false beyond its last.
    auto turn = [&](int k, TileAt &t) {
        int4 v;
        if (SPLIT) {
            const int ticket = ticket_at[k & 1], row = ticket / p.groups;
            if (row >= total) return false;
            v = tile_at[k & 1];
            t.index = v.x;
            t.seq = (int)((unsigned)v.z >> 8);
            t.t1 = v.y + (v.z & 255) + 1;
            t.group = ticket - row * p.groups;
        } else {
            const int n = (end - begin + kTile - 1) / kTile;
            if (k >= n) return false;
            const int t0 = begin + (BWD ? n - 1 - k : k) * kTile;
            v = make_int4(0, t0, 0, 2 * k + (k == n - 1));
            t.index = 0;
            t.seq = walk_seq;
            t.t1 = min(t0 + kTile, end);
            t.group = walk_group;
        }
        t.t0 = v.y;
        t.place = v.w >> 1;
        t.last = v.w & 1;
        return true;
    };
    // This warp's copies of its part of the k-th tile.
    auto start = [&](int k) {
        TileAt t;
        if (!turn(k, t)) return;
        const uint32_t stage = smem_addr(sm) + warp * S::bytes;
        const int y = t.t0 + warp * TOK;
        if constexpr (BY == BY_TMA) {
            if (lane != 0) return;
            const int c = t.group * kChan;
            const uint32_t bar = smem_addr(&bars[warp]);
            mbar_arrive_expect_tx(bar, S::bytes);
            tma_load_2d(stage + S::g, reinterpret_cast<uint64_t>(&tm_g), c, y, bar);
            tma_load_2d(stage + S::v, reinterpret_cast<uint64_t>(&tm_v), c, y, bar);
            if (BWD) tma_load_2d(stage + S::h, reinterpret_cast<uint64_t>(&tm_h), c, y - 1, bar);
            if (BWD && MIX) tma_load_2d(stage + S::x, reinterpret_cast<uint64_t>(&tm_x), c, y, bar);
        } else {
            const int c = t.group * kChan + 2 * lane, left = p.C - c;
            const uint32_t to = stage + 8 * lane, to_t = stage + 2 * (int)sizeof(T) * lane;
#pragma unroll 8
            for (int j = 0; j < TOK; ++j) {
                const int n = y + j < t.t1 ? left : 0;
                const size_t row = (size_t)(y + j), at = row * p.C + c;
                constexpr int step = kChan * (int)sizeof(T);
                fetch<PAIRS>(to + S::g + j * kChan * 4, p.g + row * p.g_stride + c, p.g, n);
                fetch<PAIRS>(to_t + S::v + j * step, BWD ? d + at : x + row * p.x_stride + c, p.g, n);
                if (BWD) fetch<PAIRS>(to_t + S::h + j * step, hs + at - p.C, p.g, y + j > 0 ? n : 0);
                if (BWD && MIX)
                    fetch<PAIRS>(to_t + S::x + j * step, x + row * p.x_stride + c, p.g, n);
            }
            cp_async_commit();
        }
    };
    // Two channels of token j of an array of the tile.
    auto gate = [&](int j) {
        return get2((const float *)(sm + warp * S::bytes + S::g + j * kChan * 4 + 8 * lane));
    };
    auto item = [&](int array, int j) {
        return get2((const T *)(sm + warp * S::bytes + array + (j * kChan + 2 * lane) * (int)sizeof(T)));
    };
    auto tokens = [&](const TileAt &t) { return max(0, min(TOK, t.t1 - t.t0 - warp * TOK)); };
    f2 fa[BWD ? 1 : TOK], fb[BWD ? 1 : TOK];  // forward: the tile's factors and terms
    unsigned polls = 0;
    // The map of this warp's tokens of the k-th tile; false if they did not come.
    auto reduce = [&](int k, const TileAt &t, auto hold) {
        bool landed = true;
        if (BY == BY_TMA) {
            landed = __all_sync(0xffffffffu, mbar_wait(smem_addr(&bars[warp]), k & 1, &abort_flag,
                                                       kWaitLimit));
            if (!landed) gave_up[polls & 1] = true;
        } else {
            cp_async_wait_all();  // every lane reads what it copied itself
        }
        const int n = tokens(t);
        f2 A = both(1.f), B = both(0.f);
        auto run = [&](auto whole) {
#pragma unroll
            for (int i = 0; i < TOK; ++i) {
                const int j = BWD ? TOK - 1 - i : i;
                f2 f = both(1.f), w, v = both(0.f);
                if (whole.value || j < n) {
                    decay2(gate(j), f, w);
                    v = item(S::v, j);
                    if (!BWD && MIX) v = mul2(w, v);
                }
                B = BWD ? mul2(f, add2(B, v)) : fma2(f, B, v);
                A = mul2(A, f);
                if constexpr (hold.value) {
                    fa[j] = f;
                    fb[j] = v;
                }
            }
        };
        if (n == TOK) run(Yes{});
        else run(No{});
        const float2 ua = un(A), ub = un(B);
        maps[k & 1][warp][lane] = make_float4(ua.x, ub.x, ua.y, ub.y);
        return landed;
    };
    // After a barrier: the map of the warps before this one, and (of use in the warp that
    // publishes it) of the tile.
    auto join = [&](int k, const TileAt &t, float4 &before, float4 &whole) {
        float4 m = make_float4(1.f, 0.f, 1.f, 0.f);
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            const int w = BWD ? kWarps - 1 - i : i;
            if (w == warp) before = m;
            const float4 v = maps[k & 1][w][lane];
            const float2 to = through(v, make_float2(m.y, m.w));
            m = make_float4(m.x * v.x, to.x, m.z * v.z, to.y);
        }
        whole = m;
        if (SPLIT && warp == 0 && !t.last && t.place % kGroup != kGroup - 1) {
            const size_t slot = ((size_t)t.index * p.groups + t.group) * kChan + 2 * lane;
            tell(p.maps + slot, m.x, m.y);
            tell(p.maps + slot + 1, m.z, m.w);
        }
    };

    start(0);
    TileAt t;
    for (int k = 0; turn(k, t); ++k) {
        int ahead_ticket = 0;
        int4 ahead;
        if (!BWD && SPLIT && threadIdx.x == 0) take(ahead_ticket, ahead);
        const int c = t.group * kChan + 2 * lane, left = p.C - c;
        // The look back's window: the maps of the group's earlier tiles, then of earlier groups
        // their maps and ends, all nearest first.  The warps read its entries in turn, for the
        // first time while the tile's tokens come, and again while they are not there.
        const int inside = t.place % kGroup, groups = t.place / kGroup;
        uint8_t *window = windows + (BWD ? 0 : (k & 1) * (p.window + kGroup - 1) * kEntry);
        const int most = inside + min(p.window, groups);
        int asked = min(inside + kFirstRead, most);
        unsigned have_maps = 0, have_ends = 0;
        auto ask = [&]() {
            const size_t pitch = (size_t)p.groups * kChan;
            for (int q = warp; q < asked; q += kWarps) {
                const int back = q < inside ? q + 1 : inside + 1 + kGroup * (q - inside);
                const size_t at = (size_t)(t.index + (BWD ? back : -back)) * pitch + t.group * kChan;
                const uint32_t to = smem_addr(window) + q * kEntry;
                if (!(have_maps >> q & 1)) cp_async16(to + 16 * lane, p.maps + at + 2 * lane, true);
                if (q >= inside && !(have_ends >> q & 1) && lane < 16)
                    cp_async16(to + kChan * 8 + 16 * lane, p.ends + at + 4 * lane, true);
            }
        };
        auto look = [&]() {
            cp_async_wait_all();
            __syncwarp();
            for (int q = warp; q < asked; q += kWarps) {
                const uint8_t *at = window + q * kEntry;
                if (!(have_maps >> q & 1)) {
                    const float4 v = *(const float4 *)(at + 16 * lane);
                    const bool a = there(v.x) && there(v.z), b = there(v.y) && there(v.w);
                    if (!__any_sync(0xffffffffu, !a || !b)) have_maps |= 1u << q;
                }
                if (q >= inside && !(have_ends >> q & 1)) {
                    const float2 v = *(const float2 *)(at + kChan * 8 + 8 * lane);
                    if (__all_sync(0xffffffffu, there(v.x) && there(v.y))) have_ends |= 1u << q;
                }
            }
            if (lane == 0) seen[polls & 1][warp] = make_uint2(have_maps, have_ends);
        };
        if (SPLIT) ask();  // into the window that this tile's turn has
        bool landed;
        if constexpr (BWD) landed = reduce(k, t, No{});
        else landed = reduce(k, t, Yes{});
        if (!BWD && SPLIT && threadIdx.x == 0) {
            ticket_at[(k + 1) & 1] = ahead_ticket;
            tile_at[(k + 1) & 1] = ahead;
        }
        if (SPLIT) look();
        __syncthreads();
        float4 before, whole;
        join(k, t, before, whole);
        if (!BWD && landed) start(k + 1);  // the tile is in registers

        // the state that enters the tile, in every warp
        float2 in, group_in = make_float2(0.f, 0.f);  // into the tile, into its group
        bool failed = false;
        if (!SPLIT) {
            in = carry[k & 1][lane];
        } else {
            bool closed = false;
            const bool closes = inside == kGroup - 1 && !t.last;
            const long long since = clock64();
            int from = 0;  // entries up to the end that is taken
            if (groups == 0)
                group_in = un(first ? load2<false>(first + (size_t)t.seq * p.C + c, left) : pk(0.f, 0.f));
            while (true) {
                unsigned all_maps = 0, all_ends = 0;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const uint2 v = seen[polls & 1][w];
                    all_maps |= v.x;
                    all_ends |= v.y;
                }
                failed = gave_up[polls & 1];
                ++polls;
                if (failed) break;
                const bool known = !(~all_maps & ((1u << inside) - 1));
                if (warp == 0 && closes && known && !closed) {  // the group's map
                    float4 m = *(const float4 *)(window + (inside - 1) * kEntry + 16 * lane);
                    for (int q = inside - 2; q >= -1; --q) {
                        const float4 v = q < 0 ? whole : *(const float4 *)(window + q * kEntry + 16 * lane);
                        const float2 to = through(v, make_float2(m.y, m.w));
                        m = make_float4(m.x * v.x, to.x, m.z * v.z, to.y);
                    }
                    const size_t slot = ((size_t)t.index * p.groups + t.group) * kChan + 2 * lane;
                    tell(p.maps + slot, m.x, m.y);
                    tell(p.maps + slot + 1, m.z, m.w);
                    whole = m;
                    closed = true;
                }
                // the nearest end, if every nearer map is there too: the same in every warp
                from = groups == 0 ? inside : __ffs(all_ends) - 1;
                if (from >= 0 && !(~all_maps & ((1u << from) - 1))) break;
                if (threadIdx.x == 0 && (polls & 63) == 0 &&
                    (clock64() - since > p.wait_limit || *(volatile unsigned *)(p.control + ABORT))) {
                    *(volatile unsigned *)(p.control + ABORT) = 1;
                    gave_up[polls & 1] = true;
                }
                if (from < 0 && __popc(all_maps) == asked) asked = min(2 * asked, most);
                ask();
                look();
                __syncthreads();
            }
            if (!failed) {
                if (groups > 0) {
                    group_in = *(const float2 *)(window + from * kEntry + kChan * 8 + 8 * lane);
#pragma unroll 4
                    for (int q = from - 1; q >= inside; --q)
                        group_in = through(*(const float4 *)(window + q * kEntry + 16 * lane), group_in);
                }
                in = group_in;
#pragma unroll 4
                for (int q = inside - 1; q >= 0; --q)
                    in = through(*(const float4 *)(window + q * kEntry + 16 * lane), in);
            }
        }
        if (failed) {  // the same in every warp
            if (threadIdx.x == 0) dev_fail(p.status, KDA_ERR_TIMEOUT);
            if (BY == BY_TMA && !BWD && landed) {  // the next tile's copies land before the block exits
                TileAt u;
                volatile int never = 0;
                if (turn(k + 1, u)) mbar_wait(smem_addr(&bars[warp]), (k + 1) & 1, &never, kWaitLimit);
            } else if (BY == BY_TMA && !landed) {  // or this one's
                volatile int never = 0;
                mbar_wait(smem_addr(&bars[warp]), k & 1, &never, kWaitLimit);
            }
            return;
        }
        if (warp == 0) {
            const bool closes = SPLIT && !t.last && t.place % kGroup == kGroup - 1;
            const float2 to = through(whole, closes ? group_in : in);
            if (closes) tell(p.ends + ((size_t)t.index * p.groups + t.group) * kChan + 2 * lane, to.x, to.y);
            if (!SPLIT) carry[(k & 1) ^ 1][lane] = to;
            if (t.last && final_out)
                store2<false>(final_out + (size_t)t.seq * p.C + c, left, pk(to.x, to.y));
        }

        if (BWD && SPLIT && threadIdx.x == 0) take(ahead_ticket, ahead);

        // this warp's tokens, from the state that enters them
        in = through(before, in);
        f2 s = pk(in.x, in.y);
        const int tok = t.t0 + warp * TOK, n = tokens(t);
        const bool starts = (BWD ? t.last : t.place == 0) && warp == 0;  // token 0 is the sequence's
        auto write = [&](auto all) {
#pragma unroll
            for (int i = 0; i < TOK; ++i) {
                const int j = BWD ? TOK - 1 - i : i;
                if (!all.value && j >= n) continue;
                const size_t row = (size_t)(tok + j) * p.C + c;
                if constexpr (!BWD) {
                    s = fma2(fa[j], s, fb[j]);
                    store2<PAIRS>((T *)p.h + row, left, s);
                } else {
                    f2 f, w, v = item(S::v, j), before = item(S::h, j);
                    decay2(gate(j), f, w);
                    if (j == 0 && starts)
                        before = p.h0 ? load2<false>(p.h0 + (size_t)t.seq * p.C + c, left) : pk(0.f, 0.f);
                    const f2 dh = add2(v, s);
                    s = mul2(f, dh);
                    if (MIX) before = fma2(item(S::x, j), both(-1.f), before);
                    store2<PAIRS>((T *)p.dx + row, left, MIX ? mul2(w, dh) : dh);
                    store2<PAIRS>(p.dg + row, left, mul2(s, before));
                }
            }
        };
        if (n == TOK) write(Yes{});
        else write(No{});
        if (BWD) {
            if (SPLIT) {
                if (threadIdx.x == 0) {
                    ticket_at[(k + 1) & 1] = ahead_ticket;
                    tile_at[(k + 1) & 1] = ahead;
                }
                __syncthreads();
            } else {
                __syncwarp();  // every lane has read this tile
            }
            start(k + 1);
        }
    }
}

// The tiles of every sequence, cleared maps and ends, the states of empty sequences, and, where
// the states are updated in place, a copy of those that chains start from: every tile of a
// chain's first group reads it, and the chain's last tile can be done before the others.
__global__ void __launch_bounds__(1024) recurrence_tiles_kernel(const __grid_constant__ RecArgs p,
                                                                bool backward, int tile, float *copy) {
    __shared__ int sums[32];
    __shared__ int base;
    __shared__ bool bad;
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (blockIdx.x > 0) {
        const long long me = (blockIdx.x - 1) * 1024ll + threadIdx.x, all = (gridDim.x - 1) * 1024ll;
        const long long pieces = (long long)p.most_tiles * p.groups * (kEntry / 16);
        uint4 *to = (uint4 *)p.maps;
        for (long long k = me; k < pieces; k += all) to[k] = make_uint4(kNone, kNone, kNone, kNone);
        const float *first = backward ? p.d_final : p.h0;
        float *final_out = backward ? p.d_h0 : p.h_final;
        if (copy)
            for (long long k = me; k < (long long)p.N * p.C; k += all) copy[k] = first[k];
        if (final_out && p.cu) {
            for (int n = blockIdx.x - 1; n < p.N; n += gridDim.x - 1) {
                if (p.cu[n] != p.cu[n + 1]) continue;
                for (int c = threadIdx.x; c < p.C; c += 1024)
                    final_out[(size_t)n * p.C + c] = first ? first[(size_t)n * p.C + c] : 0.f;
            }
        }
        return;
    }
    if (threadIdx.x == 0) {
        base = 0;
        bad = p.cu && (p.cu[0] != 0 || p.cu[p.N] != p.T);
    }
    __syncthreads();
    for (int n = threadIdx.x; n < p.N; n += 1024) {
        const int a = begin_of(p, n), b = end_of(p, n);
        if (a < 0 || b < a || b > p.T) bad = true;
    }
    __syncthreads();
    if (bad) {
        if (threadIdx.x == 0) {
            p.control[NEXT] = p.control[TILES] = p.control[ABORT] = 0;
            dev_fail(p.status, KDA_ERR_INVALID_ARG);
        }
        return;
    }
    auto entry = [&](int seq, int row, int first, int end, int place, int tiles) {
        return make_int4(row, first, (int)((unsigned)seq << 8) + min(tile, end - first) - 1,
                         2 * place + (place == tiles - 1));
    };
    if (p.N <= 32) {  // their tiles take turns, so that those that wait for each other are apart
        __shared__ int starts[33], counts[32];
        if (warp == 0) {
            const int count = lane < p.N ? (end_of(p, lane) - begin_of(p, lane) + tile - 1) / tile : 0;
            int v = count;
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += u;
            }
            counts[lane] = count;
            starts[lane + 1] = v;
            if (lane == 0) starts[0] = 0;
        }
        __syncthreads();
        for (int row = threadIdx.x; row < starts[32]; row += 1024) {
            int seq = 0;
            while (row >= starts[seq + 1]) ++seq;
            const int k = row - starts[seq], tiles = counts[seq], place = backward ? tiles - 1 - k : k;
            int turn = 0;
            for (int m = 0; m < p.N; ++m) turn += min(counts[m], place) + (m < seq && counts[m] > place);
            p.tiles[turn] = entry(seq, row, begin_of(p, seq) + k * tile, end_of(p, seq), place, tiles);
        }
        if (threadIdx.x == 0) {
            p.control[NEXT] = p.control[ABORT] = 0;
            p.control[TILES] = starts[32];
        }
        return;
    }
    for (int n0 = 0; n0 < p.N; n0 += 1024) {
        const int n = n0 + threadIdx.x;
        const int a = n < p.N ? begin_of(p, n) : 0, b = n < p.N ? end_of(p, n) : 0;
        const int count = (b - a + tile - 1) / tile;
        int v = count;
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        if (lane == 31) sums[warp] = v;
        __syncthreads();
        if (warp == 0) {
            int s = sums[lane];
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s += u;
            }
            sums[lane] = s;
        }
        __syncthreads();
        const int at = base + v - count + (warp ? sums[warp - 1] : 0);
        // a warp's sequences one after another, their tiles by its lanes
        for (int q = 0; q < 32; ++q) {
            const int tiles = __shfl_sync(0xffffffffu, count, q), to = __shfl_sync(0xffffffffu, at, q);
            const int from = __shfl_sync(0xffffffffu, a, q), end = __shfl_sync(0xffffffffu, b, q);
            for (int k = lane; k < tiles; k += 32) {
                const int place = backward ? tiles - 1 - k : k;
                p.tiles[to + place] = entry(n0 + 32 * warp + q, to + k, from + k * tile, end, place, tiles);
            }
        }
        __syncthreads();
        if (threadIdx.x == 0) base += sums[31];
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        p.control[NEXT] = p.control[ABORT] = 0;
        p.control[TILES] = base;
    }
}

// One token of every sequence: VEC channels of one of them per thread.
template <typename T, bool MIX, int VEC>
__global__ void __launch_bounds__(256)
    recurrence_step_kernel(const T *x, const float *g, const float *state, float *state_out, T *h,
                           long long x_stride, long long g_stride, int N, int C) {
    griddep_wait();
    griddep_launch_dependents();
    const int pieces = (C + VEC - 1) / VEC;
    const long long total = (long long)N * pieces;
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
        const long long n = i / pieces;
        const int c = (int)(i - n * pieces) * VEC;
        const long long at = n * C + c;
        float gv[VEC], sv[VEC], xv[VEC];
        if constexpr (VEC == 4) {
            *(float4 *)gv = *(const float4 *)(g + n * g_stride + c);
            *(float4 *)sv = *(const float4 *)(state + at);
            if constexpr (sizeof(T) == 4) {
                *(float4 *)xv = *(const float4 *)(x + n * x_stride + c);
            } else {
                const uint2 u = *(const uint2 *)(x + n * x_stride + c);
                xv[0] = __uint_as_float(u.x << 16);
                xv[1] = __uint_as_float(u.x & 0xffff0000u);
                xv[2] = __uint_as_float(u.y << 16);
                xv[3] = __uint_as_float(u.y & 0xffff0000u);
            }
        } else {
            gv[0] = g[n * g_stride + c];
            sv[0] = state[at];
            xv[0] = act_ld(x, (size_t)(n * x_stride + c));
        }
#pragma unroll
        for (int j = 0; j < VEC; j += 2) {
            f2 a, w;
            decay2(pk(gv[j], VEC > 1 ? gv[(j + 1) % VEC] : 0.f), a, w);
            f2 v = pk(xv[j], VEC > 1 ? xv[(j + 1) % VEC] : 0.f);
            if (MIX) v = mul2(w, v);
            const float2 to = un(fma2(a, pk(sv[j], VEC > 1 ? sv[(j + 1) % VEC] : 0.f), v));
            sv[j] = to.x;
            if (VEC > 1) sv[(j + 1) % VEC] = to.y;
        }
        if constexpr (VEC == 4) {
            *(float4 *)(state_out + at) = *(const float4 *)sv;
            if constexpr (sizeof(T) == 4)
                *(float4 *)(h + at) = *(const float4 *)sv;
            else
                *(uint2 *)(h + at) = make_uint2(pack_bf16x2(sv[0], sv[1]), pack_bf16x2(sv[2], sv[3]));
        } else {
            state_out[at] = sv[0];
            act_st(h, (size_t)at, sv[0]);
        }
    }
}

// ------------------------------------------------------------------ host side
size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }
bool walks(const kda_recurrence_desc_t *d) { return d->tokens <= kWalkTokens; }
long long most_tiles(long long tokens, long long seqs, int tile) {
    const long long n = tokens / tile + seqs;
    return n < tokens ? n : tokens;
}
// of any kernel that a call could take
long long most_tiles(const kda_recurrence_desc_t *d, bool bwd) {
    return most_tiles(d->tokens, d->num_seqs, tile_of(bwd, false));
}
int groups_of(const kda_recurrence_desc_t *d) { return (d->channels + kChan - 1) / kChan; }

struct Layout {
    size_t tiles, maps, total;
};
Layout layout_for(const kda_recurrence_desc_t *d, bool bwd) {
    Layout l = {};
    if (walks(d)) return l;
    const size_t n = (size_t)most_tiles(d, bwd), g = groups_of(d);
    l.tiles = round256(n * sizeof(int4));
    l.maps = n * g * kEntry;
    l.total = 256 + l.tiles + l.maps + round256((size_t)d->num_seqs * d->channels * sizeof(float));
    return l;
}

kda_status_t check(const kda_recurrence_desc_t *d) {
    if (!d) return KDA_ERR_INVALID_ARG;
    if (d->num_seqs < 1 || d->tokens < 0 || d->channels < 1) return KDA_ERR_INVALID_ARG;
    if ((d->x_stride != 0 && d->x_stride < d->channels) ||
        (d->g_stride != 0 && d->g_stride < d->channels))
        return KDA_ERR_INVALID_ARG;
    if (d->act_dtype != KDA_DTYPE_F32 && d->act_dtype != KDA_DTYPE_BF16) return KDA_ERR_UNSUPPORTED;
    if (d->write != KDA_WRITE_ADD && d->write != KDA_WRITE_MIX) return KDA_ERR_UNSUPPORTED;
    if (d->tokens > (1 << 30) || d->num_seqs > (1 << 24) || d->channels > (1 << 20))
        return KDA_ERR_UNSUPPORTED;
    if (d->x_stride > (1ll << 30) || d->g_stride > (1ll << 30)) return KDA_ERR_UNSUPPORTED;
    // tiles are numbered, and blocks counted, in 31 bits (and every block takes one more)
    if (most_tiles(d, true) * groups_of(d) > (1ll << 30) ||
        (long long)d->num_seqs * groups_of(d) > (1ll << 30))
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

RecArgs make_args(const kda_recurrence_desc_t *d) {
    RecArgs a = {};
    a.N = d->num_seqs;
    a.T = d->tokens;
    a.C = d->channels;
    a.groups = groups_of(d);
    a.x_stride = d->x_stride ? d->x_stride : d->channels;
    a.g_stride = d->g_stride ? d->g_stride : d->channels;
    return a;
}

// Copies of 64 channels of a warp's tokens from an array whose tokens are `stride` elements
// apart; false where a tensor map cannot read it.
bool encode(CUtensorMap *m, const void *base, int size, int C, int T, long long stride, int tok) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc || C < kChan || ((uintptr_t)base & 15u) || stride * size % 16) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)C, (cuuint64_t)T}, strides[1] = {(cuuint64_t)(stride * size)};
    const cuuint32_t box[2] = {kChan, (cuuint32_t)tok}, one[2] = {1, 1};
    return enc(m, size == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
               const_cast<void *>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxSmem = 180 * 1024;  // a stage of 128 KB, two windows of 24 entries


template <typename T, bool BWD, bool MIX, int BY, bool SPLIT>
cudaError_t launch_by(RecArgs &a, float *copy, const CUtensorMap (&m)[4], cudaStream_t st) {
    const auto kernel = recurrence_kernel<T, BWD, MIX, BY, SPLIT>;
    typedef Stage<T, BWD, MIX, BY == BY_TMA> S;
    const int sms = device_sms();
    long long blocks = (long long)a.N * a.groups;
    int smem = S::block + 128;
    if (SPLIT) {
        a.most_tiles = (int)most_tiles(a.T, a.N, S::warps * S::tok);
        const long long work = (long long)a.most_tiles * a.groups, pieces = work * (kEntry / 16);
        a.ends = (float *)(a.maps + work * kChan);
        const int clear = (int)(pieces / 4096 < 2 * sms ? pieces / 4096 : 2 * sms) + 1;
        const float *&first = BWD ? a.d_final : a.h0;
        if (first != (BWD ? a.d_h0 : a.h_final)) copy = nullptr;
        const cudaError_t e = launch_dependent(recurrence_tiles_kernel, dim3(1 + clear), dim3(1024), 0,
                                               st, a, BWD, S::warps * S::tok, first ? copy : nullptr);
        if (e != cudaSuccess) return e;
        if (first && copy) first = copy;
        // A look back reads a few more groups than are worked on at once in a chain.
        const int chain = S::fit(kUsualWindow) * sms / (a.groups * kGroup);
        a.window = chain + 3 < 16 ? chain + 3 : 16;
        const int entries = a.window + kGroup - 1;
        smem += (BWD ? 1 : 2) * entries * kEntry;
        const long long most = (long long)S::fit(entries) * sms;
        blocks = work < most ? work : most;
    }
    const cudaError_t e = set_max_dynamic_smem((const void *)kernel, kMaxSmem);
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, dim3((unsigned)blocks), dim3(32 * S::warps), smem, st, a, m[0], m[1],
                            m[2], m[3]);
}

template <typename T, bool BWD, bool MIX>
cudaError_t launch_t(const kda_recurrence_desc_t *d, RecArgs &a, bool pairs, void *workspace,
                     cudaStream_t st) {
    CUtensorMap m[4] = {};
    if (walks(d))
        return pairs ? launch_by<T, BWD, MIX, BY_PAIRS, false>(a, nullptr, m, st)
                     : launch_by<T, BWD, MIX, BY_ONE, false>(a, nullptr, m, st);
    const Layout l = layout_for(d, BWD);
    uint8_t *ws = (uint8_t *)workspace;
    a.control = (unsigned *)ws;
    a.tiles = (int4 *)(ws + 256);
    a.maps = (float2 *)(ws + 256 + l.tiles);
    float *copy = (float *)(ws + 256 + l.tiles + l.maps);
    constexpr int tok = tok_of(BWD, true), size = sizeof(T);
    const bool tma =
        encode(&m[0], a.g, 4, a.C, a.T, a.g_stride, tok) &&
        (BWD ? encode(&m[1], a.d, size, a.C, a.T, a.C, tok) && encode(&m[2], a.hs, size, a.C, a.T, a.C, tok) &&
                   (!MIX || encode(&m[3], a.x, size, a.C, a.T, a.x_stride, tok))
             : encode(&m[1], a.x, size, a.C, a.T, a.x_stride, tok));
    if (tma && pairs) return launch_by<T, BWD, MIX, BY_TMA, true>(a, copy, m, st);
    return pairs ? launch_by<T, BWD, MIX, BY_PAIRS, true>(a, copy, m, st)
                 : launch_by<T, BWD, MIX, BY_ONE, true>(a, copy, m, st);
}

template <bool BWD>
kda_status_t launch(const kda_recurrence_desc_t *d, RecArgs &a, bool pairs, void *workspace,
                    cudaStream_t st) {
    const bool mix = d->write == KDA_WRITE_MIX;
    typedef __nv_bfloat16 B;
    const cudaError_t e =
        d->act_dtype == KDA_DTYPE_F32
            ? (mix ? launch_t<float, BWD, true>(d, a, pairs, workspace, st)
                   : launch_t<float, BWD, false>(d, a, pairs, workspace, st))
            : (mix ? launch_t<B, BWD, true>(d, a, pairs, workspace, st)
                   : launch_t<B, BWD, false>(d, a, pairs, workspace, st));
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

int size_of(const kda_recurrence_desc_t *d) { return d->act_dtype == KDA_DTYPE_BF16 ? 2 : 4; }
bool off(const void *p, int size) { return ((uintptr_t)p & (size - 1)) != 0; }
bool bad_ws(const kda_recurrence_desc_t *d, bool bwd, const void *ws, size_t bytes) {
    const size_t need = layout_for(d, bwd).total;
    return need > 0 && (!ws || bytes < need || off(ws, 16));
}

kda_status_t forward(const kda_recurrence_desc_t *desc, const void *x, const float *g, const float *h0,
                     const int32_t *cu_seqlens, void *h, float *h_final, void *workspace,
                     size_t workspace_bytes, int32_t *dev_status, long long wait_limit, void *stream) {
    const kda_status_t rc = check(desc);
    if (rc != KDA_OK) return rc;
    const int size = size_of(desc);
    if ((desc->tokens > 0 && (!x || !g || !h)) || (!cu_seqlens && desc->num_seqs != 1))
        return KDA_ERR_INVALID_ARG;
    if (off(x, size) || off(h, size) || off(g, 4) || off(h0, 4) || off(h_final, 4) ||
        off(cu_seqlens, 4) || off(dev_status, 4))
        return KDA_ERR_INVALID_ARG;
    if (bad_ws(desc, false, workspace, workspace_bytes)) return KDA_ERR_WORKSPACE;
    RecArgs a = make_args(desc);
    a.x = x; a.g = g; a.h0 = h0; a.cu = cu_seqlens; a.h = h; a.h_final = h_final;
    a.status = dev_status;
    a.wait_limit = wait_limit;
    const bool pairs = desc->channels % 2 == 0 && a.x_stride % 2 == 0 && a.g_stride % 2 == 0 &&
                     !off(x, 2 * size) && !off(h, 2 * size) && !off(g, 8);
    return launch<false>(desc, a, pairs, workspace, (cudaStream_t)stream);
}

kda_status_t backward(const kda_recurrence_desc_t *desc, const void *d_h, const void *x,
                      const float *g, const void *h, const float *h0, const int32_t *cu_seqlens,
                      const float *d_h_final, void *dx, float *dg, float *d_h0, void *workspace,
                      size_t workspace_bytes, int32_t *dev_status, long long wait_limit, void *stream) {
    const kda_status_t rc = check(desc);
    if (rc != KDA_OK) return rc;
    const int size = size_of(desc);
    const bool mix = desc->write == KDA_WRITE_MIX;
    if ((desc->tokens > 0 && (!d_h || !g || !h || !dx || !dg || (mix && !x))) ||
        (!cu_seqlens && desc->num_seqs != 1))
        return KDA_ERR_INVALID_ARG;
    if (off(d_h, size) || off(x, size) || off(h, size) || off(dx, size) || off(g, 4) || off(dg, 4) ||
        off(h0, 4) || off(d_h_final, 4) || off(d_h0, 4) || off(cu_seqlens, 4) || off(dev_status, 4))
        return KDA_ERR_INVALID_ARG;
    if (bad_ws(desc, true, workspace, workspace_bytes)) return KDA_ERR_WORKSPACE;
    RecArgs a = make_args(desc);
    a.x = x; a.g = g; a.h0 = h0; a.cu = cu_seqlens; a.d = d_h; a.hs = h; a.d_final = d_h_final;
    a.dx = dx; a.dg = dg; a.d_h0 = d_h0;
    a.status = dev_status;
    a.wait_limit = wait_limit;
    const bool pairs = desc->channels % 2 == 0 && a.g_stride % 2 == 0 && !off(d_h, 2 * size) &&
                     !off(h, 2 * size) && !off(dx, 2 * size) && !off(g, 8) && !off(dg, 8) &&
                     (!mix || (a.x_stride % 2 == 0 && !off(x, 2 * size)));
    return launch<true>(desc, a, pairs, workspace, (cudaStream_t)stream);
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

size_t kda_recurrence_workspace_size(const kda_recurrence_desc_t *desc, int32_t backward) {
    return check(desc) == KDA_OK ? layout_for(desc, backward != 0).total : 0;
}

kda_status_t kda_recurrence_forward(const kda_recurrence_desc_t *desc, const void *x, const float *g,
                                    const float *h0, const int32_t *cu_seqlens, void *h,
                                    float *h_final, void *workspace, size_t workspace_bytes,
                                    int32_t *dev_status, void *stream) {
    return forward(desc, x, g, h0, cu_seqlens, h, h_final, workspace, workspace_bytes, dev_status,
                   kWaitLimit, stream);
}

kda_status_t kda_recurrence_backward(const kda_recurrence_desc_t *desc, const void *d_h,
                                     const void *x, const float *g, const void *h, const float *h0,
                                     const int32_t *cu_seqlens, const float *d_h_final, void *dx,
                                     float *dg, float *d_h0, void *workspace, size_t workspace_bytes,
                                     int32_t *dev_status, void *stream) {
    return backward(desc, d_h, x, g, h, h0, cu_seqlens, d_h_final, dx, dg, d_h0, workspace,
                    workspace_bytes, dev_status, kWaitLimit, stream);
}

kda_status_t kda_selftest_recurrence_timeout(const kda_recurrence_desc_t *desc, const void *x,
                                             const float *g, const void *h, void *out, float *dg,
                                             void *workspace, size_t workspace_bytes,
                                             int32_t *dev_status, void *stream) {
    if (!dev_status || !desc || desc->write != KDA_WRITE_ADD) return KDA_ERR_INVALID_ARG;
    return h ? backward(desc, x, nullptr, g, h, nullptr, nullptr, nullptr, out, dg, nullptr, workspace,
                        workspace_bytes, dev_status, 0, stream)
             : forward(desc, x, g, nullptr, nullptr, out, nullptr, workspace, workspace_bytes,
                       dev_status, 0, stream);
}

kda_status_t kda_recurrence_step(const kda_recurrence_desc_t *desc, const void *x, const float *g,
                                 const float *state, float *state_out, void *h, void *stream) {
    const kda_status_t rc = check(desc);
    if (rc != KDA_OK) return rc;
    const int size = size_of(desc);
    if (desc->tokens != desc->num_seqs || !x || !g || !state || !state_out || !h)
        return KDA_ERR_INVALID_ARG;
    if (off(x, size) || off(h, size) || off(g, 4) || off(state, 4) || off(state_out, 4))
        return KDA_ERR_INVALID_ARG;
    const RecArgs a = make_args(desc);
    const bool vec = a.C % 4 == 0 && a.x_stride % 4 == 0 && a.g_stride % 4 == 0 && !off(x, 4 * size) &&
                     !off(h, 4 * size) && !off(g, 16) && !off(state, 16) && !off(state_out, 16);
    const long long n = (long long)a.N * (vec ? a.C / 4 : a.C), need = (n + 255) / 256;
    const long long most = 64ll * device_sms();
    const dim3 grid((unsigned)(need < most ? need : most));
    const bool mix = desc->write == KDA_WRITE_MIX;
    auto run = [&](auto kernel, auto zero) {
        typedef decltype(zero) T;
        return launch_dependent(kernel, grid, dim3(256), 0, (cudaStream_t)stream, (const T *)x, g,
                                state, state_out, (T *)h, a.x_stride, a.g_stride, a.N, a.C);
    };
    cudaError_t e;
    if (size == 4)
        e = vec ? (mix ? run(recurrence_step_kernel<float, true, 4>, 0.f)
                       : run(recurrence_step_kernel<float, false, 4>, 0.f))
                : (mix ? run(recurrence_step_kernel<float, true, 1>, 0.f)
                       : run(recurrence_step_kernel<float, false, 1>, 0.f));
    else
        e = vec ? (mix ? run(recurrence_step_kernel<__nv_bfloat16, true, 4>, __nv_bfloat16())
                       : run(recurrence_step_kernel<__nv_bfloat16, false, 4>, __nv_bfloat16()))
                : (mix ? run(recurrence_step_kernel<__nv_bfloat16, true, 1>, __nv_bfloat16())
                       : run(recurrence_step_kernel<__nv_bfloat16, false, 1>, __nv_bfloat16()));
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
