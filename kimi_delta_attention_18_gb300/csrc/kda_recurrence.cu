// The gated linear recurrence: every channel c of a packed batch has a state of its own,
//     h_t = e^{g_t} h_{t-1} + w_t x_t,   w = 1 (add) or 1 - e^{g_t} (mix),
// from h0 at the start of its sequence.  Backward, from the last token to the first, with
// u_t = e^{g_t} dh_t the adjoint that a step hands to the one before it:
//     dh_t = d_t + u_{t+1},   dx_t = w_t dh_t,   dg_t = u_t (h_{t-1} [- x_t]),   dh0 = u_first.
//
// Both are scans of maps s -> A s + B (A the product of the factors e^g, B the result from a
// zero start), which compose: a tile of some tokens x 64 channels is one map per channel.
// Every element should be read and written once, so the scan takes one pass: the four warps of
// a block each run a quarter of a tile's tokens (a lane has two channels) and join their maps;
// the block publishes the tile's map, looks back along the sequence for the nearest tile whose
// end state is known, carries that state through the maps in between, publishes its own end
// state and writes its tokens.  Tiles are handed out in order by a counter, so a tile that is
// waited for is already being worked on.  A state always goes through one tile's map at a time
// and in order, whoever computes it, so the results do not depend on where a look back ended.
//
// The look back's latency is what the pass must hide: without it 81,920 x 7,168 BF16 (mix)
// takes 0.65 ms, the time of its bytes.  So maps and ends are words that a NaN of their own
// marks as absent (no flag beside the data, no fence between the two, one trip to L2 for both),
// a look back reads its whole window at once, and a block has the next tile's tokens on their
// way (TMA) while it works; with flags, and the maps read four at a time, it took 1.62 ms.
// Tiles by 16 warps with loads straight into registers, two such blocks to an SM, took 2.38.
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

constexpr int kWarps = 4, kChan = 64, kThreads = 32 * kWarps;
// Tokens of a warp in a tile: the forward pass holds them in registers, the backward pass
// reads them from shared memory twice.
constexpr int tok_of(bool bwd) { return bwd ? 16 : 32; }
constexpr long long kWaitLimit = 4000000000ll;  // ~2 s of SM clocks
// Up to so many tokens one block walks a sequence; beyond, a launch lays out the tiles of a
// batch first.
constexpr int kWalkTokens = 512;

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
    int4 *tiles;         // [tiles] sequence, first token, end, 2 (place in the chain) + last
    float2 *maps;        // [tiles][64 groups]
    float *ends;         // [tiles][64 groups], behind maps
    unsigned *control;   // next tile, tiles, a wait gave up
    int most_tiles, window;  // window: tiles that a look back reads
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
// (its own is 0x7fffffff; were this one ever to come up, that is stored instead).
constexpr uint32_t kNone = 0xffffffffu;
__device__ __forceinline__ bool there(float v) { return __float_as_uint(v) != kNone; }
__device__ __forceinline__ float told(float v) { return there(v) ? v : __uint_as_float(0x7fffffffu); }
__device__ __forceinline__ void tell(void *p, float a, float b) {  // two words at once
    asm volatile("st.relaxed.gpu.b64 [%0], %1;" ::"l"(p), "l"(pk(told(a), told(b))) : "memory");
}

struct TileAt {
    int seq, t0, t1, place, group;
    bool last;
};

// A tile's entry in a look back's window: maps of 64 channels, then their ends.
constexpr int kEntry = kChan * 12;

// The state that enters the tile in this lane's two channels from the window's `n` entries,
// nearest first; false if it does not reach an end yet.
__device__ __forceinline__ bool look_back(const uint8_t *window, int n, int lane, float2 &state) {
    int q = 0;
    bool found = false;
    for (; q < n; ++q) {
        const float2 e = *(const float2 *)(window + q * kEntry + kChan * 8 + 8 * lane);
        if (there(e.x) && there(e.y)) {
            state = e;
            found = true;
            break;
        }
        const float4 m = *(const float4 *)(window + q * kEntry + 16 * lane);
        if (!there(m.x) || !there(m.z)) break;
    }
    if (!__all_sync(0xffffffffu, found)) return false;
    for (--q; q >= 0; --q) state = through(*(const float4 *)(window + q * kEntry + 16 * lane), state);
    return true;
}

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

template <typename T, bool BWD, bool MIX>
struct Stage {  // a warp's part of a tile in shared memory
    static constexpr int tok = tok_of(BWD);
    static constexpr int g = 0, v = tok * kChan * 4, one = tok * kChan * (int)sizeof(T);
    static constexpr int h = v + one, x = h + (BWD ? one : 0), bytes = x + (BWD && MIX ? one : 0);
    static constexpr int block = kWarps * bytes;
    // blocks to an SM: by registers (the forward pass holds a tile) or shared memory
    static constexpr int most = BWD ? 5 : 3;
    static constexpr int fit(int window) {
        const int n = 227 * 1024 / (block + window * kEntry + 7 * 1024);
        return n < 1 ? 1 : n < most ? n : most;
    }
};

template <typename T, bool BWD, bool MIX, int BY, bool SPLIT>
__global__ void __launch_bounds__(kThreads, Stage<T, BWD, MIX>::fit(4))
    recurrence_kernel(const __grid_constant__ RecArgs p, const __grid_constant__ CUtensorMap tm_g,
                      const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ CUtensorMap tm_h,
                      const __grid_constant__ CUtensorMap tm_x) {
    using S = Stage<T, BWD, MIX>;
    constexpr int TOK = S::tok, kTile = TOK * kWarps;
    constexpr bool PAIRS = BY != BY_ONE;
    extern __shared__ __align__(128) uint8_t sm_raw[];
    __shared__ float4 maps[2][kWarps][32];  // (A, B) of two channels
    __shared__ float2 carry[2][32];  // without a look back
    __shared__ int4 next_tile[2];
    __shared__ int next_ticket[2];
    __shared__ __align__(8) uint64_t bars[kWarps];
    __shared__ int abort_flag;
    __shared__ bool failed;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const T *x = (const T *)p.x, *d = (const T *)p.d, *hs = (const T *)p.hs;
    const float *first = BWD ? p.d_final : p.h0;
    float *final_out = BWD ? p.d_h0 : p.h_final;
    const uint32_t bar = smem_addr(&bars[warp]);
    uint8_t *sm = sm_raw + ((128u - (smem_addr(sm_raw) & 127u)) & 127u);
    uint8_t *window = sm + S::block;
    if (threadIdx.x == 0) {
        abort_flag = 0;
        failed = false;
        if (BY == BY_TMA) {
            for (int w = 0; w < kWarps; ++w) mbar_init(smem_addr(&bars[w]), 1);
            mbar_fence_init();
        }
    }
    griddep_wait();
    griddep_launch_dependents();

    TileAt t = {};
    int total = 0, begin = 0, end = 0;
    auto take = [&](int &ticket, int4 &tile) {  // one thread
        ticket = (int)atomicAdd(p.control + NEXT, 1u);
        const int k = ticket / p.groups;
        tile = make_int4(0, 0, 0, 0);
        if (k < total) tile = p.tiles[BWD ? total - 1 - k : k];
    };
    if (SPLIT) {
        total = (int)p.control[TILES];
        if (threadIdx.x == 0) take(next_ticket[0], next_tile[0]);
    } else {
        t.seq = blockIdx.x / p.groups;
        t.group = blockIdx.x - t.seq * p.groups;
        begin = begin_of(p, t.seq);
        end = end_of(p, t.seq);
        const bool good = !p.cu || (begin >= 0 && begin <= end && end <= p.T && p.cu[0] == 0 &&
                                    p.cu[p.N] == p.T);
        if (!good) {
            if (threadIdx.x == 0) dev_fail(p.status, KDA_ERR_INVALID_ARG);
            return;
        }
        if (warp == 0) {
            const int c = t.group * kChan + 2 * lane;
            const f2 s = first ? load2<false>(first + (size_t)t.seq * p.C + c, p.C - c) : pk(0.f, 0.f);
            carry[0][lane] = un(s);
            if (begin == end && final_out)
                store2<false>(final_out + (size_t)t.seq * p.C + c, p.C - c, s);
        }
    }
    __syncthreads();

    // this warp's copies of the tile of tokens t0 .. t1 - 1
    const uint32_t stage = smem_addr(sm) + warp * S::bytes;
    auto copy = [&](int t0, int t1, int group) {
        const int y = t0 + warp * TOK;
        if constexpr (BY == BY_TMA) {
            if (lane != 0) return;
            const int c = group * kChan;
            mbar_arrive_expect_tx(bar, S::bytes);
            tma_load_2d(stage + S::g, reinterpret_cast<uint64_t>(&tm_g), c, y, bar);
            tma_load_2d(stage + S::v, reinterpret_cast<uint64_t>(&tm_v), c, y, bar);
            if (BWD) tma_load_2d(stage + S::h, reinterpret_cast<uint64_t>(&tm_h), c, y - 1, bar);
            if (BWD && MIX) tma_load_2d(stage + S::x, reinterpret_cast<uint64_t>(&tm_x), c, y, bar);
        } else {
            const int c = group * kChan + 2 * lane, left = p.C - c;
            const uint32_t to = stage + 8 * lane, to_t = stage + 2 * (int)sizeof(T) * lane;
#pragma unroll 8
            for (int j = 0; j < TOK; ++j) {
                const int n = y + j < t1 ? left : 0;
                const size_t row = (size_t)(y + j), at = row * p.C + c;
                constexpr int step = kChan * (int)sizeof(T);
                fetch<PAIRS>(to + S::g + j * kChan * 4, p.g + row * p.g_stride + c, p.g, n);
                fetch<PAIRS>(to_t + S::v + j * step, BWD ? d + at : x + row * p.x_stride + c, p.g, n);
                if (BWD) fetch<PAIRS>(to_t + S::h + j * step, hs + at - p.C, p.g, y + j > 0 ? n : 0);
                if (BWD && MIX)
                    fetch<PAIRS>(to_t + S::x + j * step, x + row * p.x_stride + c, p.g, n);
            }
        }
    };
    const uint8_t *mine = sm + warp * S::bytes + 8 * lane;  // of g
    const uint8_t *mine_t = sm + warp * S::bytes + 2 * sizeof(T) * lane;
    bool pending = false;  // this warp's copies are on their way
    auto tile_of_walk = [&](int walk) {  // without a look back
        const int n = (end - begin + kTile - 1) / kTile;
        const int t0 = begin + (BWD ? n - 1 - walk : walk) * kTile;
        return make_int4(t.seq, t0, min(t0 + kTile, end), walk >= n ? -1 : 2 * walk + (walk == n - 1));
    };
    auto start = [&](int walk) {  // of the tile after the next barrier, or the first
        if (SPLIT) {
            const int ticket = next_ticket[walk & 1], k = ticket / p.groups;
            const int4 tile = next_tile[walk & 1];
            pending = k < total;
            if (pending) copy(tile.y, tile.z, ticket - k * p.groups);
        } else {
            const int4 tile = tile_of_walk(walk);
            pending = tile.w >= 0;
            if (pending) copy(tile.y, tile.z, t.group);
        }
    };
    start(0);

    for (int walk = 0;; ++walk) {
        const int par = walk & 1;
        int index = 0, ahead_ticket = 0;
        int4 tile, ahead;
        if (SPLIT) {
            const int ticket = next_ticket[par], k = ticket / p.groups;
            if (k >= total) return;
            tile = next_tile[par];
            index = BWD ? total - 1 - k : k;
            t.group = ticket - k * p.groups;
            if (threadIdx.x == 0) take(ahead_ticket, ahead);
        } else {
            tile = tile_of_walk(walk);
            if (tile.w < 0) return;
        }
        t.seq = tile.x;
        t.t0 = tile.y;
        t.t1 = tile.z;
        t.place = tile.w >> 1;
        t.last = tile.w & 1;
        const int c = t.group * kChan + 2 * lane, left = p.C - c;
        const int tok = t.t0 + warp * TOK;  // this warp's first token
        const int n = max(0, min(TOK, t.t1 - tok));
        const bool starts = BWD ? t.last : t.place == 0;  // the tile has the sequence's first token
        bool landed = true;
        if (BY == BY_TMA) {
            landed = __all_sync(0xffffffffu, mbar_wait(bar, par, &abort_flag, kWaitLimit));
            if (!landed) failed = true;
        } else {
            cp_async_wait_all();  // every lane reads what it copied itself
        }
        pending = !landed;
        auto gate = [&](int j) { return get2((const float *)(mine + S::g + j * kChan * 4)); };
        auto item = [&](int array, int j) {
            return get2((const T *)(mine_t + array + j * kChan * sizeof(T)));
        };

        // the map of this warp's tokens
        f2 a[BWD ? 1 : TOK], b[BWD ? 1 : TOK];  // forward: factors and terms
        f2 A = both(1.f), B = both(0.f);
        auto run = [&](auto whole) {
#pragma unroll
            for (int i = 0; i < TOK; ++i) {
                const int j = BWD ? TOK - 1 - i : i;
                f2 f = both(1.f), w, v = both(0.f);
                if (whole.value || j < n) {
                    decay2(gate(j), f, w);
                    v = item(S::v, j);  // x, or backward d
                    if (!BWD && MIX) v = mul2(w, v);
                }
                if (BWD) {
                    B = mul2(f, add2(B, v));
                } else {
                    a[BWD ? 0 : j] = f;
                    b[BWD ? 0 : j] = v;
                    B = fma2(f, B, v);
                }
                A = mul2(A, f);
            }
        };
        if (n == TOK) run(Yes{});
        else run(No{});
        const float2 ua = un(A), ub = un(B);
        maps[par][warp][lane] = make_float4(ua.x, ub.x, ua.y, ub.y);
        if (SPLIT && threadIdx.x == 0) {
            next_ticket[par ^ 1] = ahead_ticket;
            next_tile[par ^ 1] = ahead;
        }
        __syncthreads();
        if (!BWD && landed) start(walk + 1);  // this tile is in registers

        // the tile's map, published by one warp
        float4 m = make_float4(1.f, 0.f, 1.f, 0.f);
        const size_t slot = (size_t)index * p.groups * kChan + c;
        if (warp == 0) {
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                const float4 v = maps[par][BWD ? kWarps - 1 - i : i][lane];
                const float2 to = through(v, make_float2(m.y, m.w));
                m = make_float4(m.x * v.x, to.x, m.z * v.z, to.y);
            }
            if (SPLIT && t.place > 0 && !t.last) {
                tell(p.maps + slot, m.x, m.y);
                tell(p.maps + slot + 1, m.z, m.w);
            }
        }
        // the state that enters the tile, in every warp
        float2 in;
        if (!SPLIT) {
            in = carry[par][lane];
        } else if (t.place == 0) {
            in = un(first ? load2<false>(first + (size_t)t.seq * p.C + c, left) : pk(0.f, 0.f));
        } else {
            const int n = min(p.window, t.place), step = BWD ? 1 : -1;
            const size_t pitch = (size_t)p.groups * kChan;
            const long long since = clock64();
            while (true) {
                for (int k = threadIdx.x; k < n * (kEntry / 16); k += kThreads) {
                    const int q = k / (kEntry / 16), part = k - q * (kEntry / 16);
                    const size_t at = (size_t)(index + step * (q + 1)) * pitch + t.group * kChan;
                    cp_async16(smem_addr(window) + 16 * k,
                               part < kChan / 2 ? (const void *)(p.maps + at + 2 * part)
                                                : (const void *)(p.ends + at + 4 * (part - kChan / 2)),
                               true);
                }
                cp_async_wait_all();
                __syncthreads();
                if (failed || look_back(window, n, lane, in)) break;  // the same in every warp
                __syncthreads();
                if (threadIdx.x == 0 && (clock64() - since > kWaitLimit ||
                                         *(volatile unsigned *)(p.control + ABORT))) {
                    *(volatile unsigned *)(p.control + ABORT) = 1;
                    failed = true;
                }
            }
        }
        if (failed) {  // (set before a barrier that everyone has passed)
            if (threadIdx.x == 0) dev_fail(p.status, KDA_ERR_TIMEOUT);
            if (BY == BY_TMA && pending) {  // let the copies land before the block exits
                volatile int never = 0;
                mbar_wait(bar, landed ? par ^ 1 : par, &never, kWaitLimit);
            }
            return;
        }
        if (warp == 0) {
            const float2 to = through(m, in);
            if (SPLIT && !t.last) tell(p.ends + slot, to.x, to.y);
            if (!SPLIT) carry[par ^ 1][lane] = to;
            if (t.last && final_out)
                store2<false>(final_out + (size_t)t.seq * p.C + c, left, pk(to.x, to.y));
        }

        // this warp's tokens, from the state that enters them
        for (int w = BWD ? kWarps - 1 : 0; w != warp; w += BWD ? -1 : 1)
            in = through(maps[par][w][lane], in);
        f2 s = pk(in.x, in.y);
        auto write = [&](auto whole) {
            if constexpr (!BWD) {
                T *to = (T *)p.h + (size_t)tok * p.C + c;
#pragma unroll
                for (int j = 0; j < TOK; ++j) {
                    s = fma2(a[j], s, b[j]);
                    if (whole.value || j < n) store2<PAIRS>(to, left, s);
                    to += p.C;
                }
            } else {
#pragma unroll
                for (int i = 0; i < TOK; ++i) {
                    const int j = TOK - 1 - i;
                    if (!whole.value && j >= n) continue;
                    const size_t row = (size_t)(tok + j) * p.C + c;
                    f2 f, w, before;
                    decay2(gate(j), f, w);
                    if (j == 0 && warp == 0 && starts)
                        before = p.h0 ? load2<false>(p.h0 + (size_t)t.seq * p.C + c, left) : pk(0.f, 0.f);
                    else
                        before = item(S::h, j);
                    const f2 dh = add2(item(S::v, j), s);
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
            __syncwarp();  // every lane has read this tile
            start(walk + 1);
        }
    }
}

// The tiles of every sequence, cleared maps and ends, and the states of empty sequences.
__global__ void __launch_bounds__(1024) recurrence_tiles_kernel(const __grid_constant__ RecArgs p,
                                                                bool backward) {
    const int kTile = kWarps * tok_of(backward);
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
    for (int n0 = 0; n0 < p.N; n0 += 1024) {
        const int n = n0 + threadIdx.x;
        const int a = n < p.N ? begin_of(p, n) : 0, b = n < p.N ? end_of(p, n) : 0;
        const int count = (b - a + kTile - 1) / kTile;
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
                p.tiles[to + k] = make_int4(n0 + 32 * warp + q, from + k * kTile,
                                            min(from + (k + 1) * kTile, end),
                                            2 * place + (place == tiles - 1));
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
long long most_tiles(const kda_recurrence_desc_t *d, bool bwd) {
    const long long n = (long long)d->tokens / (kWarps * tok_of(bwd)) + d->num_seqs;
    return n < d->tokens ? n : d->tokens;
}
int groups_of(const kda_recurrence_desc_t *d) { return (d->channels + kChan - 1) / kChan; }

struct Layout {
    size_t tiles, maps, ends, total;
};
Layout layout_for(const kda_recurrence_desc_t *d, bool bwd) {
    Layout l = {};
    if (walks(d)) return l;
    const size_t n = (size_t)most_tiles(d, bwd), g = groups_of(d);
    l.tiles = round256(n * sizeof(int4));
    l.maps = n * g * kChan * sizeof(float2);
    l.ends = n * g * kChan * sizeof(float);
    l.total = 256 + l.tiles + l.maps + l.ends;
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

constexpr int kMaxSmem = 96 * 1024;  // a stage of 64 KB, a window of 24

template <typename T, bool BWD, bool MIX, int BY, bool SPLIT>
cudaError_t launch_by(const RecArgs &a, long long blocks, const CUtensorMap (&m)[4], cudaStream_t st) {
    const auto kernel = recurrence_kernel<T, BWD, MIX, BY, SPLIT>;
    const int smem = Stage<T, BWD, MIX>::block + 128 + (SPLIT ? a.window * kEntry : 0);
    const cudaError_t e = set_max_dynamic_smem((const void *)kernel, kMaxSmem);
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, dim3((unsigned)blocks), dim3(kThreads), smem, st, a, m[0], m[1],
                            m[2], m[3]);
}

template <typename T, bool BWD, bool MIX>
cudaError_t launch_t(const kda_recurrence_desc_t *d, RecArgs &a, bool pairs, void *workspace,
                     cudaStream_t st) {
    CUtensorMap m[4] = {};
    if (walks(d)) {
        const long long blocks = (long long)a.N * a.groups;
        return pairs ? launch_by<T, BWD, MIX, BY_PAIRS, false>(a, blocks, m, st)
                     : launch_by<T, BWD, MIX, BY_ONE, false>(a, blocks, m, st);
    }
    const Layout l = layout_for(d, BWD);
    uint8_t *ws = (uint8_t *)workspace;
    a.control = (unsigned *)ws;
    a.tiles = (int4 *)(ws + 256);
    a.maps = (float2 *)(ws + 256 + l.tiles);
    a.ends = (float *)(ws + 256 + l.tiles + l.maps);
    a.most_tiles = (int)most_tiles(d, BWD);
    const long long work = (long long)a.most_tiles * a.groups, pieces = work * (kEntry / 16);
    const int sms = device_sms();
    const int clear = (int)(pieces / 4096 < 2 * sms ? pieces / 4096 : 2 * sms) + 1;
    cudaError_t e = launch_dependent(recurrence_tiles_kernel, dim3(1 + clear), dim3(1024), 0, st, a,
                                     BWD);
    if (e != cudaSuccess) return e;
    // A look back reads about as many tiles as are worked on at once in a chain: the nearest
    // of them have published maps, the furthest their ends.
    typedef Stage<T, BWD, MIX> S;
    const int chain = S::fit(4) * sms / a.groups;
    a.window = chain + 4 < 32 ? chain + 4 : 32;
    const long long most = (long long)S::fit(a.window) * sms;
    const long long blocks = work < most ? work : most;
    constexpr int tok = tok_of(BWD), size = sizeof(T);
    const bool tma =
        encode(&m[0], a.g, 4, a.C, a.T, a.g_stride, tok) &&
        (BWD ? encode(&m[1], a.d, size, a.C, a.T, a.C, tok) && encode(&m[2], a.hs, size, a.C, a.T, a.C, tok) &&
                   (!MIX || encode(&m[3], a.x, size, a.C, a.T, a.x_stride, tok))
             : encode(&m[1], a.x, size, a.C, a.T, a.x_stride, tok));
    if (tma && pairs) return launch_by<T, BWD, MIX, BY_TMA, true>(a, blocks, m, st);
    return pairs ? launch_by<T, BWD, MIX, BY_PAIRS, true>(a, blocks, m, st)
                 : launch_by<T, BWD, MIX, BY_ONE, true>(a, blocks, m, st);
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
    const bool pairs = desc->channels % 2 == 0 && a.x_stride % 2 == 0 && a.g_stride % 2 == 0 &&
                     !off(x, 2 * size) && !off(h, 2 * size) && !off(g, 8);
    return launch<false>(desc, a, pairs, workspace, (cudaStream_t)stream);
}

kda_status_t kda_recurrence_backward(const kda_recurrence_desc_t *desc, const void *d_h,
                                     const void *x, const float *g, const void *h, const float *h0,
                                     const int32_t *cu_seqlens, const float *d_h_final, void *dx,
                                     float *dg, float *d_h0, void *workspace, size_t workspace_bytes,
                                     int32_t *dev_status, void *stream) {
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
    const bool pairs = desc->channels % 2 == 0 && a.g_stride % 2 == 0 && !off(d_h, 2 * size) &&
                     !off(h, 2 * size) && !off(dx, 2 * size) && !off(g, 8) && !off(dg, 8) &&
                     (!mix || (a.x_stride % 2 == 0 && !off(x, 2 * size)));
    return launch<true>(desc, a, pairs, workspace, (cudaStream_t)stream);
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
