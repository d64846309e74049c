// The gated linear recurrence: every channel c of a packed batch has a state of its own,
//     h_t = e^{g_t} h_{t-1} + w_t x_t,   w = 1 (add) or 1 - e^{g_t} (mix),
// from h0 at the start of its sequence.  Backward, from the last token to the first, with
// u_t = e^{g_t} dh_t the adjoint that a step hands to the one before it:
//     dh_t = d_t + u_{t+1},   dx_t = w_t dh_t,   dg_t = u_t (h_{t-1} [- x_t]),   dh0 = u_first.
//
// Both are scans of maps s -> A s + B (A the product of the factors e^g, B the result from a
// zero start), which compose: a tile of 128 tokens x 64 channels is one map per channel.
// Every element should be read and written once, so the scan takes one pass: a block loads a
// tile into registers (a thread has 8 tokens of two channels), publishes the tile's map, looks
// back along the sequence for the nearest tile whose end state is known, carries that state
// through the maps in between, publishes its own end state and writes its tokens.  Tiles are
// handed out in order by a counter, so a tile that is waited for is already being worked on.
// A state always goes through one tile's map at a time and in order, whoever computes it,
// so the results do not depend on where a look back ended.
//
// Batches of few tokens have no look back: a block takes all tiles of a sequence's 64
// channels one after another.
#include <math.h>

#include "kda_internal.cuh"
#include "kda_sm100.cuh"

namespace kda {
namespace {

using sm100::griddep_launch_dependents;
using sm100::griddep_wait;
using sm100::named_bar_sync;
using sm100::pack_bf16x2;

constexpr int kTok = 8, kWarps = 16, kTile = kTok * kWarps, kChan = 64, kThreads = 32 * kWarps;
constexpr long long kWaitLimit = 4000000000ll;  // ~2 s of SM clocks
// Up to so many tokens one block walks a sequence: eight tiles at worst, which take about as
// long as the launch that lays out the tiles of a batch.
constexpr int kWalkTokens = 1024;

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
    unsigned *flags;     // [tiles][groups] 1: the map is there, 2: the end state too
    float2 *maps;        // [tiles][64 groups]
    float *ends;         // [tiles][64 groups]
    unsigned *control;   // next tile, tiles, a wait gave up
    int most_tiles;
};
enum { NEXT = 0, TILES = 1, ABORT = 2 };

__device__ __forceinline__ int begin_of(const RecArgs &p, int n) { return p.cu ? p.cu[n] : 0; }
__device__ __forceinline__ int end_of(const RecArgs &p, int n) { return p.cu ? p.cu[n + 1] : p.T; }

// a = e^g and w = 1 - e^g.  Slow decays are what a state keeps for thousands of steps, so a
// comes from the exact side: for |g| < 0.34 w is the series of 1 - e^g (seven terms, the next
// is below 2^-25 of w) and a = 1 - w is rounded once; ex2.approx alone is up to 2^-22 off,
// every step in the same direction for a constant gate.
__device__ __forceinline__ void decay(float g, float &a, float &w) {
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * 1.4426950408889634f));
    float s = fmaf(g, 1.f / 5040.f, 1.f / 720.f);
    s = fmaf(g, s, 1.f / 120.f);
    s = fmaf(g, s, 1.f / 24.f);
    s = fmaf(g, s, 1.f / 6.f);
    s = fmaf(g, s, 0.5f);
    s = fmaf(g * g, s, g);
    const bool near = fabsf(g) < 0.34f;
    a = near ? 1.f + s : e;
    w = near ? -s : 1.f - e;
}

// A state through a map; a product of growing factors may be infinite where the state is zero.
__device__ __forceinline__ float through(float A, float B, float s) {
    return s == 0.f ? B : fmaf(A, s, B);
}

// Two channels of one token.
template <typename T>
struct Pair;
template <>
struct Pair<float> {
    float2 v;
    __device__ __forceinline__ void zero() { v = make_float2(0.f, 0.f); }
    __device__ __forceinline__ void load(const float *p) { v = __ldcs((const float2 *)p); }
    __device__ __forceinline__ void load(const float *p, bool second) {
        v = make_float2(__ldcs(p), second ? __ldcs(p + 1) : 0.f);
    }
    __device__ __forceinline__ float2 get() const { return v; }
    static __device__ __forceinline__ void store(float *p, float a, float b) {
        __stcs((float2 *)p, make_float2(a, b));
    }
};
template <>
struct Pair<__nv_bfloat16> {
    uint32_t v;
    __device__ __forceinline__ void zero() { v = 0; }
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { v = __ldcs((const uint32_t *)p); }
    __device__ __forceinline__ void load(const __nv_bfloat16 *p, bool second) {
        const unsigned short *q = (const unsigned short *)p;
        v = __ldcs(q) | (second ? (uint32_t)__ldcs(q + 1) << 16 : 0u);
    }
    __device__ __forceinline__ float2 get() const {
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
    }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, float a, float b) {
        __stcs((uint32_t *)p, pack_bf16x2(a, b));
    }
};

template <bool VEC, typename T>
__device__ __forceinline__ void load_pair(Pair<T> &to, const T *p, int c, int C) {
    if (VEC) {
        if (c < C) to.load(p);
        else to.zero();
    } else if (c < C) {
        to.load(p, c + 1 < C);
    } else {
        to.zero();
    }
}
template <bool VEC, typename T>
__device__ __forceinline__ void store_pair(T *p, int c, int C, float a, float b) {
    if (c >= C) return;
    if (VEC) {
        Pair<T>::store(p, a, b);
    } else {
        act_st(p, 0, a);
        if (c + 1 < C) act_st(p, 1, b);
    }
}

__device__ __forceinline__ unsigned flag_at(const unsigned *p) {
    unsigned v;
    asm volatile("ld.acquire.gpu.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void set_flag(unsigned *p, unsigned v) {
    asm volatile("st.release.gpu.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

struct TileAt {
    int seq, t0, t1, place, group;
    bool last;
};

// The state that enters tile `i` of the table in channel `c`, from the tiles before it in
// its chain (the first of which publishes no map, only its end state).  Called by whole
// warps; false if a wait gave up.
template <bool BWD>
__device__ __forceinline__ bool look_back(const RecArgs &p, int i, const TileAt &t, int c,
                                          float &state) {
    const int lane = threadIdx.x & 31, step = BWD ? 1 : -1;
    const size_t pitch = (size_t)p.groups * kChan;
    const unsigned *mine = p.flags + (size_t)(i + step * (lane + 1)) * p.groups + t.group;
    unsigned known = lane < t.place ? 0 : 1;  // beyond the chain: nothing to wait for
    int from;
    const long long t0 = clock64();
    while (true) {
        if (lane < t.place && known < 2) known = flag_at(mine);
        const unsigned ends = __ballot_sync(0xffffffffu, known == 2);
        const unsigned gaps = __ballot_sync(0xffffffffu, known == 0);
        from = ends ? __ffs(ends) : 0;  // so many tiles back
        if (from && !(gaps & ((1u << (from - 1)) - 1))) break;  // every nearer tile's map is there
        const bool gone = clock64() - t0 > kWaitLimit || flag_at(p.control + ABORT);
        if (__any_sync(0xffffffffu, gone)) {
            if (lane == 0) {
                set_flag(p.control + ABORT, 1);
                dev_fail(p.status, KDA_ERR_TIMEOUT);
            }
            return false;
        }
    }
    __syncwarp();  // orders the other lanes' reads after the flag that one lane saw
    state = __ldcg(p.ends + (size_t)(i + step * from) * pitch + c);
#pragma unroll 4
    for (int k = from - 1; k > 0; --k) {
        const float2 m = __ldcg(p.maps + (size_t)(i + step * k) * pitch + c);
        state = through(m.x, m.y, state);
    }
    return true;
}

template <typename T, bool BWD, bool MIX, bool VEC, bool SPLIT>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 && BWD ? 1 : 2)
    recurrence_kernel(const __grid_constant__ RecArgs p) {
    __shared__ __align__(16) float2 maps[kWarps][kChan];  // a warp's map, then what comes before
    __shared__ __align__(16) float carry[kChan];
    __shared__ int4 next_tile;
    __shared__ int next_ticket;
    __shared__ bool failed;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const T *x = (const T *)p.x, *d = (const T *)p.d, *hs = (const T *)p.hs;
    T *h = (T *)p.h, *dx = (T *)p.dx;
    const float *first = BWD ? p.d_final : p.h0;
    float *final_out = BWD ? p.d_h0 : p.h_final;
    griddep_wait();
    griddep_launch_dependents();

    TileAt t = {};
    int ticket = 0, index = 0, total = 0, walk = 0, begin = 0, end = 0;
    auto take = [&](int &ticket, int4 &tile) {  // one thread
        ticket = (int)atomicAdd(p.control + NEXT, 1u);
        const int k = ticket / p.groups;
        tile = make_int4(0, 0, 0, 0);
        if (k < total) tile = p.tiles[BWD ? total - 1 - k : k];
    };
    int4 ahead;
    int ahead_ticket = 0;
    if (SPLIT) {
        total = (int)p.control[TILES];
        if (threadIdx.x == 0) {
            take(ahead_ticket, ahead);
            next_ticket = ahead_ticket;
            next_tile = ahead;
            failed = false;
        }
        __syncthreads();
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
        const int c = t.group * kChan + threadIdx.x;
        if (threadIdx.x < kChan) {
            const float s = first && c < p.C ? first[(size_t)t.seq * p.C + c] : 0.f;
            carry[threadIdx.x] = s;
            if (begin == end && final_out && c < p.C) final_out[(size_t)t.seq * p.C + c] = s;
        }
        __syncthreads();
    }

    for (;; ++walk) {
        if (SPLIT) {
            ticket = next_ticket;
            const int k = ticket / p.groups;
            if (k >= total || failed) return;
            index = BWD ? total - 1 - k : k;
            t.group = ticket - k * p.groups;
            t.seq = next_tile.x;
            t.t0 = next_tile.y;
            t.t1 = next_tile.z;
            t.place = next_tile.w >> 1;
            t.last = next_tile.w & 1;
            if (threadIdx.x == 0) take(ahead_ticket, ahead);
        } else {
            const int n = (end - begin + kTile - 1) / kTile;
            if (walk >= n) return;
            t.place = walk;
            t.t0 = begin + (BWD ? n - 1 - walk : walk) * kTile;
            t.t1 = min(t.t0 + kTile, end);
            t.last = walk == n - 1;
        }
        const int c = t.group * kChan + 2 * lane;
        const int tok = t.t0 + warp * kTok;  // this thread's first token
        const bool starts = BWD ? t.last : t.place == 0;  // the tile has the sequence's first token

        // the tile into registers; the map of this warp's tokens
        float a[kTok][2], b[kTok][2];  // forward: factor, term.  Backward: g, d
        Pair<T> px[BWD && MIX ? kTok : 1], ph[BWD ? kTok : 1];
        {
            Pair<float> pg[kTok];
            Pair<T> pv[kTok];
#pragma unroll
            for (int j = 0; j < kTok; ++j) {
                const size_t row = (size_t)(tok + j);
                const bool live = tok + j < t.t1;
                pg[j].zero();
                pv[j].zero();
                if (live) {
                    load_pair<VEC>(pg[j], p.g + row * p.g_stride + c, c, p.C);
                    load_pair<VEC>(pv[j], BWD ? d + row * p.C + c : x + row * p.x_stride + c, c, p.C);
                }
                if constexpr (BWD) {
                    ph[j].zero();
                    if (live && !(starts && tok + j == t.t0))
                        load_pair<VEC>(ph[j], hs + (row - 1) * p.C + c, c, p.C);
                    if constexpr (MIX) {
                        px[j].zero();
                        if (live) load_pair<VEC>(px[j], x + row * p.x_stride + c, c, p.C);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < kTok; ++j) {
                const float2 gg = pg[j].get(), v = pv[j].get();
                if constexpr (BWD) {
                    a[j][0] = gg.x;
                    a[j][1] = gg.y;
                    b[j][0] = v.x;
                    b[j][1] = v.y;
                } else {
                    float w0, w1;
                    decay(gg.x, a[j][0], w0);
                    decay(gg.y, a[j][1], w1);
                    b[j][0] = MIX ? w0 * v.x : v.x;
                    b[j][1] = MIX ? w1 * v.y : v.y;
                }
            }
        }
        float A[2] = {1.f, 1.f}, B[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
            const int j = BWD ? kTok - 1 - i : i;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                if constexpr (BWD) {
                    float f, w;
                    decay(a[j][q], f, w);
                    B[q] = f * (B[q] + b[j][q]);
                    A[q] *= f;
                } else {
                    B[q] = fmaf(a[j][q], B[q], b[j][q]);
                    A[q] *= a[j][q];
                }
            }
        }
        *(float4 *)&maps[warp][2 * lane] = make_float4(A[0], B[0], A[1], B[1]);
        __syncthreads();

        // two warps, a channel each: the warps' maps joined, and the state that enters
        if (warp < 2) {
            const int cc = threadIdx.x, ch = t.group * kChan + cc;
            float2 m = make_float2(1.f, 0.f);
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                const int w = BWD ? kWarps - 1 - i : i;
                const float2 v = maps[w][cc];
                maps[w][cc] = m;
                m.y = through(v.x, v.y, m.y);
                m.x *= v.x;
            }
            float s;
            if (SPLIT) {
                const size_t slot = (size_t)index * p.groups * kChan + ch;
                unsigned *flag = p.flags + (size_t)index * p.groups + t.group;
                bool ok = true;
                if (t.place > 0) {
                    if (!t.last) {
                        __stcg(p.maps + slot, m);
                        __threadfence();
                        named_bar_sync(1, kChan);
                        if (threadIdx.x == 0) set_flag(flag, 1);
                    }
                    ok = look_back<BWD>(p, index, t, ch, s);
                } else {
                    s = first && ch < p.C ? first[(size_t)t.seq * p.C + ch] : 0.f;
                }
                if (!ok) failed = true;
                if (!t.last && ok) {
                    __stcg(p.ends + slot, through(m.x, m.y, s));
                    __threadfence();
                }
                named_bar_sync(1, kChan);
                if (!t.last && threadIdx.x == 0 && !failed) set_flag(flag, 2);
            } else {
                s = carry[cc];
            }
            carry[cc] = s;
            const float to = through(m.x, m.y, s);
            if (t.last && final_out && ch < p.C && !(SPLIT && failed))
                final_out[(size_t)t.seq * p.C + ch] = to;
        }
        __syncthreads();
        if (SPLIT && failed) return;

        // this thread's tokens, from the state that enters them
        float s[2];
        {
            const float4 m = *(const float4 *)&maps[warp][2 * lane];
            const float2 in = *(const float2 *)&carry[2 * lane];
            s[0] = through(m.x, m.y, in.x);
            s[1] = through(m.z, m.w, in.y);
        }
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
            const int j = BWD ? kTok - 1 - i : i;
            const size_t row = (size_t)(tok + j);
            const bool live = tok + j < t.t1;
            if constexpr (!BWD) {
                s[0] = fmaf(a[j][0], s[0], b[j][0]);
                s[1] = fmaf(a[j][1], s[1], b[j][1]);
                if (live) store_pair<VEC>(h + row * p.C + c, c, p.C, s[0], s[1]);
            } else {
                float2 hp = ph[j].get(), xv = make_float2(0.f, 0.f);
                if constexpr (MIX) xv = px[j].get();
                if (j == 0 && warp == 0 && starts && p.h0) {
                    if (c < p.C) hp.x = p.h0[(size_t)t.seq * p.C + c];
                    if (c + 1 < p.C) hp.y = p.h0[(size_t)t.seq * p.C + c + 1];
                }
                float o[2], og[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float f, w;
                    decay(a[j][q], f, w);
                    const float dh = b[j][q] + s[q];
                    s[q] = f * dh;
                    o[q] = MIX ? w * dh : dh;
                    og[q] = s[q] * ((q ? hp.y : hp.x) - (MIX ? (q ? xv.y : xv.x) : 0.f));
                }
                if (live) {
                    store_pair<VEC>(dx + row * p.C + c, c, p.C, o[0], o[1]);
                    store_pair<VEC>(p.dg + row * p.C + c, c, p.C, og[0], og[1]);
                }
            }
        }
        if (SPLIT) {
            if (threadIdx.x == 0) {
                next_ticket = ahead_ticket;
                next_tile = ahead;
            }
            __syncthreads();
        } else if (!t.last) {
            // the state that leaves the tile: the last warp in the chain has it
            __syncthreads();
            if (warp == (BWD ? 0 : kWarps - 1)) *(float2 *)&carry[2 * lane] = make_float2(s[0], s[1]);
            __syncthreads();
        }
    }
}

// The tiles of every sequence, the cleared flags, and the states of empty sequences.
__global__ void __launch_bounds__(1024) recurrence_tiles_kernel(const __grid_constant__ RecArgs p,
                                                                bool backward) {
    __shared__ int sums[32];
    __shared__ int base;
    __shared__ bool bad;
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (blockIdx.x > 0) {
        const long long me = (blockIdx.x - 1) * 1024ll + threadIdx.x, all = (gridDim.x - 1) * 1024ll;
        const long long words = (long long)p.most_tiles * p.groups;
        for (long long k = me; k < words; k += all) p.flags[k] = 0;
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
        for (int j = 0; j < VEC; ++j) {
            float a, w;
            decay(gv[j], a, w);
            sv[j] = fmaf(a, sv[j], MIX ? w * xv[j] : xv[j]);
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
long long most_tiles(const kda_recurrence_desc_t *d) {
    const long long n = (long long)d->tokens / kTile + d->num_seqs;
    return n < d->tokens ? n : d->tokens;
}
int groups_of(const kda_recurrence_desc_t *d) { return (d->channels + kChan - 1) / kChan; }

struct Layout {
    size_t tiles, flags, maps, ends, total;
};
Layout layout_for(const kda_recurrence_desc_t *d) {
    Layout l = {};
    if (walks(d)) return l;
    const size_t n = (size_t)most_tiles(d), g = groups_of(d);
    l.tiles = round256(n * sizeof(int4));
    l.flags = round256(n * g * 4);
    l.maps = round256(n * g * kChan * sizeof(float2));
    l.ends = round256(n * g * kChan * sizeof(float));
    l.total = 256 + l.tiles + l.flags + l.maps + l.ends;
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
    if (most_tiles(d) * groups_of(d) > (1ll << 30) ||
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

template <typename T, bool BWD, bool MIX, bool VEC>
cudaError_t launch_v(const kda_recurrence_desc_t *d, RecArgs &a, void *workspace, cudaStream_t st) {
    if (walks(d))
        return launch_dependent(recurrence_kernel<T, BWD, MIX, VEC, false>, dim3(a.N * a.groups),
                                dim3(kThreads), 0, st, a);
    const Layout l = layout_for(d);
    uint8_t *ws = (uint8_t *)workspace;
    a.control = (unsigned *)ws;
    a.tiles = (int4 *)(ws + 256);
    a.flags = (unsigned *)(ws + 256 + l.tiles);
    a.maps = (float2 *)(ws + 256 + l.tiles + l.flags);
    a.ends = (float *)(ws + 256 + l.tiles + l.flags + l.maps);
    a.most_tiles = (int)most_tiles(d);
    const long long words = (long long)a.most_tiles * a.groups;
    const int clear = (int)(words / 8192 < 64 ? words / 8192 : 64) + 1;
    cudaError_t e = launch_dependent(recurrence_tiles_kernel, dim3(1 + clear), dim3(1024), 0, st, a,
                                     BWD);
    if (e != cudaSuccess) return e;
    const long long most = (sizeof(T) == 4 && BWD ? 1 : 2) * (long long)device_sms();
    return launch_dependent(recurrence_kernel<T, BWD, MIX, VEC, true>,
                            dim3((unsigned)(words < most ? words : most)), dim3(kThreads), 0, st, a);
}

template <bool BWD>
kda_status_t launch(const kda_recurrence_desc_t *d, RecArgs &a, bool vec, void *workspace,
                    cudaStream_t st) {
    const bool f32 = d->act_dtype == KDA_DTYPE_F32, mix = d->write == KDA_WRITE_MIX;
    typedef __nv_bfloat16 B;
    cudaError_t e;
    if (f32)
        e = mix ? (vec ? launch_v<float, BWD, true, true>(d, a, workspace, st)
                       : launch_v<float, BWD, true, false>(d, a, workspace, st))
                : (vec ? launch_v<float, BWD, false, true>(d, a, workspace, st)
                       : launch_v<float, BWD, false, false>(d, a, workspace, st));
    else
        e = mix ? (vec ? launch_v<B, BWD, true, true>(d, a, workspace, st)
                       : launch_v<B, BWD, true, false>(d, a, workspace, st))
                : (vec ? launch_v<B, BWD, false, true>(d, a, workspace, st)
                       : launch_v<B, BWD, false, false>(d, a, workspace, st));
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

int size_of(const kda_recurrence_desc_t *d) { return d->act_dtype == KDA_DTYPE_BF16 ? 2 : 4; }
bool off(const void *p, int size) { return ((uintptr_t)p & (size - 1)) != 0; }
bool bad_ws(const kda_recurrence_desc_t *d, const void *ws, size_t bytes) {
    const size_t need = layout_for(d).total;
    return need > 0 && (!ws || bytes < need || off(ws, 16));
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

size_t kda_recurrence_workspace_size(const kda_recurrence_desc_t *desc) {
    return check(desc) == KDA_OK ? layout_for(desc).total : 0;
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
    if (bad_ws(desc, workspace, workspace_bytes)) return KDA_ERR_WORKSPACE;
    RecArgs a = make_args(desc);
    a.x = x; a.g = g; a.h0 = h0; a.cu = cu_seqlens; a.h = h; a.h_final = h_final;
    a.status = dev_status;
    const bool vec = desc->channels % 2 == 0 && a.x_stride % 2 == 0 && a.g_stride % 2 == 0 &&
                     !off(x, 2 * size) && !off(h, 2 * size) && !off(g, 8);
    return launch<false>(desc, a, vec, workspace, (cudaStream_t)stream);
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
    if (bad_ws(desc, workspace, workspace_bytes)) return KDA_ERR_WORKSPACE;
    RecArgs a = make_args(desc);
    a.x = x; a.g = g; a.h0 = h0; a.cu = cu_seqlens; a.d = d_h; a.hs = h; a.d_final = d_h_final;
    a.dx = dx; a.dg = dg; a.d_h0 = d_h0;
    a.status = dev_status;
    const bool vec = desc->channels % 2 == 0 && a.g_stride % 2 == 0 && !off(d_h, 2 * size) &&
                     !off(h, 2 * size) && !off(dx, 2 * size) && !off(g, 8) && !off(dg, 8) &&
                     (!mix || (a.x_stride % 2 == 0 && !off(x, 2 * size)));
    return launch<true>(desc, a, vec, workspace, (cudaStream_t)stream);
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
