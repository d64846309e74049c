// Token embedding: out[t] = scale table[id_t], and its table gradient
//     d_table[v] = scale * sum over t with id_t = v, in the order of t, of d_out[t].
//
// Both move each row once and are bound by those bytes (the gradient also writes
// the rows of tokens that do not occur: all V of them).
//
// The gradient sorts the tokens by id first (stable, so the sum's order is fixed
// and there are no floating-point atomics): a radix sort of 32-bit (id, position)
// pairs with two passes of up to 10 bits for vocabularies below 2^20.  The sorted tokens
// and the V row ends are then one merged list (a row's tokens, then its end),
// which is cut into parts of equal length, so a part's work is the same whether a
// few frequent ids or many absent ones fall into it.  A part sums its tokens'
// rows in fp32 and writes every row that ends in it; a row that began in an
// earlier part is finished by a last kernel from the parts' fp32 remainders, in
// order.
//
// Measured on GB300: look-up of 4,096 x 4,096 BF16 10.6 us (6.3 TB/s).  Gradient of
// 81,920 tokens (1 / rank frequencies) into 131,072 x 4,096 BF16 314 us = 5.6 TB/s of
// the bytes it cannot do without: sums 275 us, sort (two passes of counts and moves)
// about 25, joins 14; with few tokens (333 into 257 x 250) 11 us, three launches'
// latency.
#include <math.h>

#include "kda_internal.cuh"
#include "kda_sm100.cuh"
#include "kda_vec.cuh"

namespace kda {
namespace {

using sm100::griddep_launch_dependents;
using sm100::griddep_wait;

// Token id t, or `rows` (one past the table) with the error recorded if it is
// outside it.
__device__ __forceinline__ int load_id(const void *ids, int wide, long long t, int rows,
                                       int32_t *status) {
    const long long v = wide ? ((const long long *)ids)[t] : ((const int *)ids)[t];
    if (v < 0 || v >= rows) {
        dev_fail(status, KDA_ERR_INVALID_ARG);
        return rows;
    }
    return (int)v;
}

// ------------------------------------------------------------------ look-up
// `tpr` threads per token (a power of two), each up to four pieces in flight.
template <typename T, int VEC>
__global__ void __launch_bounds__(256)
    embed_kernel(const T *table, const void *ids, int wide, T *out, int tokens, int rows, int D,
                 int tpr, float scale, int32_t *status) {
    using P = Piece<T, VEC>;
    griddep_wait();
    griddep_launch_dependents();
    const int per = 256 / tpr, g = threadIdx.x / tpr, lane = threadIdx.x - g * tpr;
    const int pieces = (D + VEC - 1) / VEC;
    for (long long t = (long long)blockIdx.x * per + g; t < tokens; t += (long long)gridDim.x * per) {
        const int id = load_id(ids, wide, t, rows, lane == 0 && blockIdx.y == 0 ? status : nullptr);
        const T *src = table + (size_t)id * D;
        T *dst = out + (size_t)t * D;
        for (int c0 = blockIdx.y * tpr * 4; c0 < pieces; c0 += gridDim.y * tpr * 4) {
            P p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = c0 + i * tpr + lane;
                p[i].zero();
                if (c < pieces && id < rows) p[i].load(src + (size_t)c * VEC);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = c0 + i * tpr + lane;
                if (c >= pieces) continue;
                float v[VEC];
                p[i].get(v);
#pragma unroll
                for (int j = 0; j < VEC; ++j) v[j] *= scale;
                P::store(dst + (size_t)c * VEC, v);
            }
        }
    }
}

// --------------------------------------------------------------------- sort
constexpr int kTile = 4096, kSortThreads = 1024, kItems = kTile / kSortThreads;
constexpr int kSortWarps = kSortThreads / 32, kFewTiles = 2;
constexpr int kMaxBits = 10, kMaxDigits = 1 << kMaxBits;
static_assert(kMaxDigits <= kSortThreads, "a thread per digit");

struct SortArgs {
    const void *ids;
    int wide, tokens, rows;
    const int *in_key, *in_pos;  // NULL: the first pass reads ids
    int *out_key, *out_pos;
    int *hist;                   // [tiles][digits]
    int *todo;                   // first pass: cleared for the sums
    int shift, bits, tiles;
    int32_t *status;
};

__device__ __forceinline__ int sort_key(const SortArgs &a, int i, bool report) {
    return a.in_key ? a.in_key[i]
                    : load_id(a.ids, a.wide, i, a.rows, report ? a.status : nullptr);
}

// Counts of this pass's digit in every tile of kTile tokens.
__global__ void __launch_bounds__(kSortThreads) sort_hist_kernel(const __grid_constant__ SortArgs a) {
    __shared__ int cnt[kMaxDigits];
    const int digits = 1 << a.bits;
    for (int d = threadIdx.x; d < digits; d += kSortThreads) cnt[d] = 0;
    griddep_wait();
    griddep_launch_dependents();
    __syncthreads();
    const int base = blockIdx.x * kTile;
    for (int k = threadIdx.x; k < kTile && base + k < a.tokens; k += kSortThreads)
        atomicAdd(&cnt[(sort_key(a, base + k, true) >> a.shift) & (digits - 1)], 1);
    __syncthreads();
    for (int d = threadIdx.x; d < digits; d += kSortThreads)
        a.hist[(size_t)blockIdx.x * digits + d] = cnt[d];
}

// Moves a tile's tokens to their places: all smaller digits, then the same digit
// in earlier tiles, then in earlier warps of this tile, then earlier in the warp
// (a warp holds consecutive tokens, 32 at a time).  With up to kFewTiles tiles each block
// counts the other tiles itself, so up to 8,192 tokens take one launch per pass (a
// frequent id makes the counting slow: at 30,000 tokens 88 us that way, 78 with a launch
// for the counts).  The pass is all latency; large tiles keep the loop over the tiles'
// counts short.
__global__ void __launch_bounds__(kSortThreads)
    sort_scatter_kernel(const __grid_constant__ SortArgs a) {
    extern __shared__ unsigned short cnt[];  // [warps][digits]: tokens, then those before
    __shared__ int first[kMaxDigits];        // place of this tile's first token per digit
    __shared__ int others[kMaxDigits];       // few tiles: tokens of the others
    __shared__ int warp_sum[kSortWarps];
    const int digits = 1 << a.bits, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    unsigned short *mine = cnt + warp * digits;
    for (int d = lane; d < digits; d += 32) mine[d] = 0;
    const bool few = a.tiles <= kFewTiles;
    first[threadIdx.x] = others[threadIdx.x] = 0;
    griddep_wait();
    griddep_launch_dependents();
    if (!a.in_key && blockIdx.x == 0 && threadIdx.x == 0) *a.todo = 0;
    __syncthreads();
    const int base = blockIdx.x * kTile + warp * (kTile / kSortWarps);
    int key[kItems], pos[kItems], rank[kItems];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        const int i = base + k * 32 + lane;
        key[k] = i < a.tokens ? sort_key(a, i, few) : -1;
        pos[k] = a.in_key && i < a.tokens ? a.in_pos[i] : i;
    }
    // thread d: tokens of digit d in all tiles, and in the tiles before this one
    const int dig = threadIdx.x;
    int before = 0, all = 0;
    if (few) {  // first: in the tiles before this one
        for (int t = 0; t < a.tiles; ++t) {
            if (t == (int)blockIdx.x) continue;
#pragma unroll
            for (int k = 0; k < kItems; ++k) {
                const int i = t * kTile + k * kSortThreads + threadIdx.x;
                if (i >= a.tokens) continue;
                const int d = (sort_key(a, i, false) >> a.shift) & (digits - 1);
                atomicAdd(&others[d], 1);
                if (t < (int)blockIdx.x) atomicAdd(&first[d], 1);
            }
        }
        __syncthreads();
        before = first[dig];
        all = others[dig];
    } else if (dig < digits) {
#pragma unroll 10
        for (int t = 0; t < a.tiles; ++t) {
            const int n = a.hist[(size_t)t * digits + dig];
            all += n;
            before += t < (int)blockIdx.x ? n : 0;
        }
    }
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        const bool in = key[k] >= 0;
        const int d = in ? (key[k] >> a.shift) & (digits - 1) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, d);
        const int ahead = __popc(same & ((1u << lane) - 1u));
        rank[k] = in ? mine[d] + ahead : 0;
        __syncwarp();
        if (in && ahead == 0) mine[d] += (unsigned short)__popc(same);
        __syncwarp();
    }
    __syncthreads();
    if (dig < digits) {
        int s = 0;
#pragma unroll 8
        for (int w = 0; w < kSortWarps; ++w) {
            const int n = cnt[w * digits + dig];
            cnt[w * digits + dig] = (unsigned short)s;
            s += n;
        }
        if (few) all += s;
    }
    // exclusive sums over the digits
    int inc = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    int ahead = warp_sum[lane < warp ? lane : 0];  // the warps' totals before this one
    if (lane >= warp) ahead = 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ahead += __shfl_xor_sync(0xffffffffu, ahead, o);
    first[dig] = ahead + inc - all + before;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        if (key[k] < 0) continue;
        const int d = (key[k] >> a.shift) & (digits - 1);
        const int to = first[d] + mine[d] + rank[k];
        a.out_key[to] = key[k];
        a.out_pos[to] = pos[k];
    }
}

// ---------------------------------------------------------------- segment sums
struct SumArgs {
    const int *key, *pos;  // sorted
    int tokens, rows, D;
    int parts;
    long long per;         // entries of the merged list per part
    float *carry, *head;   // [parts][D] fp32
    int *cut;              // [parts]: tokens before the part
    int *todo;             // their number, then the parts in which a row begun earlier ends
    float scale;
};

// Tokens among the first d entries of the merged list (token j comes before the
// end of row i when key[j] <= i).  One warp, which probes 32 places at a time.
__device__ __forceinline__ int merged_tokens(const SumArgs &a, long long d, int lane) {
    int lo = (int)(d > a.rows ? d - a.rows : 0), hi = (int)(d < a.tokens ? d : a.tokens);
    while (lo < hi) {  // the same in all lanes
        const int step = (hi - lo + 31) / 32, at = lo + lane * step;
        const bool before = at < hi && a.key[at] <= d - 1 - at;
        const int n = __popc(__ballot_sync(0xffffffffu, before));  // the first n probes hold
        if (n == 0) break;
        const int next = lo + n * step;
        lo += (n - 1) * step + 1;
        if (next < hi) hi = next;
    }
    return lo;
}

// A block has up to 128 threads, each with NC pieces of VEC columns (four single
// columns of wide rows that are not whole 16-byte pieces), and eight tokens in flight.
constexpr int kSumThreads = 128, kAhead = 8;

// Zeros for n elements: 16-byte stores between the ends, by all threads of the block.
template <typename T>
__device__ __forceinline__ void fill_zero(T *p, long long n) {
    const int lead = (int)((16 - ((uintptr_t)p & 15u)) & 15u) / (int)sizeof(T);
    const long long head = lead < n ? lead : n, pieces = (n - head) * (long long)sizeof(T) / 16;
    const long long tail = head + pieces * (16 / (int)sizeof(T));
    if (threadIdx.x < head) act_st(p, threadIdx.x, 0.f);
    for (long long k = threadIdx.x; k < pieces; k += blockDim.x)
        *(uint4 *)(p + head + k * (16 / (int)sizeof(T))) = make_uint4(0u, 0u, 0u, 0u);
    if (threadIdx.x < n - tail) act_st(p, (size_t)tail + threadIdx.x, 0.f);
}

template <typename T, int VEC, int NC>
__global__ void __launch_bounds__(kSumThreads)
    segment_sum_kernel(const __grid_constant__ SumArgs a, const T *d_out, T *d_table) {
    using P = Piece<T, VEC>;
    __shared__ int cut[2];
    griddep_wait();
    griddep_launch_dependents();
    const long long total = (long long)a.rows + a.tokens;
    const long long d0 = blockIdx.x * a.per, d1 = d0 + a.per < total ? d0 + a.per : total;
    for (int k = threadIdx.x >> 5; k < 2; k += blockDim.x >> 5) {
        const int n = merged_tokens(a, k ? d1 : d0, threadIdx.x & 31);
        if ((threadIdx.x & 31) == 0) cut[k] = n;
    }
    __syncthreads();
    if (threadIdx.x == 0 && blockIdx.y == 0) a.cut[blockIdx.x] = cut[0];
    const int c0 = (blockIdx.y * NC * blockDim.x + threadIdx.x) * VEC, step = blockDim.x * VEC;
    if (VEC > 1 && c0 >= a.D) return;
    int j = cut[0];
    const int j1 = cut[1];
    int i = (int)(d0 - j);
    const int i1 = (int)(d1 - j1);
    // a row that an earlier part began
    bool begun = j > 0 && i < a.rows && a.key[j - 1] == i;
    if (begun && i < i1 && threadIdx.x == 0 && blockIdx.y == 0)
        a.todo[1 + atomicAdd(a.todo, 1)] = blockIdx.x;  // in any order: each is joined by itself
    float acc[NC][VEC];
    auto clear = [&]() {
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
            for (int k = 0; k < VEC; ++k) acc[n][k] = 0.f;
    };
    auto keep = [&](float *to) {  // as a remainder
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
            for (int k = 0; k < VEC; ++k)
                if (c0 + n * step < a.D)
                    to[(size_t)blockIdx.x * a.D + c0 + n * step + k] = acc[n][k];
    };
    auto end_row = [&]() {
        if (begun) {
            keep(a.head);
            begun = false;
        } else {
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                float v[VEC];
#pragma unroll
                for (int k = 0; k < VEC; ++k) v[k] = acc[n][k] * a.scale;
                if (c0 + n * step < a.D) P::store(d_table + (size_t)i * a.D + c0 + n * step, v);
            }
        }
        clear();
        ++i;
    };
    // Rows up to `to` end here: the one that is summed, then rows without tokens.  Those
    // are contiguous memory whatever the width, so where rows are not whole pieces the
    // column blocks share it out as such.
    auto end_rows = [&](int to) {
        if (i < to) end_row();
        if (VEC == 1 && i + 1 < to) {
            const long long n = (long long)(to - i) * a.D, y = blockIdx.y, ny = gridDim.y;
            const long long from = n * y / ny;
            fill_zero(d_table + (size_t)i * a.D + from, n * (y + 1) / ny - from);
            i = to;
        }
        while (i < to) end_row();
    };
    clear();
    while (j < j1) {
        P p[kAhead][NC];
        int id[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            id[u] = j + u < j1 ? a.key[j + u] : -1;
            const T *row = d_out + (size_t)(id[u] >= 0 ? a.pos[j + u] : 0) * a.D + c0;
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                p[u][n].zero();
                if (id[u] >= 0 && c0 + n * step < a.D) p[u][n].load(row + n * step);
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (id[u] < 0) continue;
            end_rows(id[u] < i1 ? id[u] : i1);
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                float v[VEC];
                p[u][n].get(v);
#pragma unroll
                for (int k = 0; k < VEC; ++k) acc[n][k] += v[k];
            }
        }
        j += kAhead;
    }
    end_rows(i1);
    // what is left belongs to a row that ends in a later part
    if (j1 > cut[0] && a.key[j1 - 1] == i1) keep(a.carry);
}

// Rows that span parts: for each part on the list, the remainders of the parts from the
// row's first token on, in order, and the part's own head.  `lanes` threads x 4 columns;
// narrow rows leave room for several slices of the parts (a frequent id of a small
// vocabulary spans a hundred).
constexpr int kJoinThreads = 256;
int join_lanes(int D) { return D >= 1024 ? 256 : 64; }

template <typename T>
__global__ void __launch_bounds__(kJoinThreads)
    segment_join_kernel(const __grid_constant__ SumArgs a, T *d_table, int lanes, bool fours) {
    __shared__ int from;
    __shared__ float4 sh[kJoinThreads];
    griddep_wait();
    griddep_launch_dependents();
    const int slices = kJoinThreads / lanes, slice = threadIdx.x / lanes;
    const int lane = threadIdx.x - slice * lanes;
    const int blocks = (a.D + 4 * lanes - 1) / (4 * lanes), n_todo = *a.todo;
    for (long long w = blockIdx.x; w < (long long)n_todo * blocks; w += gridDim.x) {
        const int part = a.todo[1 + w / blocks], block = (int)(w % blocks);
        const int i = (int)(part * a.per - a.cut[part]);
        if (threadIdx.x < 32) {  // back to the part in which the row begins, 32 at a time
            int q = part - 1;
            while (true) {
                const int at = q - (int)threadIdx.x, n = at >= 0 ? a.cut[at] : 0;
                const unsigned in = __ballot_sync(0xffffffffu, n > 0 && a.key[n > 0 ? n - 1 : 0] == i);
                if (in != 0xffffffffu) {  // part `at` continues the row for the lowest lanes
                    q -= __ffs(~in) - 1;
                    break;
                }
                q -= 32;
            }
            if (threadIdx.x == 0) from = q;
        }
        __syncthreads();
        // four columns together, or `lanes` apart where rows are not whole fours
        const int c = block * 4 * lanes + lane * (fours ? 4 : 1), step = fours ? 1 : lanes;
        auto get = [&](const float *p, int q) {
            const float *r = p + (size_t)q * a.D + c;
            if (fours) return c < a.D ? *(const float4 *)r : make_float4(0.f, 0.f, 0.f, 0.f);
            return make_float4(c < a.D ? r[0] : 0.f, c + step < a.D ? r[step] : 0.f,
                               c + 2 * step < a.D ? r[2 * step] : 0.f,
                               c + 3 * step < a.D ? r[3 * step] : 0.f);
        };
        const long long n = part - from;
        const int q0 = from + (int)(n * slice / slices);
        const int q1 = from + (int)(n * (slice + 1) / slices);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int q = q0; q < q1; ++q) {
            const float4 v = get(a.carry, q);
            acc = make_float4(acc.x + v.x, acc.y + v.y, acc.z + v.z, acc.w + v.w);
        }
        sh[threadIdx.x] = acc;
        __syncthreads();
        if (slice == 0) {
            for (int k = 1; k <= slices; ++k) {
                const float4 v = k < slices ? sh[k * lanes + lane] : get(a.head, part);
                acc = make_float4(acc.x + v.x, acc.y + v.y, acc.z + v.z, acc.w + v.w);
            }
            T *r = d_table + (size_t)i * a.D;
            const float v[4] = {acc.x, acc.y, acc.z, acc.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (c + k * step < a.D) act_st(r, c + k * step, v[k] * a.scale);
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------ host side
size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

int key_bits(int rows) {  // keys 0 .. rows (rows: an id outside the table)
    int b = 1;
    while (b < 31 && (rows >> b) != 0) ++b;
    return b;
}

struct Plan {
    int passes, bits, tiles, parts;
    long long per;
    size_t pairs, hist, rem, cut, total;
};

// Columns of a block of the sums (vec per piece; four single ones per thread in wide
// rows) and its threads.
struct Columns {
    int nc, threads, blocks;
};
Columns columns_for(int D, int vec) {
    Columns c;
    c.nc = vec == 1 && D >= 512 ? 4 : 1;
    const int per = vec * c.nc, threads = ((D + per - 1) / per + 31) / 32 * 32;
    c.threads = threads < kSumThreads ? threads : kSumThreads;
    c.blocks = (D + c.threads * per - 1) / (c.threads * per);
    return c;
}

// Parts of the merged list: as many as give every SM 64 warps, but 1,216 where rows are
// wide, of at least four entries and sqrt(tokens / 32): a frequent id's n tokens are
// added up `per` at a time, then n / per remainders one after another, and text's most
// frequent id has about 1 / 16 of the tokens (5,000 tokens of 128 BF16: 42 us with parts
// of four, 29 with parts of eight).
Plan plan_for(int tokens, int rows, int D, int size) {
    Plan p;
    const int b = key_bits(rows);
    p.passes = (b + kMaxBits - 1) / kMaxBits;
    p.bits = (b + p.passes - 1) / p.passes;
    p.tiles = (tokens + kTile - 1) / kTile;
    const long long total = (long long)tokens + rows;
    const Columns c = columns_for(D, D % (16 / size) == 0 ? 16 / size : 1);
    long long most = 152ll * 64 * 32 / (c.threads * c.blocks);
    if (most < 1216) most = 1216;
    p.per = (total + most - 1) / most;
    const long long least = (long long)sqrt(tokens / 32.0);
    if (p.per < least) p.per = least;
    if (p.per < 4) p.per = 4;
    p.parts = (int)((total + p.per - 1) / p.per);
    p.pairs = round256((size_t)tokens * 4);
    p.hist = round256((size_t)p.tiles * ((size_t)1 << p.bits) * 4);
    p.rem = round256((size_t)p.parts * D * 4);
    p.cut = round256((size_t)(2 * p.parts + 1) * 4);  // cut, todo
    p.total = 4 * p.pairs + p.hist + 2 * p.rem + p.cut;
    return p;
}

bool wide_rows(int D, int size, const void *a, const void *b) {
    return D % (16 / size) == 0 && ((uintptr_t)a & 15u) == 0 && ((uintptr_t)b & 15u) == 0;
}

template <typename T, int VEC>
cudaError_t run_embed(const void *table, const void *ids, int wide, void *out, int tokens, int rows,
                      int D, float scale, int32_t *status, cudaStream_t st) {
    const int pieces = (D + VEC - 1) / VEC;
    int tpr = 8;
    while (tpr < 256 && tpr * 4 < pieces) tpr *= 2;
    const long long need = ((long long)tokens * tpr + 255) / 256, most = 8ll * device_sms();
    const unsigned gx = (unsigned)(need < most ? need : most);
    unsigned gy = (pieces + 4 * tpr - 1) / (4 * tpr);  // few tokens: a wide row over blocks
    if (gy > 64) gy = 64;
    if ((long long)gx * gy > 4 * most) gy = 1;
    return launch_dependent(embed_kernel<T, VEC>, dim3(gx, gy), dim3(256), 0, st, (const T *)table,
                            ids, wide, (T *)out, tokens, rows, D, tpr, scale, status);
}

template <typename T, int VEC, int NC>
cudaError_t run_sums(const SumArgs &a, const Columns &c, const void *d_out, void *d_table,
                     cudaStream_t st) {
    const dim3 grid(a.parts, c.blocks), block(c.threads);
    cudaError_t e = launch_dependent(segment_sum_kernel<T, VEC, NC>, grid, block, 0, st, a,
                                     (const T *)d_out, (T *)d_table);
    if (e != cudaSuccess || a.tokens == 0) return e;
    const int lanes = join_lanes(a.D);
    const long long joins = (long long)a.parts * ((a.D + 4 * lanes - 1) / (4 * lanes));
    const long long most = 8ll * device_sms();
    return launch_dependent(segment_join_kernel<T>, dim3((unsigned)(joins < most ? joins : most)),
                            dim3(kJoinThreads), 0, st, a, (T *)d_table, lanes, a.D % 4 == 0);
}

template <typename T>
cudaError_t run_sums(const SumArgs &a, bool wide, const void *d_out, void *d_table, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    const Columns c = columns_for(a.D, wide ? V : 1);
    if (wide) return run_sums<T, V, 1>(a, c, d_out, d_table, st);
    return c.nc == 4 ? run_sums<T, 1, 4>(a, c, d_out, d_table, st)
                     : run_sums<T, 1, 1>(a, c, d_out, d_table, st);
}

int size_of(const kda_embed_desc_t *d) { return d->act_dtype == KDA_DTYPE_BF16 ? 2 : 4; }

kda_status_t check(const kda_embed_desc_t *d) {
    if (!d) return KDA_ERR_INVALID_ARG;
    if (d->tokens < 0 || d->rows < 1 || d->width < 1 || !isfinite(d->scale))
        return KDA_ERR_INVALID_ARG;
    if (d->act_dtype != KDA_DTYPE_F32 && d->act_dtype != KDA_DTYPE_BF16) return KDA_ERR_UNSUPPORTED;
    if (d->id_dtype != KDA_ID_I32 && d->id_dtype != KDA_ID_I64) return KDA_ERR_UNSUPPORTED;
    if (d->width > 65536 || d->rows > (1 << 30) || d->tokens > (1 << 30)) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

kda_status_t kda_embedding_forward(const kda_embed_desc_t *desc, const void *table, const void *ids,
                                   void *out, int32_t *dev_status, void *stream) {
    kda_status_t rc = check(desc);
    if (rc != KDA_OK) return rc;
    if (desc->tokens == 0) return KDA_OK;
    const int size = size_of(desc), wide = desc->id_dtype == KDA_ID_I64;
    if (!table || !ids || !out || (uintptr_t)table % size || (uintptr_t)out % size ||
        (uintptr_t)ids % (wide ? 8 : 4) || (uintptr_t)dev_status % 4)
        return KDA_ERR_INVALID_ARG;
    const bool vec = wide_rows(desc->width, size, table, out);
    cudaStream_t st = (cudaStream_t)stream;
    const int n = desc->tokens, r = desc->rows, D = desc->width;
    const float s = desc->scale;
    cudaError_t e;
    if (size == 2)
        e = vec ? run_embed<__nv_bfloat16, 8>(table, ids, wide, out, n, r, D, s, dev_status, st)
                : run_embed<__nv_bfloat16, 1>(table, ids, wide, out, n, r, D, s, dev_status, st);
    else
        e = vec ? run_embed<float, 4>(table, ids, wide, out, n, r, D, s, dev_status, st)
                : run_embed<float, 1>(table, ids, wide, out, n, r, D, s, dev_status, st);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

size_t kda_embedding_backward_workspace_size(const kda_embed_desc_t *desc) {
    if (check(desc) != KDA_OK) return 0;
    return plan_for(desc->tokens, desc->rows, desc->width, size_of(desc)).total;
}

kda_status_t kda_embedding_backward(const kda_embed_desc_t *desc, const void *d_out,
                                    const void *ids, void *d_table, void *workspace,
                                    size_t workspace_bytes, int32_t *dev_status, void *stream) {
    kda_status_t rc = check(desc);
    if (rc != KDA_OK) return rc;
    const int size = size_of(desc), wide = desc->id_dtype == KDA_ID_I64;
    if (!d_table || (uintptr_t)d_table % size || (uintptr_t)dev_status % 4) return KDA_ERR_INVALID_ARG;
    if (desc->tokens > 0 && (!d_out || !ids || (uintptr_t)d_out % size ||
                             (uintptr_t)ids % (wide ? 8 : 4)))
        return KDA_ERR_INVALID_ARG;
    const Plan p = plan_for(desc->tokens, desc->rows, desc->width, size_of(desc));
    if (!workspace || workspace_bytes < p.total || ((uintptr_t)workspace & 15u))
        return KDA_ERR_WORKSPACE;
    cudaStream_t st = (cudaStream_t)stream;
    uint8_t *w = (uint8_t *)workspace;
    int *keys[2] = {(int *)w, (int *)(w + p.pairs)};
    int *poss[2] = {(int *)(w + 2 * p.pairs), (int *)(w + 3 * p.pairs)};
    int *cut = (int *)(w + 4 * p.pairs + p.hist + 2 * p.rem);
    int last = 0;
    if (desc->tokens > 0) {
        SortArgs a = {};
        a.ids = ids;
        a.wide = wide;
        a.tokens = desc->tokens;
        a.rows = desc->rows;
        a.hist = (int *)(w + 4 * p.pairs);
        a.bits = p.bits;
        a.tiles = p.tiles;
        a.status = dev_status;
        a.todo = cut + p.parts;
        const size_t scatter_smem = ((size_t)2 * kSortWarps) << p.bits;
        if (set_max_dynamic_smem((const void *)sort_scatter_kernel, (2 * kSortWarps) << kMaxBits) !=
            cudaSuccess)
            return KDA_ERR_CUDA;
        for (int k = 0; k < p.passes; ++k) {
            a.shift = k * p.bits;
            a.in_key = k ? keys[last] : nullptr;
            a.in_pos = k ? poss[last] : nullptr;
            last = k ? 1 - last : 0;
            a.out_key = keys[last];
            a.out_pos = poss[last];
            if ((p.tiles > kFewTiles && launch_dependent(sort_hist_kernel, dim3(p.tiles), dim3(kSortThreads),
                                                 0, st, a) != cudaSuccess) ||
                launch_dependent(sort_scatter_kernel, dim3(p.tiles), dim3(kSortThreads), scatter_smem,
                                 st, a) != cudaSuccess)
                return KDA_ERR_CUDA;
        }
    }
    SumArgs s = {};
    s.key = keys[last];
    s.pos = poss[last];
    s.tokens = desc->tokens;
    s.rows = desc->rows;
    s.D = desc->width;
    s.parts = p.parts;
    s.per = p.per;
    s.carry = (float *)(w + 4 * p.pairs + p.hist);
    s.head = (float *)(w + 4 * p.pairs + p.hist + p.rem);
    s.cut = cut;
    s.todo = cut + p.parts;
    s.scale = desc->scale;
    const bool vec = wide_rows(desc->width, size, d_out, d_table);
    const cudaError_t e = size == 2 ? run_sums<__nv_bfloat16>(s, vec, d_out, d_table, st)
                                    : run_sums<float>(s, vec, d_out, d_table, st);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
