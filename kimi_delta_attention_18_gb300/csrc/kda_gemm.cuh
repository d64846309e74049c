// What the products of the cross entropy and of the gated feed-forward block share: their
// arguments, tiles and epilogues.  The kernels are in kda_gemm_kernel.cuh (BF16 operands)
// and kda_ce_w32.cu (an fp32 weight, few tokens).
#pragma once

#include "kda_internal.cuh"
#include "kda_sm100.cuh"

namespace kda {

using namespace sm100;

constexpr int BM = 128, BN = 256, BK = 64;  // rows per CTA, columns, contraction per stage
constexpr int kABytes = BM * BK * 2, kBBytes = BN * BK * 2, kBox = 64 * BK * 2;
constexpr int kEpiWarps = 8, kThreads = 32 * (2 + kEpiWarps);
constexpr int kGroupRows = 2048;  // rows whose tiles share a sweep over the column tiles
constexpr long long kWaitLimit = 4000000000ll;  // ~2 s of SM clocks
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr uint32_t kTmemCols = 512;  // two 256-column accumulators

// EPI_GLU, EPI_DGLU: B's rows are taken from two matrices in turn, 32 of the first and 32 of
// the second, so 64 accumulator columns are both projections of 32 of the block's channels.
enum { EPI_STATS = 0, EPI_DZ = 1, EPI_OUT = 2, EPI_GLU = 3, EPI_DGLU = 4 };
enum { ACT_SIGMOID = 1, ACT_SILU = 2, ACT_GELU = 3 };  // kda_ffn_act_t

struct Targets {
    const void *ids;
    int wide, vocab;
    long long ignore;
    int32_t *status;
    // The target of row t; -1 where it is to be ignored (or, recorded, outside
    // the vocabulary).
    __device__ __forceinline__ int at(long long t, bool report) const {
        const long long y = wide ? ((const long long *)ids)[t] : ((const int *)ids)[t];
        if (y == ignore) return -1;
        if (y < 0 || y >= vocab) {
            if (report) dev_fail(status, KDA_ERR_INVALID_ARG);
            return -1;
        }
        return (int)y;
    }
};

struct GemmArgs {
    int M, N;                  // rows and columns of the product that exist
    int cols;                  // columns of the outputs: N, or of one of EPI_GLU's matrices
    int k_blocks, splits, pairs;
    // Operands of more than one matrix, [planes][groups][rows][pitch]: groups > 1 adds the
    // matrices' products up (dx = da Wg + db Wu), batches > 1 keeps them apart (dWg, dWu).
    int groups, batches;
    int a_group, b_group;      // matrices in A's and B's planes
    int chunk;                 // FINE: stages per accumulator
    int m_tiles, n_tiles, bn;  // set at the launch (bn, columns per tile, unless the caller did:
                               // a multiple of 64)
    int ctas;                  // CTAs of a tile, 0: as use_pairs says
    int b_row0;                // B's first row (of the vocabulary's piece)
    int bk_row0;               // the same where the contraction is along B's rows
    // EPI_STATS, EPI_DZ
    Targets y;
    float2 *part;              // [2 n_tiles][M] (maximum, sum)
    float *z_y;                // [M]
    unsigned *ticket;          // cleared for the join kernel
    const float *lse, *d_loss;
    __nv_bfloat16 *dz;         // [planes][M][pitch]
    int pitch, planes;
    // BF16: the unit of dz (the largest |d_loss|, or its significand); EPI_OUT multiplies by it
    const float *unit;
    // EPI_OUT: value (+ acc_in) to acc_out, both [splits][batches][M][cols] fp32, or to out
    // (batches out_batch elements apart)
    long long out_batch;
    const float *acc_in;
    float *acc_out;
    void *out;
    int out_bf16, vec;
    // EPI_GLU: act(a) b to out [M][out_ld].  EPI_DGLU: from d_h [M][out_ld] the adjoints of
    // a and b to dz's first and second matrix.
    int act, out_ld;
    const void *d_h;
    int32_t *status;
};

// Arguments of a product of one matrix by another.
inline GemmArgs one_product() {
    GemmArgs p = {};
    p.splits = p.groups = p.batches = p.a_group = p.b_group = 1;
    return p;
}

// The activation of a gated block and its derivative.  ex2.approx and rcp.approx are within
// 2^-22; the exponent's rounding adds |a| 2^-24 of it, where |a| is large a vanishing value.
__device__ __forceinline__ void glu_act(int act, float a, float &f, float &df) {
    if (act == ACT_GELU) {
        const float cdf = 0.5f * erfcf(a * -0.70710678118654752f);
        f = a * cdf;
        df = fmaf(a * 0.39894228040143268f, exp2f(a * a * (-0.5f * kLog2e)), cdf);
        return;
    }
    float e, p;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-a * kLog2e));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(p) : "f"(1.f + e));
    // 1 - p = e p; e may have overflowed where p is 0
    const float q = 1.f - p;
    f = act == ACT_SILU ? a * p : p;
    df = act == ACT_SILU ? p * fmaf(a, q, 1.f) : p * q;
}

// MN-major operand with 128-byte swizzle, as boxes of 64 elements x `rows` rows lay it
// down: 8 rows (along K) of 128 bytes form an atom, atoms follow each other along
// K (1024 bytes), boxes along M / N (128 rows bytes).
__device__ __forceinline__ uint64_t umma_desc_mn_sw128(uint32_t saddr, int rows) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)((rows * 128) >> 4) << 16;  // between 64-element boxes
    d |= (uint64_t)(1024 >> 4) << 32;        // between 8-row atoms along K
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
}

struct Tile {
    int m, n, split, batch, kb0, kb1;
};
template <int CTAS>
__device__ __forceinline__ Tile tile_at(const GemmArgs &p, int w) {
    constexpr int G = kGroupRows / (BM * CTAS);
    Tile t;
    const int per = p.m_tiles * p.n_tiles;
    t.split = w / per;
    const int r = w - t.split * per;
    t.batch = 0;
    if (p.batches > 1) {
        t.batch = t.split % p.batches;
        t.split /= p.batches;
    }
    const int g = r / (G * p.n_tiles), q = r - g * G * p.n_tiles;
    const int gm = min(G, p.m_tiles - g * G);
    t.n = q / gm;
    t.m = g * G + (q - t.n * gm);
    t.kb0 = (int)((long long)p.k_blocks * t.split / p.splits);
    t.kb1 = (int)((long long)p.k_blocks * (t.split + 1) / p.splits);
    return t;
}

// Terms of pair i of an fp32 product, smallest weight first: (1,1) (2,0) (0,2)
// (1,0) (0,1) (0,0); a single pair is (0,0).
__device__ __forceinline__ int term_a(int i, int pairs) {
    return pairs == 1 ? 0 : (0x001021 >> (4 * (i))) & 3;
}
__device__ __forceinline__ int term_b(int i, int pairs) {
    return pairs == 1 ? 0 : (0x010201 >> (4 * (i))) & 3;
}

// A warp's 32 rows x 128 bytes on their way to memory: a thread has a row, but a store
// should have whole lines (with a row per thread each store instruction touched 32 of
// them, and storing three terms of dz took as long as half of the tile's products).
struct Turn {
    uint32_t at;
    int lane;
    // 16-byte piece q of this thread's row
    __device__ __forceinline__ void put(int q, uint4 v) const {
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(
                         at + lane * 128 + ((q ^ (lane & 7)) << 4)),
                     "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                     : "memory");
    }
    __device__ __forceinline__ int row(int it) const { return 4 * it + (lane >> 3); }
    // piece lane % 8 of row(it), it = 0 .. 7
    __device__ __forceinline__ uint4 get(int it) const {
        uint4 v;
        const int r = row(it);
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "r"(at + r * 128 + (((lane & 7) ^ (r & 7)) << 4))
                     : "memory");
        return v;
    }
    // piece q of this thread's row
    __device__ __forceinline__ float4 own(int q) const {
        float4 v;
        asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                     : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                     : "r"(at + lane * 128 + ((q ^ (lane & 7)) << 4))
                     : "memory");
        return v;
    }
    // word `lane` of row r
    __device__ __forceinline__ void set_word(int r, float v) const {
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) +
                                                     4 * (lane & 3)),
                     "f"(v)
                     : "memory");
    }
    __device__ __forceinline__ float word(int r) const {
        float v;
        asm volatile("ld.shared.f32 %0, [%1];"
                     : "=f"(v)
                     : "r"(at + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + 4 * (lane & 3))
                     : "memory");
        return v;
    }
};

constexpr int kBatch = 8;  // rows whose words are read before any is stored

// One thread's part of the epilogue: a row and up to 128 of the tile's columns, taken
// 32 at a time.  BF16: the product may be stored so.
template <int EPI, bool BF16>
struct Row {
    int row0;       // the warp's first row
    long long row;  // this thread's
    bool live;
    int c0;  // first column, in the launch's columns
    int y;   // the target's column (negative: none)
    float mx, sum, lse2, g;

    __device__ __forceinline__ void begin(const GemmArgs &p, const Tile &t, int first_row, int lane,
                                          int half, int half_cols) {
        row0 = first_row;
        row = first_row + lane;
        live = row < p.M;
        c0 = t.n * p.bn + half * half_cols;
        y = -1;
        mx = -INFINITY;
        sum = lse2 = g = 0.f;
        if ((EPI == EPI_STATS || EPI == EPI_DZ) && live) {
            y = p.y.at(row, t.n == 0 && half == 0);
            if (EPI == EPI_DZ) {
                lse2 = p.lse[row] * kLog2e;
                g = y >= 0 ? p.d_loss[row] : 0.f;
                if (p.unit) g /= *p.unit;
            }
            y = y >= 0 ? y - p.b_row0 : -1;
        }
        if (EPI == EPI_OUT && BF16) g = p.unit ? *p.unit : 1.f;
    }

    // 32 values as BF16 into half `h` of the warp's lines; what the rounding left stays
    // in v if LEFT.
    template <bool LEFT>
    __device__ __forceinline__ void put_bf16(const Turn &turn, int h, float (&v)[32]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                w[k] = pack_bf16x2(v[8 * i + 2 * k], v[8 * i + 2 * k + 1]);
                if (LEFT) {
                    v[8 * i + 2 * k] -= __uint_as_float(w[k] << 16);
                    v[8 * i + 2 * k + 1] -= __uint_as_float(w[k] & 0xffff0000u);
                }
            }
            turn.put(4 * h + i, make_uint4(w[0], w[1], w[2], w[3]));
        }
    }
    // The lines to memory: row r's at base + r pitch.
    __device__ __forceinline__ void lines(const GemmArgs &p, const Turn &turn, __nv_bfloat16 *base,
                                          size_t pitch) {
        __syncwarp();
#pragma unroll
        for (int it = 0; it < 8; ++it) {
            const long long r = row0 + turn.row(it);
            const uint4 u = turn.get(it);
            if (r < p.M) *(uint4 *)(base + (size_t)r * pitch + 8 * (turn.lane & 7)) = u;
        }
        __syncwarp();
    }

    // The same to rows of any width, n of the 64 columns: words aligned in memory, and a
    // row's odd ends by themselves (107 x 58,219 x 6,404: d_weight 368 us, 819 column by column)
    __device__ __forceinline__ void ragged(const GemmArgs &p, const Turn &turn, __nv_bfloat16 *base,
                                           size_t pitch, int n) {
        __syncwarp();
        const int rows = (int)(p.M - row0 < 32 ? p.M - row0 : 32), l = turn.lane;
        for (int r0 = 0; r0 < rows; r0 += kBatch) {
            uint32_t w[kBatch], next[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) w[k] = __float_as_uint(turn.word(r0 + k));
#pragma unroll
            for (int k = 0; k < kBatch; ++k) next[k] = __shfl_down_sync(0xffffffffu, w[k], 1);
            __nv_bfloat16 *to = base + (size_t)(row0 + r0) * pitch;
#pragma unroll
            for (int k = 0; k < kBatch; ++k, to += pitch) {
                if (r0 + k >= rows) break;
                const int odd = ((uintptr_t)to >> 1) & 1, c = 2 * l + odd;
                const uint32_t v = odd ? __funnelshift_r(w[k], next[k], 16) : w[k];
                if (c + 1 < n) *(uint32_t *)(to + c) = v;
                if (c + 1 == n) *(uint16_t *)(to + c) = (uint16_t)v;
                if (odd && l == 0) *(uint16_t *)to = (uint16_t)w[k];
            }
        }
        __syncwarp();
    }

    // v -> d_loss (softmax - onehot) for columns c .. c + 31
    __device__ __forceinline__ void dz_of(const GemmArgs &p, int c, float (&v)[32]) {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const float e = g * exp2f(fmaf(v[i], kLog2e, -lse2));
            v[i] = g != 0.f && c + i < p.N ? e : 0.f;
        }
        if (__any_sync(0xffffffffu, y >= c && y < c + 32)) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] -= c + i == y ? g : 0.f;
        }
    }

    __device__ __forceinline__ void stats(const GemmArgs &p, int c, float (&v)[32]) {
        if (c + 32 > p.N) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = c + i < p.N ? v[i] : -INFINITY;
        }
        const bool mine = y >= c && y < c + 32;
        if (__any_sync(0xffffffffu, mine)) {
            float z = 0.f;
#pragma unroll
            for (int i = 0; i < 32; ++i) z = c + i == y ? v[i] : z;
            if (mine) p.z_y[row] = z;
        }
        float m = mx;
#pragma unroll
        for (int i = 0; i < 32; ++i) m = fmaxf(m, v[i]);
        const float ref = m == -INFINITY ? 0.f : m * kLog2e;
        sum *= exp2f(mx == -INFINITY ? -INFINITY : fmaf(mx, kLog2e, -ref));
        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 32; ++i) s[i & 3] += exp2f(fmaf(v[i], kLog2e, -ref));
        sum += (s[0] + s[1]) + (s[2] + s[3]);
        mx = m;
    }

    // 32 columns of fp32 (+ acc_in) to acc_out or out
    __device__ __forceinline__ void out32(const GemmArgs &p, const Tile &t, const Turn &turn, int c,
                                          float (&v)[32]) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            turn.put(i, make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                                   __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3])));
        __syncwarp();
        const bool narrow = BF16 && p.out && p.out_bf16;
        const size_t part = ((size_t)t.split * p.batches + t.batch) * p.M * p.cols;
        const size_t ld = EPI == EPI_GLU ? p.out_ld : p.cols;
        float *o32 = p.out ? (float *)p.out + t.batch * p.out_batch : p.acc_out + part;
        const float *in = p.acc_in ? p.acc_in + part : nullptr;
        __nv_bfloat16 *o16 = (__nv_bfloat16 *)p.out + t.batch * p.out_batch;
        if (p.vec) {  // widths and bases of whole pieces: four columns are in or out together
            const int col = c + 4 * (turn.lane & 7);
#pragma unroll
            for (int it = 0; it < 8; ++it) {
                const long long r = row0 + turn.row(it);
                const uint4 u = turn.get(it);
                if (r >= p.M || col >= p.cols) continue;
                const size_t at = (size_t)r * ld + col;
                float4 f = make_float4(__uint_as_float(u.x), __uint_as_float(u.y),
                                       __uint_as_float(u.z), __uint_as_float(u.w));
                if (in) {
                    const float4 a = *(const float4 *)(in + at);
                    f = make_float4(f.x + a.x, f.y + a.y, f.z + a.z, f.w + a.w);
                }
                if (narrow)
                    *(uint2 *)(o16 + at) = make_uint2(pack_bf16x2(f.x, f.y), pack_bf16x2(f.z, f.w));
                else
                    *(float4 *)(o32 + at) = f;
            }
        } else {
            const int rows = (int)(p.M - row0 < 32 ? p.M - row0 : 32);
#pragma unroll 4
            for (int r = 0; r < rows; ++r) {
                float f = turn.word(r);
                if (c + turn.lane >= p.cols) continue;
                const size_t at = (size_t)(row0 + r) * ld + c + turn.lane;
                if (in) f += in[at];
                if (narrow) o16[at] = __float2bfloat16_rn(f);
                else o32[at] = f;
            }
        }
        __syncwarp();
    }

    // The warp's half lines (pieces 0-3) to `first` and, if given, pieces 4-7 to `second`: 32
    // columns of each, 64 contiguous bytes of a row.
    __device__ __forceinline__ void half_lines(const GemmArgs &p, const Turn &turn,
                                               __nv_bfloat16 *first, __nv_bfloat16 *second,
                                               size_t pitch) {
        __syncwarp();
#pragma unroll
        for (int it = 0; it < 8; ++it) {
            const int piece = turn.lane & 7;
            const long long r = row0 + turn.row(it);
            const uint4 u = turn.get(it);
            __nv_bfloat16 *to = piece < 4 ? first : second;
            if (r < p.M && to) *(uint4 *)(to + (size_t)r * pitch + 8 * (piece & 3)) = u;
        }
        __syncwarp();
    }

    // act(a) b of channels f .. f + 31
    __device__ __forceinline__ void glu(const GemmArgs &p, const Tile &t, const Turn &turn, int f,
                                        float (&a)[32], float (&b)[32]) {
        if (f >= p.cols) return;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            float v, dv;
            glu_act(p.act, a[i], v, dv);
            a[i] = v * b[i];
        }
        if (!BF16) {
            out32(p, t, turn, f, a);
            return;
        }
        __nv_bfloat16 *out = (__nv_bfloat16 *)p.out + f;
        put_bf16<false>(turn, 0, a);
        if (p.vec && f + 32 <= p.cols) half_lines(p, turn, out, nullptr, p.out_ld);
        else ragged(p, turn, out, p.out_ld, p.cols - f < 32 ? p.cols - f : 32);
    }

    // dz of channels f .. f + 31: d_h b act'(a) and d_h act(a), zeros past the last channel
    // (dz's pitch is a multiple of 64, and the next products read whole steps of 64)
    __device__ __forceinline__ void dglu(const GemmArgs &p, const Turn &turn, int f,
                                         float (&a)[32], float (&b)[32]) {
        if (f >= (p.cols + 63) / 64 * 64) return;
        const int n = p.cols - f;
        const size_t at = (size_t)row * p.out_ld + f;
        if (!p.vec) {  // rows of any width: a row at a time (777 x 515 x 1,003, BF16: 27 us, each
                       // thread its own row 28)
            const int rows = (int)(p.M - row0 < 32 ? p.M - row0 : 32), l = turn.lane;
            __syncwarp();
            for (int r0 = 0; r0 < 32; r0 += kBatch) {
                float v[kBatch];
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    const size_t e = (size_t)(row0 + r0 + k) * p.out_ld + f + l;
                    const bool in = r0 + k < rows && l < n;
                    if (p.planes == 1) v[k] = in ? act_ld((const __nv_bfloat16 *)p.d_h, e) : 0.f;
                    else v[k] = in ? act_ld((const float *)p.d_h, e) : 0.f;
                }
#pragma unroll
                for (int k = 0; k < kBatch; ++k) turn.set_word(r0 + k, v[k]);
            }
            __syncwarp();
        }
#pragma unroll
        for (int i0 = 0; i0 < 32; i0 += 8) {
            float d[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) d[k] = 0.f;
            if (live && p.vec && i0 < n) {  // pieces of eight are in or out together
                if (p.planes == 1) {
                    const uint4 u = *(const uint4 *)((const __nv_bfloat16 *)p.d_h + at + i0);
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        d[2 * k] = __uint_as_float(w[k] << 16);
                        d[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
                    }
                } else {
                    *(float4 *)d = *(const float4 *)((const float *)p.d_h + at + i0);
                    *(float4 *)(d + 4) = *(const float4 *)((const float *)p.d_h + at + i0 + 4);
                }
            } else if (!p.vec) {
                *(float4 *)d = turn.own(i0 / 4);
                *(float4 *)(d + 4) = turn.own(i0 / 4 + 1);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                float v, dv;
                glu_act(p.act, a[i0 + k], v, dv);
                a[i0 + k] = d[k] * b[i0 + k] * dv;
                b[i0 + k] = d[k] * v;
            }
        }
        __syncwarp();  // the lines are read
        // One plane (BF16): dz is rounded to the products' operand type, 2^-8 of a term at
        // most and at random, as large an error as the outputs' own rounding.
        for (int pl = 0; pl < p.planes; ++pl) {
            put_bf16<true>(turn, 0, a);
            put_bf16<true>(turn, 1, b);
            __nv_bfloat16 *to = p.dz + (size_t)(2 * pl) * p.M * p.pitch + f;
            half_lines(p, turn, to, to + (size_t)p.M * p.pitch, p.pitch);
        }
    }

    // Columns c0 + 64 q .. + 63 as two halves a, b.
    __device__ __forceinline__ void pair(const GemmArgs &p, const Tile &t, const Turn &turn, int q,
                                         float (&a)[32], float (&b)[32]) {
        const int c = c0 + 64 * q;
        if (EPI == EPI_OUT && BF16) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                a[i] *= g;
                b[i] *= g;
            }
        }
        if (EPI == EPI_GLU) {
            glu(p, t, turn, c / 2, a, b);
        } else if (EPI == EPI_DGLU) {
            dglu(p, turn, c / 2, a, b);
        } else if (EPI == EPI_STATS) {
            stats(p, c, a);
            stats(p, c + 32, b);
        } else if (EPI == EPI_DZ) {
            // BF16 (one plane): dz is rounded to the products' operand type, up to 2^-8 of a term
            // and at random.  At 8,192 x 131,072 x 4,096 dx is 1.666e-3 of its norm off and
            // d_weight 1.657e-3, of which the outputs' own rounding is 1.665e-3 and 1.656e-3; a
            // second term would cost both products once more.
            dz_of(p, c, a);
            dz_of(p, c + 32, b);
            for (int pl = 0; pl < p.planes; ++pl) {
                put_bf16<true>(turn, 0, a);
                put_bf16<true>(turn, 1, b);
                lines(p, turn, p.dz + (size_t)pl * p.M * p.pitch + c, p.pitch);
            }
        } else if (BF16 && p.out && p.out_bf16 && !p.acc_in && p.vec && c + 64 <= p.N) {
            put_bf16<false>(turn, 0, a);
            put_bf16<false>(turn, 1, b);
            lines(p, turn, (__nv_bfloat16 *)p.out + t.batch * p.out_batch + c, p.N);
        } else if (BF16 && p.out && p.out_bf16 && !p.acc_in && !p.vec) {
            if (c >= p.N) return;
            put_bf16<false>(turn, 0, a);
            put_bf16<false>(turn, 1, b);
            ragged(p, turn, (__nv_bfloat16 *)p.out + t.batch * p.out_batch + c, p.N,
                   p.N - c < 64 ? p.N - c : 64);
        } else {
            if (c < p.N) out32(p, t, turn, c, a);
            if (c + 32 < p.N) out32(p, t, turn, c + 32, b);
        }
    }

    __device__ __forceinline__ void end(const GemmArgs &p, const Tile &t, int half) {
        if (EPI == EPI_STATS && live)
            p.part[(size_t)(2 * t.n + half) * p.M + row] = make_float2(mx, sum);
    }
};

__device__ __forceinline__ void add_pair(float &x, float &y, float ax, float ay) {
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
        "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(ax), "f"(ay));
}

inline int cdiv(long long a, long long b) { return (int)((a + b - 1) / b); }

// C = A B^T with A as three BF16 planes [3][p.M][a_inner], K-major, and B an fp32 weight
// [w_rows][width] (EPI_OUT: its rows are the contraction's, else its columns; EPI_GLU: two
// matrices of p.cols rows).
// p.k_blocks counts kW32Step; tiles have kW32Cols columns.
struct W32Operands {
    const void *a;
    int a_inner;
    const float *w;
    long long w_rows;
    int width;
};
constexpr int kW32Step = 32, kW32Cols = 128;
cudaError_t launch_w32(int epi, const GemmArgs &p, const W32Operands &o, cudaStream_t st);

}  // namespace kda
