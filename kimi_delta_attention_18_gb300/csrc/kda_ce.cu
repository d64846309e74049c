// Softmax cross entropy over a vocabulary from the last hidden states, without the
// logits ever being an array.  x [T][D], W [V][D], z = x W^T:
//     lse_t = log sum_v exp(z_tv),   loss_t = lse_t - z_t,y_t
//     dz_tv = d_loss_t (exp(z_tv - lse_t) - [v = y_t]),  dx = dz W,  dW = dz^T x.
//
// Forward: one product whose epilogue keeps, per row and 128 columns, the running
// maximum and the sum of exponentials (and picks the target's logit); a second
// kernel joins them.  Backward, per piece of the vocabulary: the piece's logits
// again, their dz in BF16 (the only array of that shape, one piece wide), then the
// two products that read it.  The logits cost 2 T V D operations once more; keeping
// them would cost T V words.
//
// All four products run in one persistent kernel on tcgen05 (gemm_kernel).  fp32
// operands are split into three BF16 terms (8 + 8 + 8 bits of the fp32 mantissa's
// 24) and the six products of terms whose weight is 2^-16 or more are accumulated,
// smallest first, so an fp32 problem is the same kernel with six times the steps.
#include <math.h>

#include "kda_internal.cuh"
#include "kda_sm100.cuh"

namespace kda {
namespace {

using namespace sm100;

constexpr int BM = 128, BN = 256, BK = 64;  // rows per CTA, columns, contraction per stage
constexpr int kABytes = BM * BK * 2, kBBytes = BN * BK * 2, kBox = 64 * BK * 2;
constexpr int kEpiWarps = 8, kThreads = 32 * (2 + kEpiWarps);
constexpr int kGroupRows = 2048;  // rows whose tiles share a sweep over the column tiles
constexpr long long kWaitLimit = 4000000000ll;  // ~2 s of SM clocks
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr uint32_t kTmemCols = 512;  // two 256-column accumulators

// Shared memory of a CTA alone (CTAS = 1) or of each CTA of a pair: a pair's CTAs
// hold half of B's rows each.
template <int CTAS>
struct Smem {
    static constexpr int stage = kABytes + kBBytes / CTAS, stages = CTAS == 1 ? 4 : 6;
    static constexpr int out = stages * stage;  // 4 KB per epilogue warp
    static constexpr int full = out + kEpiWarps * 4096, empty = full + 8 * stages, accf = empty + 8 * stages,
                         acce = accf + 16, fin = acce + 16, misc = fin + 8;
    static constexpr int bytes = misc + 16 + 1024;
    static_assert(bytes <= 227 * 1024, "shared memory budget");
};

enum { EPI_STATS = 0, EPI_DZ = 1, EPI_OUT = 2 };

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
    int k_blocks, splits, pairs;
    int chunk;                 // FINE: stages per accumulator
    int m_tiles, n_tiles, bn;  // set at the launch; bn: columns per tile, a multiple of 64
    int a_row0, b_row0;        // added to the operands' non-contraction coordinate
    int ak_row0, bk_row0;      // added to the contraction coordinate of MN-major operands
    // EPI_STATS, EPI_DZ
    Targets y;
    float2 *part;              // [2 n_tiles][M] (maximum, sum)
    float *z_y;                // [M]
    unsigned *ticket;          // cleared for the join kernel
    const float *lse, *d_loss;
    __nv_bfloat16 *dz;         // [planes][M][pitch]
    int pitch, planes;
    // EPI_OUT: value (+ acc_in) to acc_out [splits][M][N] fp32, or to out
    const float *acc_in;
    float *acc_out;
    void *out;
    int out_bf16, vec;
    int32_t *status;
};

// MN-major operand with 128-byte swizzle, as boxes of 64 elements x BK rows lay it
// down: 8 rows (along K) of 128 bytes form an atom, atoms follow each other along
// K (1024 bytes), boxes along M / N (8192 bytes).
__device__ __forceinline__ uint64_t umma_desc_mn_sw128(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)((BK * 128) >> 4) << 16;  // between 64-element boxes
    d |= (uint64_t)(1024 >> 4) << 32;        // between 8-row atoms along K
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
}

struct Tile {
    int m, n, split, kb0, kb1;
};
template <int CTAS>
__device__ __forceinline__ Tile tile_at(const GemmArgs &p, int w) {
    constexpr int G = kGroupRows / (BM * CTAS);
    Tile t;
    const int per = p.m_tiles * p.n_tiles;
    t.split = w / per;
    const int r = w - t.split * per, g = r / (G * p.n_tiles), q = r - g * G * p.n_tiles;
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
    // word `lane` of row r
    __device__ __forceinline__ float word(int r) const {
        float v;
        asm volatile("ld.shared.f32 %0, [%1];"
                     : "=f"(v)
                     : "r"(at + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + 4 * (lane & 3))
                     : "memory");
        return v;
    }
};

// One thread's part of the epilogue: a row and up to 128 of the tile's columns, taken
// 32 at a time.
template <int EPI>
struct Row {
    int row0;       // the warp's first row
    long long row;  // this thread's
    bool live;
    int c0;  // first column, in the launch's columns
    int y;   // the target's column (negative: none)
    float mx, sum, lse2, g;

    __device__ __forceinline__ void begin(const GemmArgs &p, const Tile &t, int first_row, int lane,
                                          int half) {
        row0 = first_row;
        row = first_row + lane;
        live = row < p.M;
        c0 = t.n * p.bn + half * 128;
        y = -1;
        mx = -INFINITY;
        sum = lse2 = g = 0.f;
        if (EPI != EPI_OUT && live) {
            y = p.y.at(row, t.n == 0 && half == 0);
            if (EPI == EPI_DZ) {
                lse2 = p.lse[row] * kLog2e;
                g = y >= 0 ? p.d_loss[row] : 0.f;
            }
            y = y >= 0 ? y - p.b_row0 : -1;
        }
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
        const bool narrow = p.out && p.out_bf16;
        float *o32 = p.out ? (float *)p.out : p.acc_out + (size_t)t.split * p.M * p.N;
        __nv_bfloat16 *o16 = (__nv_bfloat16 *)p.out;
        if (p.vec) {  // widths and bases of whole pieces: four columns are in or out together
            const int col = c + 4 * (turn.lane & 7);
#pragma unroll
            for (int it = 0; it < 8; ++it) {
                const long long r = row0 + turn.row(it);
                const uint4 u = turn.get(it);
                if (r >= p.M || col >= p.N) continue;
                const size_t at = (size_t)r * p.N + col;
                float4 f = make_float4(__uint_as_float(u.x), __uint_as_float(u.y),
                                       __uint_as_float(u.z), __uint_as_float(u.w));
                if (p.acc_in) {
                    const float4 a = *(const float4 *)(p.acc_in + at);
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
                if (c + turn.lane >= p.N) continue;
                const size_t at = (size_t)(row0 + r) * p.N + c + turn.lane;
                if (p.acc_in) f += p.acc_in[at];
                if (narrow) o16[at] = __float2bfloat16_rn(f);
                else o32[at] = f;
            }
        }
        __syncwarp();
    }

    // Columns c0 + 64 q .. + 63 as two halves a, b.
    __device__ __forceinline__ void pair(const GemmArgs &p, const Tile &t, const Turn &turn, int q,
                                         float (&a)[32], float (&b)[32]) {
        const int c = c0 + 64 * q;
        if (EPI == EPI_STATS) {
            stats(p, c, a);
            stats(p, c + 32, b);
        } else if (EPI == EPI_DZ) {
            dz_of(p, c, a);
            dz_of(p, c + 32, b);
            for (int pl = 0; pl < p.planes; ++pl) {
                put_bf16<true>(turn, 0, a);
                put_bf16<true>(turn, 1, b);
                lines(p, turn, p.dz + (size_t)pl * p.M * p.pitch + c, p.pitch);
            }
        } else if (p.out && p.out_bf16 && !p.acc_in && p.vec && c + 64 <= p.N) {
            put_bf16<false>(turn, 0, a);
            put_bf16<false>(turn, 1, b);
            lines(p, turn, (__nv_bfloat16 *)p.out + c, p.N);
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

__device__ __forceinline__ void add2(float &x, float &y, float ax, float ay) {
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
        "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(ax), "f"(ay));
}

// C = A B^T over tiles of 128 CTAS x 256 and steps of 64 along the contraction,
// one persistent CTA per SM, alone or in pairs (CTAS = 2):
//   warp 0   one thread loads the CTA's rows of both operands (TMA, 128-byte
//            swizzle) into four or six stages;
//   warp 1   one thread (of the pair's even CTA) issues four tcgen05.mma (128 CTAS x
//            256 x 16) per stage into one of two TMEM accumulators;
//   warps 2-9 the epilogue of the other accumulator: thread = row, 128 columns.
// A pair reads each operand row from shared memory once for 256 x 256 products
// instead of 128 x 256, and fetches a third fewer bytes from L2.
// An operand is K-major (its contraction index contiguous) or MN-major (its row
// index contiguous: W and x in dx = dz W, dz and x in dW = dz^T x), so nothing is
// transposed in memory.
//
// FINE, for results that are held in fp32 (lse, loss, and all of an fp32 problem):
// the tensor core adds each step of 16 to its accumulator with truncation, about
// 2^-24 of the sum per step and always towards zero, so a long contraction loses
// bits (at 7,168 measured 2.3e-6 of lse, against 1.4e-7 with fp32 arithmetic).  The
// accumulator is then handed over every `chunk` stages and added up, rounded to
// nearest, in the epilogue's registers, while the other accumulator fills.  16
// stages for BF16 operands (lse within 3e-7, no slower than one accumulator for
// all: 1.93 ms at 2,048 x 131,072 x 7,168), 8 for fp32 ones (gradients within
// 6e-7); 4 would cost a third more time, the hand-over then being longer than the
// products it overlaps.
constexpr int kChunkBf16 = 16, kChunkF32 = 8;

template <int EPI, bool A_MN, bool B_MN, bool FINE, int CTAS>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_kernel(const __grid_constant__ GemmArgs p, const __grid_constant__ CUtensorMap tm_a,
                const __grid_constant__ CUtensorMap tm_b) {
    using S = Smem<CTAS>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t sb = smem_addr(sm);
    auto full_bar = [&](int s) { return sb + S::full + 8 * s; };
    auto empty_bar = [&](int s) { return sb + S::empty + 8 * s; };
    auto accf_bar = [&](int i) { return sb + S::accf + 8 * (i & 1); };
    auto acce_bar = [&](int i) { return sb + S::acce + 8 * (i & 1); };
    volatile int *abort = (volatile int *)(sm + S::misc);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = CTAS == 1 ? 0 : (int)cluster_ctarank();
    const int work = p.m_tiles * p.n_tiles * p.splits;
    const int w0 = blockIdx.x / CTAS, wstep = gridDim.x / CTAS;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::stages; ++i) {
            mbar_init(full_bar(i), 1);
            mbar_init(empty_bar(i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(accf_bar(i), 1);
            mbar_init(acce_bar(i), kEpiWarps * CTAS);
        }
        mbar_init(sb + S::fin, 1);
        *abort = 0;
        mbar_fence_init();
    }
    if (warp == 0) tmem_alloc_group<CTAS>(sb + S::misc + 4, kTmemCols);
    tc_fence_before();
    __syncthreads();
    if (CTAS == 2) cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = *(volatile uint32_t *)(sm + S::misc + 4);
    griddep_wait();
    griddep_launch_dependents();
    if (EPI == EPI_STATS && blockIdx.x == 0 && threadIdx.x == 0) *p.ticket = 0;

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t ta = reinterpret_cast<uint64_t>(&tm_a);
            const uint64_t tb = reinterpret_cast<uint64_t>(&tm_b);
            const int boxes = (p.bn / CTAS + 63) / 64;  // of B
            int it = 0;
            bool ok = true;
            for (int w = w0; w < work && ok; w += wstep) {
                const Tile t = tile_at<CTAS>(p, w);
                const int ar = (t.m * CTAS + rank) * BM + p.a_row0;
                const int br = t.n * p.bn + rank * (p.bn / CTAS) + p.b_row0;
                for (int pr = 0; pr < p.pairs && ok; ++pr) {
                    const int pa = term_a(pr, p.pairs), pb = term_b(pr, p.pairs);
                    for (int kb = t.kb0; kb < t.kb1; ++kb, ++it) {
                        const int s = it % S::stages;
                        ok = mbar_wait(empty_bar(s), ((it / S::stages) & 1) ^ 1, abort, kWaitLimit);
                        if (!ok) break;
                        const uint32_t a = sb + s * S::stage, b = a + kABytes;
                        uint32_t full = full_bar(s);
                        if (CTAS == 2) full = cluster_map(full, 0);  // the issuing CTA waits for
                                                                     // both CTAs' bytes
                        if (rank == 0)
                            mbar_arrive_expect_tx(full_bar(s), CTAS * (kABytes + boxes * kBox));
                        // boxes of 64 x 64: 64 rows of the contraction's 64, or the other
                        // way round
#pragma unroll
                        for (int i = 0; i < BM / 64; ++i)
                            tma_load_3d<CTAS>(a + i * kBox, ta, A_MN ? ar + 64 * i : kb * BK,
                                              A_MN ? kb * BK + p.ak_row0 : ar + 64 * i, pa, full);
                        for (int i = 0; i < boxes; ++i)
                            tma_load_3d<CTAS>(b + i * kBox, tb, B_MN ? br + 64 * i : kb * BK,
                                              B_MN ? kb * BK + p.bk_row0 : br + 64 * i, pb, full);
                    }
                }
            }
            if (*abort) {  // let the copies in flight land before the CTA exits
                if (rank == 0) {
                    volatile int never = 0;
                    for (int k = it > S::stages ? it - S::stages : 0; k < it; ++k)
                        mbar_wait(full_bar(k % S::stages), (k / S::stages) & 1, &never, kWaitLimit);
                } else {  // their barrier is the other CTA's
                    const long long t0 = clock64();
                    while (clock64() - t0 < 4000000) {
                    }
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            const uint32_t idesc = umma_idesc_bf16(BM * CTAS, p.bn) | (A_MN ? 1u << 15 : 0u) |
                                   (B_MN ? 1u << 16 : 0u);
            int it = 0, i = 0;
            bool ok = true;
            for (int w = w0; w < work && ok; w += wstep, ++i) {
                const Tile t = tile_at<CTAS>(p, w);
                const int steps = (t.kb1 - t.kb0) * p.pairs;
                int first = 0;  // stages in this accumulator
                for (int k = 0; k < steps; ++k, ++it, ++first) {
                    if (FINE && first == p.chunk) first = 0;
                    if (first == 0) {
                        if (k > 0) umma_commit_group<CTAS>(accf_bar(i++));
                        ok = CTAS == 1 ? mbar_wait(acce_bar(i), ((i >> 1) & 1) ^ 1, abort, kWaitLimit)
                                       : mbar_wait_cluster(acce_bar(i), ((i >> 1) & 1) ^ 1, abort,
                                                           kWaitLimit);
                        if (!ok) break;
                        tc_fence_after();
                    }
                    const int s = it % S::stages;
                    ok = mbar_wait(full_bar(s), (it / S::stages) & 1, abort, kWaitLimit);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t a = sb + s * S::stage, b = a + kABytes;
#pragma unroll
                    for (int kk = 0; kk < BK / 16; ++kk)
                        umma_bf16_group<CTAS>(tmem + BN * (i & 1),
                                              A_MN ? umma_desc_mn_sw128(a + kk * 2048)
                                                   : umma_desc_sw128(a + kk * 32, 1024),
                                              B_MN ? umma_desc_mn_sw128(b + kk * 2048)
                                                   : umma_desc_sw128(b + kk * 32, 1024),
                                              idesc, first + kk > 0);
                    umma_commit_group<CTAS>(empty_bar(s));
                }
                if (ok) umma_commit_group<CTAS>(accf_bar(i));
            }
            if (*abort) {  // products in flight complete before TMEM is freed
                umma_commit_group<CTAS>(sb + S::fin);
                volatile int never = 0;
                mbar_wait(sb + S::fin, 0, &never, kWaitLimit);
            }
        }
    } else {
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        const int chunks = min(4, max(0, p.bn / 32 - 4 * half));  // of 32 columns
        const Turn turn = {sb + S::out + (warp - 2) * 4096, lane};
        const uint32_t src = tmem + ((uint32_t)(32 * quarter) << 16) + 128 * half;
        int i = 0;  // accumulators taken
        auto full = [&]() {
            const bool ok =
                __all_sync(0xffffffffu, mbar_wait(accf_bar(i), (i >> 1) & 1, abort, kWaitLimit));
            tc_fence_after();
            return ok;
        };
        auto release = [&]() {  // the accumulator is in registers
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (CTAS == 1) mbar_arrive(acce_bar(i));
                else mbar_arrive_cluster(cluster_map(acce_bar(i), 0));
            }
            ++i;
        };
        bool ok = true;
        for (int w = w0; w < work && ok; w += wstep) {
            const Tile t = tile_at<CTAS>(p, w);
            Row<EPI> r;
            r.begin(p, t, (t.m * CTAS + rank) * BM + 32 * quarter, lane, half);
            __syncwarp();
            if constexpr (FINE) {
                float acc[4][32];
#pragma unroll
                for (int ch = 0; ch < 4; ++ch)
#pragma unroll
                    for (int j = 0; j < 32; ++j) acc[ch][j] = 0.f;
                const int steps = (t.kb1 - t.kb0) * p.pairs;
                for (int k = 0; k < steps && ok; k += p.chunk) {
                    ok = full();
                    if (!ok) break;
#pragma unroll
                    for (int ch = 0; ch < 4; ++ch) {
                        if (ch >= chunks) break;
                        float v[32];
                        tmem_ld32(src + BN * (i & 1) + 32 * ch, v);
#pragma unroll
                        for (int j = 0; j < 32; j += 2)
                            add2(acc[ch][j], acc[ch][j + 1], v[j], v[j + 1]);
                    }
                    release();
                }
                if (!ok) break;
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    if (2 * q < chunks) r.pair(p, t, turn, q, acc[2 * q], acc[2 * q + 1]);
            } else {
                ok = full();
                if (!ok) break;
                const uint32_t at = src + BN * (i & 1);
                if (chunks == 0) release();
#pragma unroll 1
                for (int ch = 0; ch < chunks; ch += 2) {
                    float v[64];
                    __syncwarp();
                    tmem_ld64(at + 32 * ch, v);
                    if (ch == chunks - 2) release();
                    r.pair(p, t, turn, ch / 2, *(float (*)[32])v, *(float (*)[32])(v + 32));
                }
            }
            r.end(p, t, half);
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (CTAS == 2) cluster_sync_all();  // the pair's products read both CTAs' memory
    if (threadIdx.x == 0 && *abort) dev_fail(p.status, KDA_ERR_TIMEOUT);
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc_group<CTAS>(tmem, kTmemCols);
    }
}

// Joins the row statistics: 8 rows per block and 128 slices of the partial sums, each
// slice in order, then the slices pairwise.  Writes lse and the loss (0 where the
// target is ignored), and the mean over the others: per block (sum, count), added up
// in block order by the block that finishes last.
constexpr int kJoinRows = 8, kJoinSlices = 128;
__global__ void __launch_bounds__(kJoinRows * kJoinSlices)
    ce_join_kernel(const float2 *part, int parts, int M, Targets y, const float *z_y, float *loss,
                   float *lse, float *mean, float2 *sums, unsigned *ticket) {
    __shared__ float2 sh[kJoinSlices][kJoinRows + 1];
    __shared__ bool last;
    griddep_wait();
    griddep_launch_dependents();
    const int r = threadIdx.x % kJoinRows, sl = threadIdx.x / kJoinRows, lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * kJoinRows + r;
    auto join = [](float2 a, float2 b) {
        const float m = fmaxf(a.x, b.x);
        if (m == -INFINITY) return make_float2(m, a.y + b.y);
        return make_float2(m, a.y * exp2f((a.x - m) * kLog2e) + b.y * exp2f((b.x - m) * kLog2e));
    };
    float2 v = make_float2(-INFINITY, 0.f);
    if (row < M) {
#pragma unroll 8
        for (int q = sl; q < parts; q += kJoinSlices) v = join(v, part[(size_t)q * M + row]);
    }
    sh[sl][r] = v;
    __syncthreads();
    for (int o = kJoinSlices / 2; o > 0; o >>= 1) {
        if (sl < o) sh[sl][r] = join(sh[sl][r], sh[sl + o][r]);
        __syncthreads();
    }
    if (threadIdx.x < 32) {
        float l = 0.f, n = 0.f;
        if (sl == 0 && row < M) {
            v = sh[0][r];
            const float e = v.x + kLn2 * log2f(v.y);
            if (y.at(row, false) >= 0) {
                l = e - z_y[row];
                n = 1.f;
            }
            lse[row] = e;
            loss[row] = l;
        }
        if (mean) {
#pragma unroll
            for (int o = kJoinRows / 2; o > 0; o >>= 1) {
                l += __shfl_xor_sync(0xffffffffu, l, o);
                n += __shfl_xor_sync(0xffffffffu, n, o);
            }
            if (lane == 0) {
                sums[blockIdx.x] = make_float2(l, n);
                __threadfence();
                last = atomicAdd(ticket, 1u) == gridDim.x - 1;
            }
        }
    }
    if (!mean) return;
    __syncthreads();
    if (!last) return;
    __threadfence();
    float2 s = make_float2(0.f, 0.f);
    for (int b = threadIdx.x; b < (int)gridDim.x; b += kJoinRows * kJoinSlices) {
        const float2 u = __ldcg(&sums[b]);
        s.x += u.x;
        s.y += u.y;
    }
    float2 *flat = &sh[0][0];  // kJoinSlices (kJoinRows + 1) entries
    __syncthreads();
    flat[threadIdx.x] = s;
    __syncthreads();
    for (int o = kJoinRows * kJoinSlices / 2; o > 0; o >>= 1) {
        if (threadIdx.x < o) {
            flat[threadIdx.x].x += flat[threadIdx.x + o].x;
            flat[threadIdx.x].y += flat[threadIdx.x + o].y;
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) *mean = flat[0].y > 0.f ? flat[0].x / flat[0].y : 0.f;  // none counts: 0
}

// Rows of an operand as `planes` BF16 terms with a pitch of whole 16-byte pieces
// (zeros past the width): fp32 operands, and BF16 ones whose rows a tensor map
// cannot address.
// x and W in one launch.
template <typename T>
__global__ void __launch_bounds__(256)
    pack_kernel(const T *x, long long x_rows, __nv_bfloat16 *xp, const T *w, long long w_rows,
                __nv_bfloat16 *wp, int D, int pitch, int planes) {
    griddep_wait();
    griddep_launch_dependents();
    const int pieces = pitch / 8;
    const long long total = (x_rows + w_rows) * pieces;
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
        long long r = i / pieces;
        const int c = (int)(i - r * pieces) * 8;
        const bool second = r >= x_rows;
        if (second) r -= x_rows;
        const T *src = second ? w : x;
        __nv_bfloat16 *dst = second ? wp : xp;
        const long long rows = second ? w_rows : x_rows;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = c + j < D ? act_ld(src, (size_t)(r * D + c + j)) : 0.f;
        for (int pl = 0; pl < planes; ++pl) {
            uint32_t u[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                u[k] = pack_bf16x2(v[2 * k], v[2 * k + 1]);
                v[2 * k] -= __uint_as_float(u[k] << 16);
                v[2 * k + 1] -= __uint_as_float(u[k] & 0xffff0000u);
            }
            *(uint4 *)(dst + ((size_t)pl * rows + r) * pitch + c) = make_uint4(u[0], u[1], u[2], u[3]);
        }
    }
}

// out = sum over splits of acc[s], in order.
template <typename T>
__global__ void __launch_bounds__(256) split_sum_kernel(const float *acc, T *out, long long n,
                                                        int splits) {
    griddep_wait();
    griddep_launch_dependents();
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) {
        float s = 0.f;
#pragma unroll 4
        for (int k = 0; k < splits; ++k) s += acc[(size_t)k * n + i];
        act_st(out, (size_t)i, s);
    }
}

// ------------------------------------------------------------------ host side
size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }
int cdiv(long long a, long long b) { return (int)((a + b - 1) / b); }

// Width of dz's buffer: at most 512 MiB of BF16 (or three fp32 terms) in whole
// column tiles, unless the caller says.
int piece_cols(const kda_ce_desc_t *d, int planes) {
    const long long all = (long long)cdiv(d->vocab, BN) * BN;
    long long cols = d->piece;
    if (cols <= 0) {
        cols = (512ll << 20) / ((long long)(d->tokens > 0 ? d->tokens : 1) * planes * 2);
        if (cols < 4096) cols = 4096;
        if (cols < all) {  // equal pieces
            const int n = cdiv(all, cols);
            cols = cdiv(all, n);
        }
    }
    cols = (long long)cdiv(cols, BN) * BN;
    return (int)(cols < all ? cols : all);
}

struct Layout {
    int planes, pairs, chunk, pitch, piece, pieces, dx_splits;
    bool pack;
    size_t xp, wp, part, zy, sums, dz, acc, total;
};

// Pieces of the workspace.  pack: operands are copied (fp32 terms, or BF16 rows
// whose width is no multiple of the 16 bytes that a tensor map needs).
Layout layout_for(const kda_ce_desc_t *d, bool backward) {
    Layout l = {};
    const bool pack = d->act_dtype == KDA_DTYPE_F32 || d->width % 8 != 0;
    const size_t T = d->tokens, V = d->vocab;
    l.planes = d->act_dtype == KDA_DTYPE_F32 ? 3 : 1;
    l.pairs = l.planes == 3 ? 6 : 1;
    l.chunk = l.planes == 3 ? kChunkF32 : kChunkBf16;
    // whole 128-byte lines: with rows of 1,040 bytes the copies of 128-byte boxes ran at
    // half the rate
    l.pitch = (d->width + 63) / 64 * 64;
    l.pack = pack;
    l.xp = pack ? round256(T * l.pitch * l.planes * 2) : 0;
    l.wp = pack ? round256(V * l.pitch * l.planes * 2) : 0;
    if (!backward) {
        l.part = round256((size_t)2 * cdiv(V, BN) * T * sizeof(float2));
        l.zy = round256(T * 4);
        l.sums = round256((T / kJoinRows + 1) * sizeof(float2)) + 256;
    } else {
        l.piece = piece_cols(d, l.planes);
        l.pieces = cdiv(V, l.piece);
        l.dz = round256(T * l.piece * l.planes * 2);
        // dx has few tiles when T and D are small: its contraction over the
        // vocabulary is then split so that every SM has a share
        const int tiles = cdiv(T, BM) * cdiv(d->width, BN), n = device_sms();
        l.dx_splits = 1;
        if (l.pieces == 1 && tiles > 0 && tiles < n) {
            l.dx_splits = n / tiles;
            const int most = l.piece / BK / 4;  // at least four steps each
            if (l.dx_splits > most) l.dx_splits = most < 1 ? 1 : most;
        }
        if (l.pieces > 1 || l.dx_splits > 1)
            l.acc = round256((size_t)l.dx_splits * T * d->width * 4);
    }
    l.total = l.xp + l.wp + l.part + l.zy + l.sums + l.dz + l.acc;
    return l;
}

kda_status_t check(const kda_ce_desc_t *d) {
    if (!d) return KDA_ERR_INVALID_ARG;
    if (d->tokens < 0 || d->vocab < 1 || d->width < 1 || d->piece < 0) return KDA_ERR_INVALID_ARG;
    if (d->act_dtype != KDA_DTYPE_F32 && d->act_dtype != KDA_DTYPE_BF16) return KDA_ERR_UNSUPPORTED;
    if (d->id_dtype != KDA_ID_I32 && d->id_dtype != KDA_ID_I64) return KDA_ERR_UNSUPPORTED;
    // tile and coordinate arithmetic is 32-bit
    if (d->tokens > (1 << 24) || d->vocab > (1 << 24) || d->width > (1 << 17))
        return KDA_ERR_UNSUPPORTED;
    if ((long long)cdiv(d->tokens, BM) * cdiv(d->vocab, BN) > (1ll << 30)) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

// An operand [planes][rows][pitch] in boxes of 64 x 64 elements, for either of its
// indexes as the contraction's.
bool encode(CUtensorMap *tm, const void *base, int inner, long long rows, int planes) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)rows, (cuuint64_t)planes};
    const cuuint64_t strides[2] = {(cuuint64_t)inner * 2, (cuuint64_t)(rows * inner) * 2};
    const cuuint32_t box[3] = {64, 64, 1}, estr[3] = {1, 1, 1};
    return enc(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int EPI, bool A_MN, bool B_MN, bool FINE, int CTAS>
cudaError_t start_gemm(GemmArgs p, const CUtensorMap &ta, const CUtensorMap &tb, int n,
                       cudaStream_t st) {
    const auto kernel = gemm_kernel<EPI, A_MN, B_MN, FINE, CTAS>;
    cudaError_t e = set_max_dynamic_smem((const void *)kernel, Smem<CTAS>::bytes);
    if (e != cudaSuccess) return e;
    p.m_tiles = cdiv(p.M, BM * CTAS);
    p.n_tiles = cdiv(p.N, BN);
    p.bn = cdiv(cdiv(p.N, p.n_tiles), 64) * 64;  // tiles of about equal width
    const long long work = (long long)p.m_tiles * p.n_tiles * p.splits;
    const int groups = (int)(work < n / CTAS ? work : n / CTAS);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(groups * CTAS);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Smem<CTAS>::bytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CTAS;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CTAS == 1 ? 1 : 2;
    return cudaLaunchKernelEx(&cfg, kernel, p, ta, tb);
}

// Pairs of CTAs unless single ones finish in fewer rounds over the SMs (few rows:
// a pair's second half would be idle).
bool use_pairs(const GemmArgs &p, int n) {
    const long long cols = (long long)cdiv(p.N, BN) * p.splits;
    const long long one = (cdiv(p.M, BM) * cols + n - 1) / n;
    const long long two = (cdiv(p.M, 2 * BM) * cols + n / 2 - 1) / (n / 2);
    return n >= 2 && two <= one;
}

template <int EPI, bool A_MN, bool B_MN, bool FINE>
cudaError_t run_gemm(const GemmArgs &p, const CUtensorMap &ta, const CUtensorMap &tb,
                     cudaStream_t st) {
    const int n = device_sms();
    return use_pairs(p, n) ? start_gemm<EPI, A_MN, B_MN, FINE, 2>(p, ta, tb, n, st)
                           : start_gemm<EPI, A_MN, B_MN, FINE, 1>(p, ta, tb, n, st);
}
// The backward's products: in fp32 problems FINE, in BF16 ones (whose results are
// rounded to 2^-8 of their value) not.
template <int EPI, bool A_MN, bool B_MN>
cudaError_t run_gemm(const GemmArgs &p, bool fine, const CUtensorMap &ta, const CUtensorMap &tb,
                     cudaStream_t st) {
    return fine ? run_gemm<EPI, A_MN, B_MN, true>(p, ta, tb, st)
                : run_gemm<EPI, A_MN, B_MN, false>(p, ta, tb, st);
}

cudaError_t run_pack(const kda_ce_desc_t *d, const Layout &l, const void *x, const void *w,
                     uint8_t *ws, cudaStream_t st) {
    __nv_bfloat16 *xp = (__nv_bfloat16 *)ws, *wp = (__nv_bfloat16 *)(ws + l.xp);
    const long long T = d->tokens, V = d->vocab;
    const long long need = ((T + V) * (l.pitch / 8) + 255) / 256, most = 16ll * device_sms();
    const dim3 grid((unsigned)(need < most ? need : most));
    if (d->act_dtype == KDA_DTYPE_F32)
        return launch_dependent(pack_kernel<float>, grid, dim3(256), 0, st, (const float *)x, T, xp,
                                (const float *)w, V, wp, d->width, l.pitch, l.planes);
    return launch_dependent(pack_kernel<__nv_bfloat16>, grid, dim3(256), 0, st,
                            (const __nv_bfloat16 *)x, T, xp, (const __nv_bfloat16 *)w, V, wp,
                            d->width, l.pitch, l.planes);
}

bool bad_ids(const kda_ce_desc_t *d, const void *ids) {
    return !ids || (uintptr_t)ids % (d->id_dtype == KDA_ID_I64 ? 8 : 4);
}
bool bad16(const void *p) { return !p || ((uintptr_t)p & 15u); }
bool bad_f32(const void *p) { return !p || ((uintptr_t)p & 3u); }
bool bad_act(const kda_ce_desc_t *d, const void *p) {
    return !p || (uintptr_t)p % (d->act_dtype == KDA_DTYPE_BF16 ? 2 : 4);
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

size_t kda_linear_ce_workspace_size(const kda_ce_desc_t *desc, int32_t backward) {
    if (check(desc) != KDA_OK || desc->tokens == 0) return 0;
    return layout_for(desc, backward != 0).total;
}

kda_status_t kda_linear_ce_forward(const kda_ce_desc_t *desc, const void *x, const void *weight,
                                   const void *targets, float *loss, float *lse, float *mean,
                                   void *workspace, size_t workspace_bytes, int32_t *dev_status,
                                   void *stream) {
    kda_status_t rc = check(desc);
    if (rc != KDA_OK) return rc;
    cudaStream_t st = (cudaStream_t)stream;
    if (((uintptr_t)mean & 3u) || ((uintptr_t)dev_status & 3u)) return KDA_ERR_INVALID_ARG;
    if (desc->tokens == 0) {
        if (mean && cudaMemsetAsync(mean, 0, 4, st) != cudaSuccess) return KDA_ERR_CUDA;
        return KDA_OK;
    }
    if (bad16(x) || bad16(weight) || bad_ids(desc, targets) || bad_f32(loss) ||
        bad_f32(lse))
        return KDA_ERR_INVALID_ARG;
    const Layout l = layout_for(desc, false);
    if (!workspace || workspace_bytes < l.total || ((uintptr_t)workspace & 15u))
        return KDA_ERR_WORKSPACE;
    uint8_t *ws = (uint8_t *)workspace;
    const __nv_bfloat16 *xp = (const __nv_bfloat16 *)x, *wp = (const __nv_bfloat16 *)weight;
    float2 *part = (float2 *)(ws + l.xp + l.wp);
    float *zy = (float *)(ws + l.xp + l.wp + l.part);
    float2 *sums = (float2 *)(ws + l.xp + l.wp + l.part + l.zy);
    unsigned *ticket = (unsigned *)(ws + l.total - 256);
    if (l.pack) {
        if (run_pack(desc, l, x, weight, ws, st) != cudaSuccess) return KDA_ERR_CUDA;
        xp = (const __nv_bfloat16 *)ws;
        wp = (const __nv_bfloat16 *)(ws + l.xp);
    }
    const int inner = l.pack ? l.pitch : desc->width;
    CUtensorMap ta, tb;
    if (!encode(&ta, xp, inner, desc->tokens, l.planes) ||
        !encode(&tb, wp, inner, desc->vocab, l.planes))
        return KDA_ERR_CUDA;
    GemmArgs p = {};
    p.M = desc->tokens;
    p.N = desc->vocab;
    p.k_blocks = cdiv(desc->width, BK);
    p.splits = 1;
    p.pairs = l.pairs;
    p.chunk = l.chunk;
    p.y = {targets, desc->id_dtype == KDA_ID_I64, desc->vocab, desc->ignore_index, dev_status};
    p.part = part;
    p.z_y = zy;
    p.ticket = ticket;
    p.status = dev_status;
    if (run_gemm<EPI_STATS, false, false, true>(p, ta, tb, st) != cudaSuccess) return KDA_ERR_CUDA;
    if (launch_dependent(ce_join_kernel, dim3(cdiv(p.M, kJoinRows)), dim3(kJoinRows * kJoinSlices), 0, st,
                         (const float2 *)part, 2 * cdiv(p.N, BN), p.M, p.y, (const float *)zy, loss, lse,
                         mean, sums, ticket) != cudaSuccess)
        return KDA_ERR_CUDA;
    return KDA_OK;
}

kda_status_t kda_linear_ce_backward(const kda_ce_desc_t *desc, const void *x, const void *weight,
                                    const void *targets, const float *lse, const float *d_loss,
                                    void *dx, void *d_weight, void *workspace,
                                    size_t workspace_bytes, int32_t *dev_status, void *stream) {
    kda_status_t rc = check(desc);
    if (rc != KDA_OK) return rc;
    cudaStream_t st = (cudaStream_t)stream;
    const size_t size = desc->act_dtype == KDA_DTYPE_BF16 ? 2 : 4;
    if ((dx && bad_act(desc, dx)) || (d_weight && bad_act(desc, d_weight)) ||
        ((uintptr_t)dev_status & 3u))
        return KDA_ERR_INVALID_ARG;
    if (desc->tokens == 0) {
        if (d_weight && cudaMemsetAsync(d_weight, 0, (size_t)desc->vocab * desc->width * size, st) !=
                            cudaSuccess)
            return KDA_ERR_CUDA;
        return KDA_OK;
    }
    if (bad16(x) || bad16(weight) || bad_ids(desc, targets) || bad_f32(lse) ||
        bad_f32(d_loss))
        return KDA_ERR_INVALID_ARG;
    if (!dx && !d_weight) return KDA_OK;
    const Layout l = layout_for(desc, true);
    if (!workspace || workspace_bytes < l.total || ((uintptr_t)workspace & 15u))
        return KDA_ERR_WORKSPACE;
    uint8_t *ws = (uint8_t *)workspace;
    const __nv_bfloat16 *xp = (const __nv_bfloat16 *)x, *wp = (const __nv_bfloat16 *)weight;
    __nv_bfloat16 *dz = (__nv_bfloat16 *)(ws + l.xp + l.wp);
    float *acc = (float *)(ws + l.xp + l.wp + l.dz);
    if (l.pack) {
        if (run_pack(desc, l, x, weight, ws, st) != cudaSuccess) return KDA_ERR_CUDA;
        xp = (const __nv_bfloat16 *)ws;
        wp = (const __nv_bfloat16 *)(ws + l.xp);
    }
    const int T = desc->tokens, V = desc->vocab, D = desc->width;
    const bool fine = l.planes > 1;
    const int inner = l.pack ? l.pitch : D;
    CUtensorMap tx, tw, tz;
    if (!encode(&tx, xp, inner, T, l.planes) || !encode(&tw, wp, inner, V, l.planes) ||
        !encode(&tz, dz, l.piece, T, l.planes))
        return KDA_ERR_CUDA;
    for (int k = 0; k < l.pieces; ++k) {
        const int v0 = k * l.piece, cols = V - v0 < l.piece ? V - v0 : l.piece;
        GemmArgs p = {};
        p.status = dev_status;
        p.pairs = l.pairs;
        p.chunk = l.chunk;
        p.splits = 1;
        p.M = T;
        p.N = cols;
        p.k_blocks = cdiv(D, BK);
        p.b_row0 = v0;
        p.y = {targets, desc->id_dtype == KDA_ID_I64, V, desc->ignore_index, dev_status};
        p.lse = lse;
        p.d_loss = d_loss;
        p.dz = dz;
        p.pitch = l.piece;
        p.planes = l.planes;
        if (run_gemm<EPI_DZ, false, false>(p, fine, tx, tw, st) != cudaSuccess) return KDA_ERR_CUDA;
        if (dx) {
            GemmArgs q = {};
            q.status = dev_status;
            q.pairs = l.pairs;
            q.chunk = l.chunk;
            q.splits = l.dx_splits;
            q.M = T;
            q.N = D;
            q.k_blocks = cdiv(cols, BK);
            q.bk_row0 = v0;
            q.acc_in = k > 0 ? acc : nullptr;
            if (l.dx_splits == 1 && k == l.pieces - 1) q.out = dx;
            else q.acc_out = acc;
            q.out_bf16 = size == 2;
            q.vec = D % 8 == 0 && ((uintptr_t)dx & 15u) == 0;
            if (q.splits > q.k_blocks) return KDA_ERR_CUDA;
            if (run_gemm<EPI_OUT, false, true>(q, fine, tz, tw, st) != cudaSuccess)
                return KDA_ERR_CUDA;
            if (l.dx_splits > 1) {
                const long long n = (long long)T * D, need = (n + 255) / 256, most = 16ll * device_sms();
                const dim3 grid((unsigned)(need < most ? need : most));
                const cudaError_t e =
                    size == 2 ? launch_dependent(split_sum_kernel<__nv_bfloat16>, grid, dim3(256), 0,
                                                 st, (const float *)acc, (__nv_bfloat16 *)dx, n,
                                                 l.dx_splits)
                              : launch_dependent(split_sum_kernel<float>, grid, dim3(256), 0, st,
                                                 (const float *)acc, (float *)dx, n, l.dx_splits);
                if (e != cudaSuccess) return KDA_ERR_CUDA;
            }
        }
        if (d_weight) {
            GemmArgs q = {};
            q.status = dev_status;
            q.pairs = l.pairs;
            q.chunk = l.chunk;
            q.splits = 1;
            q.M = cols;
            q.N = D;
            q.k_blocks = cdiv(T, BK);
            q.out = (uint8_t *)d_weight + (size_t)v0 * D * size;
            q.out_bf16 = size == 2;
            q.vec = D % 8 == 0 && ((uintptr_t)d_weight & 15u) == 0;
            if (run_gemm<EPI_OUT, true, true>(q, fine, tz, tx, st) != cudaSuccess)
                return KDA_ERR_CUDA;
        }
    }
    return KDA_OK;
}

}  // extern "C"
