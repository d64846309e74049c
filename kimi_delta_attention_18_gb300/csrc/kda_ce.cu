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
// All four products run in persistent kernels on tcgen05.  fp32 operands are split
// into three BF16 terms (8 + 8 + 8 bits of the fp32 mantissa's 24) and the six
// products of terms whose weight is 2^-16 or more are accumulated, smallest first.
// They are stored as such terms first; only W, where there are few tokens, is split on
// its way through shared memory instead (kda_ce_w32.cu).
//
// Measured on GB300: gradient of 8,192 x 131,072 x 4,096 BF16 15.2 ms = 1.74 PFLOP/s of
// its 6 T V D, in a loop under the power cap (cuBLAS sustains 1.73 there; each product
// alone takes 1.14-1.17 ms per 32,768 columns, 1.89-1.93 PFLOP/s); losses of 256 x
// 131,072 x 7,168 325 us (5.8 TB/s of W, 1.48 PFLOP/s: near both bounds); fp32 gradient
// of 777 x 10,007 x 515 203 us.
#include <float.h>
#include <math.h>

#include "kda_ce_gemm.cuh"

namespace kda {
namespace {

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
// FINE, for results that are held in fp32 (lse, loss, and all of an fp32 problem) and for
// long contractions: the tensor core adds each step of 16 to its accumulator with
// truncation, up to 2^-23 of the sum per step and always towards zero, so bits are lost
// (at 7,168 measured 2.3e-6 of lse, against 1.4e-7 with fp32 arithmetic).  The accumulator
// is then handed over every `chunk` stages and added up, rounded to nearest, in the
// epilogue's registers, while the other accumulator fills.  16
// stages for BF16 operands (lse within 3e-7, no slower than one accumulator for
// all: 1.93 ms at 2,048 x 131,072 x 7,168), 8 for fp32 ones (gradients within 6e-7).
constexpr int kChunkBf16 = 16, kChunkF32 = 8;
// BF16 gradients: one accumulator up to so many stages (32,768 elements), which leaves the
// sum 2e-4 short at worst (4e-7 a stage where all terms have one sign; the output's own
// rounding is 1.7e-3 of the norm); FINE beyond (d_weight over 2^20 tokens was 6.5e-3 short).
// FINE for all is 4-7 % slower (8,192 x 131,072 x 4,096: 15.2 and 15.8 ms; its epilogue has a
// whole tile in registers), but not for long sums (d_weight of 81,920 x 8,192 x 2,048, 1,280
// stages: 3.60 ms with one accumulator, 3.52 FINE).
constexpr int kLongStages = 512;

template <int EPI, bool A_MN, bool B_MN, bool FINE, bool BF16, int CTAS>
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
            // boxes of 64 x 64 of B; K-major ones come in twos
            const int boxes = B_MN ? (p.bn / CTAS + 63) / 64 : 2 * ((p.bn / CTAS + 127) / 128);
            int it = 0;
            bool ok = true;
            for (int w = w0; w < work && ok; w += wstep) {
                const Tile t = tile_at<CTAS>(p, w);
                const int ar = (t.m * CTAS + rank) * BM;
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
                        // K-major: boxes of 128 rows x 64 of the contraction; MN-major: of
                        // 64 rows of the contraction x 64
                        if (A_MN) {
#pragma unroll
                            for (int i = 0; i < BM / 64; ++i)
                                tma_load_3d<CTAS>(a + i * kBox, ta, ar + 64 * i,
                                                  kb * BK, pa, full);
                        } else {
                            tma_load_3d<CTAS>(a, ta, kb * BK, ar, pa, full);
                        }
                        for (int i = 0; i < boxes; i += B_MN ? 1 : 2)
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
                                              A_MN ? umma_desc_mn_sw128(a + kk * 2048, BK)
                                                   : umma_desc_sw128(a + kk * 32, 1024),
                                              B_MN ? umma_desc_mn_sw128(b + kk * 2048, BK)
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
                else mbar_arrive_tmem(cluster_map(acce_bar(i), 0));
            }
            ++i;
        };
        bool ok = true;
        for (int w = w0; w < work && ok; w += wstep) {
            const Tile t = tile_at<CTAS>(p, w);
            Row<EPI, BF16> r;
            r.begin(p, t, (t.m * CTAS + rank) * BM + 32 * quarter, lane, half, 128);
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

// Joins the row statistics: ROWS rows per block, the partial sums in as many slices as
// its 1,024 threads allow, each slice in order, then the slices pairwise.  Writes lse and
// the loss (0 where the target is ignored), and the mean over the others: per block (sum,
// count), added up in block order by the block that finishes last.
constexpr int kJoinThreads = 1024, kJoinFew = 8, kJoinMany = 32;
template <int ROWS>
__global__ void __launch_bounds__(kJoinThreads)
    ce_join_kernel(const float2 *part, int parts, int M, Targets y, const float *z_y, float *loss,
                   float *lse, float *mean, float2 *sums, unsigned *ticket) {
    constexpr int kSlices = kJoinThreads / ROWS;
    __shared__ float2 sh[kSlices][ROWS + 1];
    __shared__ bool last;
    griddep_wait();
    griddep_launch_dependents();
    const int r = threadIdx.x % ROWS, sl = threadIdx.x / ROWS, lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * ROWS + r;
    auto join = [](float2 a, float2 b) {
        const float m = fmaxf(a.x, b.x);
        if (m == -INFINITY) return make_float2(m, a.y + b.y);
        return make_float2(m, a.y * exp2f((a.x - m) * kLog2e) + b.y * exp2f((b.x - m) * kLog2e));
    };
    float2 v = make_float2(-INFINITY, 0.f);
    if (row < M) {
#pragma unroll 8
        for (int q = sl; q < parts; q += kSlices) v = join(v, part[(size_t)q * M + row]);
    }
    sh[sl][r] = v;
    __syncthreads();
    for (int o = kSlices / 2; o > 0; o >>= 1) {
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
            for (int o = ROWS / 2; o > 0; o >>= 1) {
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
    for (int b = threadIdx.x; b < (int)gridDim.x; b += kJoinThreads) {
        const float2 u = __ldcg(&sums[b]);
        s.x += u.x;
        s.y += u.y;
    }
    float2 *flat = &sh[0][0];  // kSlices (ROWS + 1) entries
    __syncthreads();
    flat[threadIdx.x] = s;
    __syncthreads();
    for (int o = kJoinThreads / 2; o > 0; o >>= 1) {
        if (threadIdx.x < o) {
            flat[threadIdx.x].x += flat[threadIdx.x + o].x;
            flat[threadIdx.x].y += flat[threadIdx.x + o].y;
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) *mean = flat[0].y > 0.f ? flat[0].x / flat[0].y : 0.f;  // none counts: 0
}

// The eight BF16 values from element e of p (a 16-byte base, n elements).
__device__ __forceinline__ uint4 eight_from(const __nv_bfloat16 *p, long long e, long long n) {
    uint32_t v[8] = {};
    const long long a = e & ~7ll;
    if (a + 16 <= n) {
        *(uint4 *)v = *(const uint4 *)(p + a);
        *(uint4 *)(v + 4) = *(const uint4 *)(p + a + 8);
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (a + j < n) v[j / 2] |= (uint32_t)((const uint16_t *)p)[a + j] << (16 * (j & 1));
    }
    const int by = (int)(e & 7);
#pragma unroll
    for (int k = 0; k < 6; ++k) v[k] = by & 4 ? v[k + 2] : v[k];
#pragma unroll
    for (int k = 0; k < 5; ++k) v[k] = by & 2 ? v[k + 1] : v[k];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = by & 1 ? __funnelshift_r(v[k], v[k + 1], 16) : v[k];
    return make_uint4(v[0], v[1], v[2], v[3]);
}

// Rows of x and, if w_rows, of W as `planes` BF16 terms with a pitch of whole 128-byte
// lines (zeros past the width): fp32 operands, and BF16 rows whose width is no multiple
// of the 16 bytes that a tensor map needs.  With targets, rows of x whose target is
// ignored become zeros: dW is a sum over all rows, and what a padded position holds
// (NaN perhaps) has no part in it.  With d_loss the first block only finds dz's unit, from
// the largest of its magnitudes that counts (1 if none does).
template <typename T>
__global__ void __launch_bounds__(256)
    pack_kernel(const T *x, long long x_rows, __nv_bfloat16 *xp, const T *w, long long w_rows,
                __nv_bfloat16 *wp, int D, int pitch, int planes, Targets y, const float *d_loss,
                float *unit) {
    griddep_wait();
    griddep_launch_dependents();
    if (d_loss && blockIdx.x == 0) {
        __shared__ float sh[8];
        float m = 0.f;
#pragma unroll 4
        for (long long r = threadIdx.x; r < x_rows; r += 256) {
            const float g = fabsf(d_loss[r]);
            m = g <= FLT_MAX && y.at(r, false) >= 0 ? fmaxf(m, g) : m;
        }
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (threadIdx.x % 32 == 0) sh[threadIdx.x / 32] = m;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int k = 1; k < 8; ++k) m = fmaxf(m, sh[k]);
            // from 2 on its significand alone: dz then keeps d_loss's own exponents (a row of
            // 1e-20 next to one of 1e30 would be zero in units of 1e30)
            if (m >= 2.f) m = __int_as_float((__float_as_int(m) & 0x7fffff) | 0x3f800000);
            *unit = m >= FLT_MIN ? m : 1.f;
        }
        return;
    }
    const int first = d_loss ? 1 : 0;  // the block that copies first
    const int pieces = pitch / 8;
    const long long total = (x_rows + w_rows) * pieces;
    const long long step = (gridDim.x - first) * 256ll;
    for (long long i = (blockIdx.x - first) * 256ll + threadIdx.x; i < total; i += step) {
        long long r = i / pieces;
        const int c = (int)(i - r * pieces) * 8;
        const bool second = r >= x_rows;
        if (second) r -= x_rows;
        const T *src = second ? w : x;
        __nv_bfloat16 *dst = second ? wp : xp;
        const long long rows = second ? w_rows : x_rows;
        if constexpr (sizeof(T) == 2) {
            uint4 u = make_uint4(0, 0, 0, 0);
            if (c < D && !(!second && y.ids && y.at(r, false) < 0)) {
                u = eight_from(src, r * D + c, rows * D);
                uint32_t *word = &u.x;
                if (D - c < 8) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        word[k] &= D - c >= 2 * k + 2 ? 0xffffffffu : D - c > 2 * k ? 0xffffu : 0u;
                }
            }
            *(uint4 *)(dst + r * pitch + c) = u;
            continue;
        }
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = c + j < D ? act_ld(src, (size_t)(r * D + c + j)) : 0.f;
        if (!second && y.ids && y.at(r, false) < 0) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = 0.f;
        }
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
// Width of dz's buffer, unless the caller says: 512 MiB of BF16 (or three fp32 terms), but
// 4,096 columns at least (from 65,536 tokens of BF16 on more bytes than that: 8 GiB at
// 2^20), in equal pieces of whole column tiles.
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
    bool f32, w32, pack_x, pack_w;
    int planes, pairs, chunk, x_pitch, w_pitch, piece, pieces, dx_splits, dw_splits;
    size_t xp, wp, part, zy, sums, dz, acc, dw_acc, unit, total;
};

// In how many parts the contraction of an M x N product is taken so that its tiles fill
// the rounds over the SMs: a stage of a tile is about a third of a microsecond, and the
// parts are written and read once more (fp32, 1,000 x 58,219 x 2,502: dx has 80 tiles).
int splits_for(long long M, int N, int cols, int k_blocks, int pairs) {
    const int n = device_sms(), most = k_blocks / 4;  // at least four steps each
    const long long tiles = (long long)cdiv(M, BM) * cdiv(N, cols);
    auto microseconds = [&](int s) {
        const double stages = (double)cdiv(k_blocks, s) * pairs;
        const double parts = s > 1 ? 5. + (double)s * M * N * 8. / 6.5e6 : 0.;
        return cdiv(tiles * s, n) * (stages / 3. + 1.) + parts;
    };
    int best = 1;
    double least = microseconds(1);
    for (int rounds = 1; rounds <= 12; ++rounds) {  // as many parts as fit in them
        const long long fit = (long long)rounds * n / tiles;
        const int s = (int)(fit < most ? fit : most);
        if (s < 2 || s == best) continue;
        const double us = microseconds(s);
        if (us < 0.97 * least) {
            best = s;
            least = us;
        }
    }
    return best;
}

// Pieces of the workspace.
Layout layout_for(const kda_ce_desc_t *d, bool backward) {
    Layout l = {};
    const size_t T = d->tokens, V = d->vocab;
    const int D = d->width;
    l.f32 = d->act_dtype == KDA_DTYPE_F32;
    // fp32: a weight that is read for one row of tiles only is split on its way; one that
    // is read more often is copied in terms (at 2,000 x 20,000 x 1,024 334 us, against
    // 423), and so is one whose rows a tensor map cannot address
    l.w32 = l.f32 && d->tokens <= BM && d->width % 4 == 0;
    l.planes = l.f32 ? 3 : 1;
    l.pairs = l.f32 ? 6 : 1;
    l.chunk = l.f32 ? kChunkF32 : kChunkBf16;
    // Copies: x in a backward pass (ignored rows become zeros); whole 128-byte lines where
    // x and W are copied as BF16 (with rows of 1,040 bytes the copies of 128-byte boxes ran
    // at half the rate)
    l.pack_x = l.f32 || D % 8 != 0 || backward;
    l.pack_w = l.f32 ? !l.w32 : D % 8 != 0;
    l.x_pitch = l.pack_x ? (D + 63) / 64 * 64 : D;
    l.w_pitch = l.pack_w ? (D + 63) / 64 * 64 : D;
    l.xp = l.pack_x ? round256(T * l.x_pitch * l.planes * 2) : 0;
    l.wp = l.pack_w ? round256(V * l.w_pitch * l.planes * 2) : 0;
    if (!backward) {
        l.part = round256((size_t)2 * cdiv(V, l.w32 ? kW32Cols : BN) * T * sizeof(float2));
        l.zy = round256(T * 4);
        l.sums = round256((T / kJoinFew + 1) * sizeof(float2)) + 256;
    } else {
        l.piece = piece_cols(d, l.planes);
        l.pieces = cdiv(V, l.piece);
        l.dz = round256(T * l.piece * l.planes * 2);
        // dx has few tiles when T and D are small, d_weight when V and D are
        const int last = (int)V - (l.pieces - 1) * l.piece;
        l.dx_splits = splits_for(T, D, l.w32 ? kW32Cols : BN, last / BK, l.pairs);
        // (not where the caller bounds the workspace with pieces: d_weight's parts would
        // outgrow a small piece's dz)
        l.dw_splits = d->piece > 0 && l.pieces > 1
                          ? 1 : splits_for(l.piece, D, BN, cdiv(T, BK), l.pairs);
        if (l.pieces > 1 || l.dx_splits > 1) l.acc = round256((size_t)l.dx_splits * T * D * 4);
        if (l.dw_splits > 1) l.dw_acc = round256((size_t)l.dw_splits * l.piece * D * 4);
        l.unit = 256;
    }
    l.total = l.xp + l.wp + l.part + l.zy + l.sums + l.dz + l.acc + l.dw_acc + l.unit;
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

constexpr int kMajor = 128, kMnMajor = BK;  // rows of a box

// An operand [planes][rows][pitch] in boxes of 128 rows x 64 elements of the contraction
// (K-major), or 64 rows of the contraction x 64 (MN-major).
bool encode(CUtensorMap *tm, const void *base, int inner, long long rows, int planes, int box_rows) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)rows, (cuuint64_t)planes};
    const cuuint64_t strides[2] = {(cuuint64_t)inner * 2, (cuuint64_t)(rows * inner) * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1}, estr[3] = {1, 1, 1};
    return enc(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int EPI, bool A_MN, bool B_MN, bool FINE, bool BF16, int CTAS>
cudaError_t start_gemm(GemmArgs p, const CUtensorMap &ta, const CUtensorMap &tb, int n,
                       cudaStream_t st) {
    const auto kernel = gemm_kernel<EPI, A_MN, B_MN, FINE, BF16, CTAS>;
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

template <int EPI, bool A_MN, bool B_MN, bool FINE, bool BF16>
cudaError_t run_gemm(const GemmArgs &p, const CUtensorMap &ta, const CUtensorMap &tb,
                     cudaStream_t st) {
    const int n = device_sms();
    return use_pairs(p, n) ? start_gemm<EPI, A_MN, B_MN, FINE, BF16, 2>(p, ta, tb, n, st)
                           : start_gemm<EPI, A_MN, B_MN, FINE, BF16, 1>(p, ta, tb, n, st);
}

// A backward pass's product: FINE for fp32 operands and for long contractions.
template <int EPI, bool A_MN, bool B_MN>
cudaError_t run_backward(const GemmArgs &p, bool f32, const CUtensorMap &ta, const CUtensorMap &tb,
                         cudaStream_t st) {
    constexpr bool BF16 = EPI == EPI_OUT;
    if (f32) return run_gemm<EPI, A_MN, B_MN, true, false>(p, ta, tb, st);
    return cdiv(p.k_blocks, p.splits) > kLongStages
               ? run_gemm<EPI, A_MN, B_MN, true, BF16>(p, ta, tb, st)
               : run_gemm<EPI, A_MN, B_MN, false, BF16>(p, ta, tb, st);
}

// dst = the sum of `splits` parts of n values.
cudaError_t sum_splits(const float *acc, void *dst, long long n, int splits, bool bf16,
                       cudaStream_t st) {
    const long long need = (n + 255) / 256, most = 16ll * device_sms();
    const dim3 grid((unsigned)(need < most ? need : most));
    return bf16 ? launch_dependent(split_sum_kernel<__nv_bfloat16>, grid, dim3(256), 0, st, acc,
                                   (__nv_bfloat16 *)dst, n, splits)
                : launch_dependent(split_sum_kernel<float>, grid, dim3(256), 0, st, acc,
                                   (float *)dst, n, splits);
}

// Copies x and W where the layout wants them; xp, wp are what the products read.
cudaError_t run_pack(const kda_ce_desc_t *d, const Layout &l, const void *x, const void *w,
                     const Targets &y, const float *d_loss, float *unit, uint8_t *ws,
                     const void *&xp, const void *&wp, cudaStream_t st) {
    xp = l.pack_x ? ws : x;
    wp = l.pack_w ? ws + l.xp : w;
    if (!l.pack_x) return cudaSuccess;
    const long long T = d->tokens, V = l.pack_w ? d->vocab : 0, most = 16ll * device_sms();
    const long long need = ((T + V) * (l.x_pitch / 8) + 255) / 256;
    const dim3 grid((unsigned)(need < most ? need : most) + (d_loss ? 1 : 0));
    __nv_bfloat16 *to = (__nv_bfloat16 *)ws, *to_w = (__nv_bfloat16 *)(ws + l.xp);
    if (l.f32)
        return launch_dependent(pack_kernel<float>, grid, dim3(256), 0, st, (const float *)x, T, to,
                                (const float *)w, V, to_w, d->width, l.x_pitch, l.planes, y, d_loss, unit);
    return launch_dependent(pack_kernel<__nv_bfloat16>, grid, dim3(256), 0, st,
                            (const __nv_bfloat16 *)x, T, to, (const __nv_bfloat16 *)w, V, to_w,
                            d->width, l.x_pitch, l.planes, y, d_loss, unit);
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
    float2 *part = (float2 *)(ws + l.xp + l.wp);
    float *zy = (float *)(ws + l.xp + l.wp + l.part);
    float2 *sums = (float2 *)(ws + l.xp + l.wp + l.part + l.zy);
    unsigned *ticket = (unsigned *)(ws + l.total - 256);
    const void *xp, *wp;
    if (run_pack(desc, l, x, weight, Targets{}, nullptr, nullptr, ws, xp, wp, st) != cudaSuccess)
        return KDA_ERR_CUDA;
    GemmArgs p = {};
    p.M = desc->tokens;
    p.N = desc->vocab;
    p.splits = 1;
    p.pairs = l.pairs;
    p.chunk = l.chunk;
    p.y = {targets, desc->id_dtype == KDA_ID_I64, desc->vocab, desc->ignore_index, dev_status};
    p.part = part;
    p.z_y = zy;
    p.ticket = ticket;
    p.status = dev_status;
    cudaError_t e;
    const int tile_cols = l.w32 ? kW32Cols : BN;
    if (l.w32) {
        p.k_blocks = cdiv(desc->width, kW32Step);
        e = launch_w32(EPI_STATS, p, {xp, l.x_pitch, (const float *)wp, p.N, l.w_pitch}, st);
    } else {
        CUtensorMap ta, tb;
        p.k_blocks = cdiv(desc->width, BK);
        if (!encode(&ta, xp, l.x_pitch, p.M, l.planes, kMajor) ||
            !encode(&tb, wp, l.w_pitch, p.N, l.planes, kMajor))
            return KDA_ERR_CUDA;
        e = run_gemm<EPI_STATS, false, false, true, false>(p, ta, tb, st);
    }
    if (e != cudaSuccess) return KDA_ERR_CUDA;
    // 8 rows to a block while all blocks are resident (8 rows and 32: 1,024 x 131,072 9.0
    // us and 13.6; 4,992 x 36,995 19.1 and 10.7; 8,128 x 277 18.2 and 7.8)
    const bool many = cdiv(p.M, kJoinFew) > 2 * device_sms();
    if (launch_dependent(many ? ce_join_kernel<kJoinMany> : ce_join_kernel<kJoinFew>,
                         dim3(cdiv(p.M, many ? kJoinMany : kJoinFew)), dim3(kJoinThreads), 0, st,
                         (const float2 *)part, 2 * cdiv(p.N, tile_cols), p.M, p.y,
                         (const float *)zy, loss, lse, mean, sums, ticket) != cudaSuccess)
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
    __nv_bfloat16 *dz = (__nv_bfloat16 *)(ws + l.xp + l.wp);
    float *acc = (float *)(ws + l.xp + l.wp + l.dz), *dw_acc = acc + l.acc / 4;
    const void *xp, *wp;
    const Targets y = {targets, desc->id_dtype == KDA_ID_I64, desc->vocab, desc->ignore_index,
                       dev_status};
    // BF16: dz is kept in units of the largest d_loss (or its significand) and dx and
    // d_weight are multiplied by the unit.  A mean's 1 / N, the same for every row, rounded
    // into dz would move the whole gradient by up to 2^-8 (34 rows: error 2.6e-3 of the
    // gradient, 1.7e-3 of it the output's rounding).
    float *unit = l.f32 ? nullptr : (float *)(ws + l.total - 256);
    if (run_pack(desc, l, x, weight, y, l.f32 ? nullptr : d_loss, unit, ws, xp, wp, st) !=
        cudaSuccess)
        return KDA_ERR_CUDA;
    const int T = desc->tokens, V = desc->vocab, D = desc->width;
    const int step = l.w32 ? kW32Step : BK;
    // as K-major and MN-major operands
    CUtensorMap xk, xm, zk, zm, wk, wm;
    if (!encode(&xm, xp, l.x_pitch, T, l.planes, kMnMajor) ||
        !encode(&zm, dz, l.piece, T, l.planes, kMnMajor))
        return KDA_ERR_CUDA;
    if (!l.w32 && (!encode(&xk, xp, l.x_pitch, T, l.planes, kMajor) ||
                   !encode(&zk, dz, l.piece, T, l.planes, kMajor) ||
                   !encode(&wk, wp, l.w_pitch, V, l.planes, kMajor) ||
                   !encode(&wm, wp, l.w_pitch, V, l.planes, kMnMajor)))
        return KDA_ERR_CUDA;
    const W32Operands logits = {xp, l.x_pitch, (const float *)wp, V, l.w_pitch};
    const W32Operands back = {dz, l.piece, (const float *)wp, V, l.w_pitch};
    for (int k = 0; k < l.pieces; ++k) {
        const int v0 = k * l.piece, cols = V - v0 < l.piece ? V - v0 : l.piece;
        GemmArgs p = {};
        p.status = dev_status;
        p.pairs = l.pairs;
        p.chunk = l.chunk;
        p.splits = 1;
        p.M = T;
        p.N = cols;
        p.k_blocks = cdiv(D, step);
        p.b_row0 = v0;
        p.y = y;
        p.lse = lse;
        p.d_loss = d_loss;
        p.unit = unit;
        p.dz = dz;
        p.pitch = l.piece;
        p.planes = l.planes;
        if ((l.w32 ? launch_w32(EPI_DZ, p, logits, st)
                   : run_backward<EPI_DZ, false, false>(p, l.f32, xk, wk, st)) != cudaSuccess)
            return KDA_ERR_CUDA;
        if (dx) {
            GemmArgs q = {};
            q.status = dev_status;
            q.pairs = l.pairs;
            q.unit = unit;
            q.chunk = l.chunk;
            q.splits = l.dx_splits;
            q.M = T;
            q.N = D;
            q.k_blocks = cdiv(cols, step);
            q.bk_row0 = v0;
            q.acc_in = k > 0 ? acc : nullptr;
            if (l.dx_splits == 1 && k == l.pieces - 1) q.out = dx;
            else q.acc_out = acc;
            q.out_bf16 = size == 2;
            q.vec = D % 8 == 0 && ((uintptr_t)dx & 15u) == 0;
            if (q.splits > q.k_blocks) return KDA_ERR_CUDA;
            if ((l.w32 ? launch_w32(EPI_OUT, q, back, st)
                       : run_backward<EPI_OUT, false, true>(q, l.f32, zk, wm, st)) != cudaSuccess)
                return KDA_ERR_CUDA;
            if (l.dx_splits > 1 && k == l.pieces - 1 &&
                sum_splits(acc, dx, (long long)T * D, l.dx_splits, size == 2, st) != cudaSuccess)
                return KDA_ERR_CUDA;
        }
        if (d_weight) {
            GemmArgs q = {};
            q.status = dev_status;
            q.pairs = l.pairs;
            q.unit = unit;
            q.chunk = l.chunk;
            q.splits = l.dw_splits;
            q.M = cols;
            q.N = D;
            q.k_blocks = cdiv(T, BK);
            void *to = (uint8_t *)d_weight + (size_t)v0 * D * size;
            if (l.dw_splits > 1) q.acc_out = dw_acc;
            else q.out = to;
            q.out_bf16 = size == 2;
            q.vec = D % 8 == 0 && ((uintptr_t)d_weight & 15u) == 0;
            if (run_backward<EPI_OUT, true, true>(q, l.f32, zm, xm, st) != cudaSuccess)
                return KDA_ERR_CUDA;
            if (l.dw_splits > 1 && sum_splits(dw_acc, to, (long long)cols * D, l.dw_splits,
                                              size == 2, st) != cudaSuccess)
                return KDA_ERR_CUDA;
        }
    }
    return KDA_OK;
}

}  // extern "C"
