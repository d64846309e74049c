// The persistent tcgen05 product that the cross entropy and the gated feed-forward block run
// on, the copies that make its operands, and their launches.  Included by the files that
// launch it: every instantiation belongs to one of them.
#pragma once

#include <float.h>
#include <math.h>

#include "kda_gemm.cuh"

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
    const int work = p.m_tiles * p.n_tiles * p.splits * p.batches;
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
            constexpr bool TWO = EPI == EPI_GLU || EPI == EPI_DGLU;
            // boxes of 64 x 64 of B; K-major ones come in twos, of two matrices in halves
            const int boxes = B_MN ? (p.bn / CTAS + 63) / 64
                              : TWO ? p.bn / CTAS / 32 : 2 * ((p.bn / CTAS + 127) / 128);
            const int box_bytes = TWO ? kBox / 2 : kBox;
            const int passes = p.pairs * p.groups;
            int it = 0;
            bool ok = true;
            for (int w = w0; w < work && ok; w += wstep) {
                const Tile t = tile_at<CTAS>(p, w);
                const int ar = (t.m * CTAS + rank) * BM;
                const int br = t.n * p.bn + rank * (p.bn / CTAS) + p.b_row0;
                for (int pr = 0; pr < passes && ok; ++pr) {
                    const int term = pr % p.pairs, which = p.batches > 1 ? t.batch : pr / p.pairs;
                    const int pa = term_a(term, p.pairs) * p.a_group + (p.a_group > 1 ? which : 0);
                    const int pb = term_b(term, p.pairs) * p.b_group + (p.b_group > 1 ? which : 0);
                    for (int kb = t.kb0; kb < t.kb1; ++kb, ++it) {
                        const int s = it % S::stages;
                        ok = mbar_wait(empty_bar(s), ((it / S::stages) & 1) ^ 1, abort, kWaitLimit);
                        if (!ok) break;
                        const uint32_t a = sb + s * S::stage, b = a + kABytes;
                        uint32_t full = full_bar(s);
                        if (CTAS == 2) full = cluster_map(full, 0);  // the issuing CTA waits for
                                                                     // both CTAs' bytes
                        if (rank == 0)
                            mbar_arrive_expect_tx(full_bar(s), CTAS * (kABytes + boxes * box_bytes));
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
                        if (TWO) {
                            const int first = rank * boxes;  // of the tile's
                            for (int i = 0; i < boxes; ++i)
                                tma_load_3d<CTAS>(b + i * box_bytes, tb, kb * BK,
                                                  t.n * (p.bn / 2) + p.b_row0 + 32 * ((first + i) >> 1),
                                                  2 * pb + ((first + i) & 1), full);
                            continue;
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
                const int steps = (t.kb1 - t.kb0) * p.pairs * p.groups;
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
                const int steps = (t.kb1 - t.kb0) * p.pairs * p.groups;
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
                            add_pair(acc[ch][j], acc[ch][j + 1], v[j], v[j + 1]);
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

constexpr int kMajor = 128, kMnMajor = BK;  // rows of a box
constexpr cuuint64_t kSmallMap = 128 * 1024;

// An operand [planes][rows][pitch] in boxes of 128 rows x 64 elements of the contraction
// (K-major), or 64 rows of the contraction x 64 (MN-major).
bool encode(CUtensorMap *tm, const void *base, int inner, long long rows, int planes, int box_rows) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)rows, (cuuint64_t)planes};
    cuuint64_t strides[2] = {(cuuint64_t)inner * 2, (cuuint64_t)(rows * inner) * 2};
    // An operand of less than 128 KB that all SMs read comes slower (BF16 feed-forward block of 9
    // tokens, 7,168 x 14,336, 93 us, of 10, 143 KB, 69; 4,096 channels: 15 tokens 58, 16 43).
    // A second plane that no copy asks for makes the map larger.
    if (planes == 1 && strides[1] < kSmallMap) {
        dims[2] = 2;
        strides[1] = kSmallMap;
    }
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
    p.n_tiles = cdiv(p.N, p.bn ? p.bn : BN);
    if (!p.bn) p.bn = cdiv(cdiv(p.N, p.n_tiles), 64) * 64;  // tiles of about equal width
    const long long work = (long long)p.m_tiles * p.n_tiles * p.splits * p.batches;
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
    const long long cols = (long long)cdiv(p.N, p.bn ? p.bn : BN) * p.splits * p.batches;
    const long long one = (cdiv(p.M, BM) * cols + n - 1) / n;
    const long long two = (cdiv(p.M, 2 * BM) * cols + n / 2 - 1) / (n / 2);
    return n >= 2 && two <= one;
}

template <int EPI, bool A_MN, bool B_MN, bool FINE, bool BF16>
cudaError_t run_gemm(const GemmArgs &p, const CUtensorMap &ta, const CUtensorMap &tb,
                     cudaStream_t st) {
    const int n = device_sms();
    return (p.ctas ? p.ctas == 2 : use_pairs(p, n)) ? start_gemm<EPI, A_MN, B_MN, FINE, BF16, 2>(p, ta, tb, n, st)
                           : start_gemm<EPI, A_MN, B_MN, FINE, BF16, 1>(p, ta, tb, n, st);
}

// A backward pass's product: FINE for fp32 operands and for long contractions.
template <int EPI, bool A_MN, bool B_MN>
cudaError_t run_backward(const GemmArgs &p, bool f32, const CUtensorMap &ta, const CUtensorMap &tb,
                         cudaStream_t st) {
    constexpr bool BF16 = EPI == EPI_OUT;
    if (f32) return run_gemm<EPI, A_MN, B_MN, true, false>(p, ta, tb, st);
    return cdiv(p.k_blocks, p.splits) * p.groups > kLongStages
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

bool bad16(const void *p) { return !p || ((uintptr_t)p & 15u); }

}  // namespace
}  // namespace kda
