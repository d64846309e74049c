// The cross entropy's products with an fp32 weight and few tokens (at most 128: one row
// of tiles): z = x W^T (its statistics, or dz) and dx = dz W.
//
// These are bound by W's bytes.  It is read as it is, 4 bytes an element, and split into
// its three BF16 terms on the way from one place in shared memory to another; x and dz
// come as terms.  (With W copied in terms first, 6 bytes more to write and 6 to read,
// 31 x 56,064 x 2,112 took 441 us; what bounds it here is the bandwidth of shared memory:
// per 16 KB of W the products read 96 KB, the split moves 40 and the copies 40.)
//
// Persistent CTAs, one per SM, tiles of 128 x 128, steps of 32 along the contraction:
//   warp 0      one thread loads A's three terms (two stages of two steps) and W (three
//               stages), each with one copy per 128 rows: their number bounds them, not
//               their bytes;
//   warps 10-13 split a stage of W into the B operand's terms (two stages);
//   warp 1      one thread issues 6 x 2 tcgen05.mma (128 x 128 x 16) per step;
//   warps 2-9   the epilogue: after every third step the accumulator is handed over
//               and added up in registers (rounded to nearest; the tensor core
//               truncates), 64 columns per thread.
// A is K-major with 128-byte swizzle, B (along W's channels) K-major with 64-byte
// swizzle or (along the vocabulary) MN-major with 128-byte swizzle.
#include "kda_ce_gemm.cuh"

namespace kda {
namespace {

constexpr int NB = kW32Cols, KB = kW32Step, kHandOver = 3;
constexpr int kStagesA = 2, kStagesW = 3, kStagesB = 2;
constexpr int kTerm = NB * KB * 2;       // one term of B's 128 x 32
constexpr int kTermA = BM * 2 * KB * 2;  // one term of A's 128 x 64
constexpr int kStageA = 3 * kTermA, kStageB = 3 * kTerm, kStageW = NB * KB * 4;
constexpr int kSplitWarps = 4, kThreads32 = 32 * (2 + kEpiWarps + kSplitWarps);
constexpr uint32_t kCols = 2 * NB;  // two accumulators
constexpr int kOffB = kStagesA * kStageA, kOffW = kOffB + kStagesB * kStageB,
              kOffOut = kOffW + kStagesW * kStageW, kOffBar = kOffOut + kEpiWarps * 4096;
enum { W_AF = 0, W_AE = W_AF + kStagesA, W_WF = W_AE + kStagesA, W_WE = W_WF + kStagesW,
       W_BF = W_WE + kStagesW, W_BE = W_BF + kStagesB, W_ACCF = W_BE + kStagesB, W_ACCE = W_ACCF + 2,
       W_FIN = W_ACCE + 2, W_N = W_FIN + 1 };
constexpr int kOffMisc = kOffBar + W_N * 8, kBytes = kOffMisc + 16 + 1024;
static_assert(kBytes <= 227 * 1024, "shared memory budget");
// K-major operand of 32 BF16 per row with 64-byte swizzle (16-byte piece c of row r at
// c ^ (r / 2 mod 4)): 8-row groups 512 bytes apart; a step of 16 starts 32 bytes on.
__device__ __forceinline__ uint64_t umma_desc_sw64(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)1u << 16;  // LBO (unused with swizzling)
    d |= (uint64_t)(512 >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)4u << 61;  // layout type: 64-byte swizzle
    return d;
}

__device__ __forceinline__ float4 lds4(uint32_t at) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}

// Four fp32 values as three terms of four BF16 at `to`, kTerm bytes apart.
__device__ __forceinline__ void split4(float4 v, uint32_t to) {
#pragma unroll
    for (int t = 0; t < 3; ++t) {
        const uint32_t a = pack_bf16x2(v.x, v.y), b = pack_bf16x2(v.z, v.w);
        v.x -= __uint_as_float(a << 16);
        v.y -= __uint_as_float(a & 0xffff0000u);
        v.z -= __uint_as_float(b << 16);
        v.w -= __uint_as_float(b & 0xffff0000u);
        asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(to + t * kTerm), "r"(a), "r"(b)
                     : "memory");
    }
}

template <int EPI>
__global__ void __launch_bounds__(kThreads32, 1)
    gemm_w32_kernel(const __grid_constant__ GemmArgs p, const __grid_constant__ CUtensorMap tm_a,
                    const __grid_constant__ CUtensorMap tm_w) {
    constexpr bool ROWS = EPI == EPI_OUT;  // the contraction runs along W's rows
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t sb = smem_addr(sm);
    auto bar = [&](int i) { return sb + kOffBar + 8 * i; };
    volatile int *abort = (volatile int *)(sm + kOffMisc);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int work = p.m_tiles * p.n_tiles * p.splits;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStagesA; ++i) mbar_init(bar(W_AF + i), 1), mbar_init(bar(W_AE + i), 1);
        for (int i = 0; i < kStagesW; ++i)
            mbar_init(bar(W_WF + i), 1), mbar_init(bar(W_WE + i), kSplitWarps);
        for (int i = 0; i < kStagesB; ++i)
            mbar_init(bar(W_BF + i), kSplitWarps), mbar_init(bar(W_BE + i), 1);
        for (int i = 0; i < 2; ++i)
            mbar_init(bar(W_ACCF + i), 1), mbar_init(bar(W_ACCE + i), kEpiWarps);
        mbar_init(bar(W_FIN), 1);
        *abort = 0;
        mbar_fence_init();
    }
    if (warp == 0) tmem_alloc_group<1>(sb + kOffMisc + 4, kCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *(volatile uint32_t *)(sm + kOffMisc + 4);
    griddep_wait();
    griddep_launch_dependents();
    if (EPI == EPI_STATS && blockIdx.x == 0 && threadIdx.x == 0) *p.ticket = 0;

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t ta = reinterpret_cast<uint64_t>(&tm_a);
            const uint64_t tw = reinterpret_cast<uint64_t>(&tm_w);
            int it = 0, ia = 0;  // steps; stages of A
            bool ok = true;
            for (int w = blockIdx.x; w < work && ok; w += gridDim.x) {
                const Tile t = tile_at<1>(p, w);
                const int wn = t.n * NB + p.b_row0;
                for (int kb = t.kb0; kb < t.kb1; ++kb, ++it) {
                    const int sw = it % kStagesW;
                    // W first: it comes from farther and is worked on before A is needed
                    ok = mbar_wait(bar(W_WE + sw), ((it / kStagesW) & 1) ^ 1, abort, kWaitLimit);
                    if (!ok) break;
                    mbar_arrive_expect_tx(bar(W_WF + sw), kStageW);
                    tma_load_2d(sb + kOffW + sw * kStageW, tw, ROWS ? wn : kb * KB,
                                ROWS ? kb * KB + p.bk_row0 : wn, bar(W_WF + sw));
                    if ((kb - t.kb0) & 1) continue;
                    const int sa = ia % kStagesA;
                    ok = mbar_wait(bar(W_AE + sa), ((ia / kStagesA) & 1) ^ 1, abort, kWaitLimit);
                    if (!ok) {  // W's stage is in flight: the count below covers it
                        ++it;
                        break;
                    }
                    mbar_arrive_expect_tx(bar(W_AF + sa), kStageA);
#pragma unroll
                    for (int q = 0; q < 3; ++q)
                        tma_load_3d<1>(sb + sa * kStageA + q * kTermA, ta, kb * KB, t.m * BM, q,
                                       bar(W_AF + sa));
                    ++ia;
                }
            }
            if (*abort) {  // let the copies in flight land before the CTA exits
                volatile int never = 0;
                for (int k = it > kStagesW ? it - kStagesW : 0; k < it; ++k)
                    mbar_wait(bar(W_WF + k % kStagesW), (k / kStagesW) & 1, &never, kWaitLimit / 8);
                for (int k = ia > kStagesA ? ia - kStagesA : 0; k < ia; ++k)
                    mbar_wait(bar(W_AF + k % kStagesA), (k / kStagesA) & 1, &never, kWaitLimit / 8);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = umma_idesc_bf16(BM, NB) | (ROWS ? 1u << 16 : 0u);
            int it = 0, i = 0, ia = 0;
            bool ok = true;
            for (int w = blockIdx.x; w < work && ok; w += gridDim.x, ++i) {
                const Tile t = tile_at<1>(p, w);
                int first = 0;  // steps in this accumulator
                for (int kb = t.kb0; kb < t.kb1; ++kb, ++it, ++first) {
                    if (first == kHandOver) {
                        umma_commit(bar(W_ACCF + (i++ & 1)));
                        first = 0;
                    }
                    if (first == 0) {
                        ok = mbar_wait(bar(W_ACCE + (i & 1)), ((i >> 1) & 1) ^ 1, abort, kWaitLimit);
                        if (!ok) break;
                        tc_fence_after();
                    }
                    const int sa = ia % kStagesA, sp = it % kStagesB, odd = (kb - t.kb0) & 1;
                    ok = mbar_wait(bar(W_AF + sa), (ia / kStagesA) & 1, abort, kWaitLimit) &&
                         mbar_wait(bar(W_BF + sp), (it / kStagesB) & 1, abort, kWaitLimit);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t a = sb + sa * kStageA + odd * 64, b = sb + kOffB + sp * kStageB;
#pragma unroll
                    for (int pr = 0; pr < 6; ++pr)
#pragma unroll
                        for (int kk = 0; kk < KB / 16; ++kk) {
                            const uint32_t bt = b + term_b(pr, 6) * kTerm;
                            umma_bf16(tmem + NB * (i & 1),
                                      umma_desc_sw128(a + term_a(pr, 6) * kTermA + kk * 32, 1024),
                                      ROWS ? umma_desc_mn_sw128(bt + kk * 2048, KB)
                                           : umma_desc_sw64(bt + kk * 32),
                                      idesc, first + pr + kk > 0);
                        }
                    umma_commit(bar(W_BE + sp));
                    if (odd || kb + 1 == t.kb1) {  // A's stage: two steps, or a tile's last
                        umma_commit(bar(W_AE + sa));
                        ++ia;
                    }
                }
                if (ok) umma_commit(bar(W_ACCF + (i & 1)));
            }
            if (*abort) {  // products in flight complete before TMEM is freed
                umma_commit(bar(W_FIN));
                volatile int never = 0;
                mbar_wait(bar(W_FIN), 0, &never, kWaitLimit);
            }
        }
    } else if (warp >= 2 + kEpiWarps) {
        const int tid = threadIdx.x - 32 * (2 + kEpiWarps);
        int it = 0;
        bool ok = true;
        for (int w = blockIdx.x; w < work && ok; w += gridDim.x) {
            const Tile t = tile_at<1>(p, w);
            for (int kb = t.kb0; kb < t.kb1; ++kb, ++it) {
                const int sw = it % kStagesW, sp = it % kStagesB;
                ok = mbar_wait(bar(W_WF + sw), (it / kStagesW) & 1, abort, kWaitLimit);
                float4 v[8];  // four values each; all loads before the first store
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    v[q] = lds4(sb + kOffW + sw * kStageW + (tid + 128 * q) * 16);
                ok = ok && mbar_wait(bar(W_BE + sp), ((it / kStagesB) & 1) ^ 1, abort, kWaitLimit);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const uint32_t to = sb + kOffB + sp * kStageB;
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const int at = tid + 128 * q;
                    if (ROWS) {  // row k of 128 channels, in boxes of 64
                        const int k = at >> 5, n = 4 * (at & 31);
                        split4(v[q], to + (n >> 6) * (KB * 128) + k * 128 +
                                         ((((n & 63) >> 3) ^ (k & 7)) << 4) + (n & 4) * 2);
                    } else {  // row r of 32 channels
                        const int r = at >> 3, c = at & 7;
                        split4(v[q], to + r * 64 + (((c >> 1) ^ ((r >> 1) & 3)) << 4) + (c & 1) * 8);
                    }
                }
                fence_async_smem();  // the tensor core reads what was written here
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(W_BF + sp));
                    mbar_arrive(bar(W_WE + sw));
                }
            }
        }
    } else {
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        const uint32_t src = tmem + ((uint32_t)(32 * quarter) << 16) + 64 * half;
        const Turn turn = {sb + kOffOut + (warp - 2) * 4096, lane};
        int i = 0;
        bool ok = true;
        for (int w = blockIdx.x; w < work && ok; w += gridDim.x) {
            const Tile t = tile_at<1>(p, w);
            Row<EPI, false> r;
            r.begin(p, t, t.m * BM + 32 * quarter, lane, half, 64);
            __syncwarp();
            float acc[2][32];
#pragma unroll
            for (int ch = 0; ch < 2; ++ch)
#pragma unroll
                for (int j = 0; j < 32; ++j) acc[ch][j] = 0.f;
            for (int kb = t.kb0; kb < t.kb1; kb += kHandOver) {
                ok = __all_sync(0xffffffffu, mbar_wait(bar(W_ACCF + (i & 1)), (i >> 1) & 1, abort,
                                                       kWaitLimit));
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int ch = 0; ch < 2; ++ch) {
                    float v[32];
                    tmem_ld32(src + NB * (i & 1) + 32 * ch, v);
#pragma unroll
                    for (int j = 0; j < 32; j += 2) add2(acc[ch][j], acc[ch][j + 1], v[j], v[j + 1]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(W_ACCE + (i & 1)));
                ++i;
            }
            if (!ok) break;
            r.pair(p, t, turn, 0, acc[0], acc[1]);
            r.end(p, t, half);
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *abort) dev_fail(p.status, KDA_ERR_TIMEOUT);
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc_group<1>(tmem, kCols);
    }
}

// `rows` x `inner` elements of type `type` (planes of them) in boxes of box_rows x
// box_inner.
bool encode(CUtensorMap *tm, CUtensorMapDataType type, int size, const void *base, int inner,
            long long rows, int planes, int box_inner, int box_rows, CUtensorMapSwizzle swizzle) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)rows, (cuuint64_t)planes};
    const cuuint64_t strides[2] = {(cuuint64_t)inner * size, (cuuint64_t)(rows * inner) * size};
    const cuuint32_t box[3] = {(cuuint32_t)box_inner, (cuuint32_t)box_rows, 1}, estr[3] = {1, 1, 1};
    return enc(tm, type, planes > 1 ? 3 : 2, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int EPI>
cudaError_t launch(GemmArgs p, const W32Operands &o, cudaStream_t st) {
    cudaError_t e = set_max_dynamic_smem((const void *)gemm_w32_kernel<EPI>, kBytes);
    if (e != cudaSuccess) return e;
    p.bn = NB;
    p.m_tiles = cdiv(p.M, BM);
    p.n_tiles = cdiv(p.N, NB);
    const bool by_rows = EPI == EPI_OUT;
    CUtensorMap ta, tw;
    if (!encode(&ta, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, o.a, o.a_inner, p.M, 3, 2 * KB, BM,
                CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode(&tw, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, o.w, o.width, o.w_rows, 1,
                by_rows ? NB : KB, by_rows ? KB : NB, CU_TENSOR_MAP_SWIZZLE_NONE))
        return cudaErrorInvalidValue;
    const long long work = (long long)p.m_tiles * p.n_tiles * p.splits;
    const int n = device_sms();
    return launch_dependent(gemm_w32_kernel<EPI>, dim3((unsigned)(work < n ? work : n)),
                            dim3(kThreads32), kBytes, st, p, ta, tw);
}

}  // namespace

cudaError_t launch_w32(int epi, const GemmArgs &p, const W32Operands &o, cudaStream_t st) {
    switch (epi) {
        case EPI_STATS: return launch<EPI_STATS>(p, o, st);
        case EPI_DZ: return launch<EPI_DZ>(p, o, st);
    }
    return launch<EPI_OUT>(p, o, st);
}

}  // namespace kda
