// The norms of many rows: rows stream through shared memory (bulk copies, a
// ring of stages), so the bytes in flight do not depend on the registers that the
// arithmetic takes, and rows of odd widths need no aligned access of their own: a tile
// of eight (BF16) or four (fp32) of them, or a multiple, starts on a 16-byte boundary.
//
// Measured on GB300 (BF16; a copy of this size runs at 6.4-6.8 TB/s): gradient of the
// gated norm of 81,920 x 56 x 128 876-880 us (6.7 TB/s; with rows loaded straight into
// registers 1,026, bound by the loads that 25 % of the warps can have in flight); of the
// residual norm of 40,960 x 7,168 440-442 us (6.7 TB/s; 518 without the ring).  A row of
// 5,120 in a tile by itself is bound by its latency (26,214 rows, forward: 175 us, a copy
// 159; with 512 threads instead of the 384 that it needs 194).
#include "kda_norm_math.cuh"
#include "kda_sm100.cuh"

namespace kda {
namespace {

using namespace sm100;

// 512 working threads and a warpgroup of which one thread copies.  Launched with 96
// registers each; that warpgroup gives up 72 of them and the others take 16 more:
// 512 x 112 + 128 x 24 = 60,416 of the 61,440 at launch.
constexpr int kWork = 512, kWarps = kWork / 32, kThreads = kWork + 128;
constexpr long long kWaitLimit = 4000000000ll;  // ~2 s of SM clocks
constexpr int kRingBytes = 208 * 1024, kMaxStages = 8;

struct Ring {
    int tpr, rows, arrays, stages;  // threads per row, rows per tile, arrays read
    int work, warps, join;  // threads with a row; a row's warps, and a power of two for them
    int array_bytes, stage_bytes, skew;
    long long tiles;
};

// The stages, as bytes in flight in an SM.  Few are faster where the arithmetic keeps up:
// 256 M elements of BF16 (gated norm forward, 8 x 128: 277 us with 192 KB, 230 with 96;
// the norm alone 188 with 128 KB, 168 with 64; residual norm, 512: forward 356 with 192,
// 350 with 96, 313 with 64; 7,168: 335 with 115, 318 with 86; its gradient, 512: 456 with
// 144, 426 with 96; 128 M of fp32, gated norm forward, 4 x 100: 250 with 154, 229 with 102).
// The gradient of the gated norm (400-411 from 96 to 200) and rows as pairs (residual norm
// forward, 125: 798 with 64 KB, 702 with 160; backward, 33: 1,250 with 76, 1,212 with 152,
// 1,292 with 203) are bound by more than the copies.
int bytes_in_flight(int op, bool bwd, int size, bool pairs) {
    if (pairs || (bwd && size == 2 && (op == OP_SIGMOID || op == OP_SILU))) return 160 * 1024;
    if (bwd || size == 4 || op == OP_SIGMOID || op == OP_SILU) return 96 * 1024;
    return op == OP_NORM ? 64 * 1024 : 88 * 1024;  // as many bytes written as read
}

// A thread holds 16 elements: 16-byte pieces (two of BF16, four of fp32), or eight pairs
// where rows are not whole pieces (`pairs`).  A tile is one row per group of tpr
// threads: 16 KB per array where the width fills its threads.
Ring ring_for(const NormArgs &a, int op, bool bwd, int size, bool pairs) {
    Ring r = {};
    const int vec = pairs ? 2 : 16 / size, pieces = (a.D + vec - 1) / vec, nv = 16 / vec;
    r.tpr = 1;
    while (r.tpr * nv < pieces) r.tpr *= 2;
    if (!pairs && r.tpr > (size == 2 ? 32 : 256)) {
        // whole warps, and as many on each scheduler where a tile is one row (128 M elements,
        // BF16 forward, 1,280: 180 -> 166 us, 5,120: 194 -> 175; not for shorter rows of fp32:
        // more rows in a tile are more bytes in flight, backward, 2,560: 437 -> 444)
        const int unit = r.tpr > 256 ? 128 : 32;
        r.tpr = ((pieces + nv - 1) / nv + unit - 1) / unit * unit;
    }
    if (pieces < nv || r.tpr > kWork) return r;  // arrays = 0: does not apply
    r.warps = r.tpr / 32;
    r.join = 1;
    while (r.join < r.warps) r.join *= 2;
    r.rows = kWork / r.tpr;
    r.work = r.rows * r.tpr;
    if (pairs && r.rows % (16 / size) != 0) return r;  // tiles would start anywhere
    r.tiles = (a.rows + r.rows - 1) / r.rows;
    r.arrays = 1 + (bwd ? 1 : 0);
    if (op == OP_SIGMOID || op == OP_SILU || (is_residual(op) && (bwd ? a.d_res : a.gate)))
        ++r.arrays;
    r.array_bytes = r.rows * a.D * size;
    r.stage_bytes = r.arrays * r.array_bytes;
    // SKEW pays in BF16 gradients of the gated norm, whose arithmetic is the longest (SiLU,
    // 1,170 x 8 x 7,168 145 us, 187 without, 8,190 x 8 x 1,024 120 and 134; sigmoid, 65,536 x
    // 2,048 225 and 244), not of the residual norm (32,768 x 4,096 225 and 219, 131,072 x
    // 1,024 230 and 220, 16,384 x 8,192 225 and 206).
    // Dropout's random words are as long (40,960 x 7,168 678 us, 725 without, 81,920 x 1,024 169
    // and 172; forward, where they must come before the sums, 637 and 548).
    r.skew = size == 2 && bwd && !pairs && r.tpr > 32 &&
             (op == OP_SIGMOID || op == OP_SILU || op == OP_DROP);
    const int most = kRingBytes / r.stage_bytes;
    r.stages = r.skew ? most : bytes_in_flight(op, bwd, size, pairs) / r.stage_bytes;
    if (r.stages < 2) r.stages = 2;
    if (r.stages > most) r.stages = most;
    if (r.stages > kMaxStages) r.stages = kMaxStages;
    return r;
}

// SKEW, for rows of more than a warp (it needs four stages): a row's outputs come after
// the next row's sums, so no warp waits at a barrier for its row's other warps.  The
// pieces are then read from shared memory twice and the stage is released after the
// outputs.
// APART: x's and the gate's tokens lie apart, one copy for each token's part of a tile,
// issued by the producer's whole warp.
template <int OP, bool BWD, typename T, bool SKEW, bool PAIRS, bool APART>
__global__ void __launch_bounds__(kThreads, 1)
    norm_ring_kernel(const __grid_constant__ NormArgs p, const __grid_constant__ Ring r) {
    constexpr int VEC = PAIRS ? 2 : 16 / sizeof(T), NV = 16 / VEC, VP = kPairs<VEC>;
    constexpr int kRed = SKEW ? 4 : 2;
    using P = Piece<T, VEC>;
    extern __shared__ __align__(128) uint8_t sm[];
    __shared__ __align__(8) uint64_t bars[2 * kMaxStages];
    __shared__ __align__(8) uint64_t sum_bars[kRed][kWarps / 2];
    __shared__ float2 red[kRed][2 * kWarps];  // r.join for a row, those beyond r.warps zero
    __shared__ __align__(16) uint32_t keys[OP == OP_DROP ? kKeys : 4];
    __shared__ int abort_flag;
    volatile int *abort = &abort_flag;
    const uint32_t sb = smem_addr(sm), bb = smem_addr(bars);
    auto full = [&](int s) { return bb + 8 * s; };
    auto empty = [&](int s) { return bb + 8 * (kMaxStages + s); };
    const int warp = threadIdx.x >> 5, wl = threadIdx.x & 31;
    for (int k = threadIdx.x; k < kRed * 2 * kWarps; k += kThreads)
        red[k / (2 * kWarps)][k % (2 * kWarps)] = make_float2(0.f, 0.f);
    if (threadIdx.x == 0) {
        for (int s = 0; s < r.stages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), r.work / 32);
        }
        if (SKEW)
            for (int k = 0; k < kRed; ++k)
                for (int g = 0; g < r.rows; ++g) mbar_init(smem_addr(&sum_bars[k][g]), r.tpr / 32);
        abort_flag = 0;
        mbar_fence_init();
    }
    __syncthreads();
    griddep_wait();

    if (warp >= kWarps) {  // producer
        regs_dealloc<24>();
        if (APART ? warp > kWarps : threadIdx.x != kWork) return;
        const uint8_t *src[3] = {(const uint8_t *)p.x, nullptr, nullptr};
        int n = 1;
        const void *second = is_residual(OP) && BWD ? p.d_res : p.gate;
        if (OP != OP_NORM && second) src[n++] = (const uint8_t *)second;
        if (BWD) src[n++] = (const uint8_t *)p.d_out;
        const long long row_bytes = p.D * (long long)sizeof(T);
        int i = 0;
        for (long long t = blockIdx.x; t < r.tiles; t += gridDim.x, ++i) {
            const int s = i % r.stages;
            int ok = 1;
            if (wl == 0) ok = mbar_wait(empty(s), ((i / r.stages) & 1) ^ 1, abort, kWaitLimit);
            if (APART) ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            const long long row = t * r.rows, left = p.rows - row;
            const long long rows = left < r.rows ? left : r.rows;
            const uint32_t bytes = (uint32_t)(rows * row_bytes), at = sb + s * r.stage_bytes;
            const uint32_t whole = bytes & ~15u;  // the last tile may end inside a piece
            if (wl == 0) {
                for (int k = 0; PAIRS && k < n && whole < bytes; ++k)
                    for (uint32_t b = whole; b < bytes; b += sizeof(T))
                        *(T *)(sm + s * r.stage_bytes + k * r.array_bytes + b) =
                            *(const T *)(src[k] + row * row_bytes + b);
                mbar_arrive_expect_tx(full(s), n * whole);
                for (int k = APART ? 2 : 0; k < n && whole > 0; ++k)
                    bulk_g2s(at + k * r.array_bytes, src[k] + row * row_bytes, whole, full(s));
            }
            if constexpr (APART) {
                __syncwarp();
                const long long last = (row + rows - 1) / p.heads;
                for (long long tok = row / p.heads + wl; tok <= last; tok += 32) {
                    const long long first = tok * p.heads, next = first + p.heads;
                    const long long r0 = first > row ? first : row;
                    const long long r1 = next < row + rows ? next : row + rows;
#pragma unroll 1  // unrolled it would spill with 24 registers
                    for (int k = 0; k < 2; ++k) {
                        const long long from = tok * (k ? p.gate_stride : p.x_stride);
                        bulk_g2s(at + k * r.array_bytes + (uint32_t)((r0 - row) * row_bytes),
                                 src[k] + from * (long long)sizeof(T) + (r0 - first) * row_bytes,
                                 (uint32_t)((r1 - r0) * row_bytes), full(s));
                    }
                }
            }
        }
        if (wl == 0 && *abort) {  // let the copies in flight land before the block exits
            volatile int never = 0;
            for (int k = i > r.stages ? i - r.stages : 0; k < i; ++k)
                mbar_wait(full(k % r.stages), (k / r.stages) & 1, &never, kWaitLimit);
        }
        return;
    }

    regs_alloc<112>();
    if (threadIdx.x >= r.work) return;  // beyond the tile's last row
    const int group = threadIdx.x / r.tpr, lane = threadIdx.x - group * r.tpr;
    const int slot = group * r.join + (lane >> 5);
    auto column = [&](int i) { return (lane + i * r.tpr) * VEC; };
    auto load_w = [&](int i, f2 (&w)[VP]) {
#pragma unroll
        for (int j = 0; j < VP; ++j) {
            w[j] = both(1.f);
            const int c = column(i) + 2 * j;
            if (p.w && c < p.D) {
                if (PAIRS) w[j] = pk(p.w[c], c + 1 < p.D ? p.w[c + 1] : 1.f);
                else w[j] = *(const f2 *)(p.w + c);
            }
        }
    };
    RowMath<is_residual(OP) ? OP_RESIDUAL : OP, BWD, T, VEC, NV, !SKEW> math;
    math.begin(load_w);
    if constexpr (OP == OP_DROP) {
        Keep::lay_keys(p.drop, keys, threadIdx.x);
        named_bar_sync(15, r.work);
    }
    const Keep keep(OP == OP_DROP ? p.drop : Drop{}, keys);
    bool failed = false;  // a wait gave up: go through the motions, store nothing
    P px[NV], pg[NV], pd[NV];
    auto row_of = [&](long long t) { return t * r.rows + group; };
    // Every lane waits for itself: what one lane has acquired would reach the others only
    // through __syncwarp (a shuffle exchanges registers and orders no memory), and that is
    // slower (residual norm's gradient of 40,960 x 7,168: 442 us so, 483 with one lane
    // waiting; gated, SiLU, 9,360 x 7,168: 145 and 416).
    auto wait = [&](uint32_t bar, int parity) {
        const bool ok = mbar_wait(bar, parity, abort, kWaitLimit);
        failed = failed || !__all_sync(0xffffffffu, ok);
    };
    auto load = [&](long long t, int i) {
        const uint8_t *at = sm + (i % r.stages) * r.stage_bytes + (size_t)group * p.D * sizeof(T);
        const int second = r.array_bytes, third = (r.arrays - 1) * r.array_bytes;
        const bool live = row_of(t) < p.rows, has_g = r.arrays == (BWD ? 3 : 2);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = column(k);
            px[k].zero();
            pg[k].zero();
            pd[k].zero();
            if (live && c < p.D) {
                auto get = [&](P &to, const uint8_t *from) {
                    if constexpr (PAIRS) to.load((const T *)from + c, c + 1 < p.D);
                    else to.load((const T *)from + c);
                };
                get(px[k], at);
                if (OP != OP_NORM && has_g) get(pg[k], at + second);
                if (BWD) get(pd[k], at + third);
            }
        }
    };
    auto release = [&](int i) {
        __syncwarp();
        if (wl == 0) mbar_arrive(empty(i % r.stages));
    };
    auto warp_sums = [&](float &ss, float &se, int w) {
        for (int o = w >> 1; o > 0; o >>= 1) {
            ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (BWD) se += __shfl_xor_sync(0xffffffffu, se, o);
        }
    };
    auto row_sums = [&](int buf, float &ss, float &se) {
        const float2 u = red[buf][group * r.join + (wl & (r.join - 1))];
        ss = u.x;
        se = u.y;
        warp_sums(ss, se, r.join);
    };
    auto outputs = [&](long long t, float ss, float se, uint32_t kept = 0) {
        const long long row = row_of(t);
        math.outputs(p, px, pg, pd, load_w, ss, se, [&](int k, f2 (&a1)[VP], f2 (&a2)[VP]) {
            const int c = column(k);
            if (row >= p.rows || failed || c >= p.D) return;
            auto put = [&](void *to, f2 (&o)[VP]) {
                float v[VEC];
                floats<VEC>(o, v);
                if constexpr (OP == OP_DROP && BWD)
                    if (to == p.o2) {
                        if constexpr (SKEW) {
#pragma unroll
                            for (int j = 0; j < VEC; ++j)
                                v[j] = kept >> (VEC * k + j) & 1 ? v[j] : 0.f;
                        } else {
                            keep.template floats<false>(v, row, c);
                        }
                    }
                if constexpr (PAIRS) P::store((T *)to + row * p.D + c, v, c + 1 < p.D);
                else P::store((T *)to + row * p.D + c, v);
            };
            if (p.o1) put(p.o1, a1);
            if ((BWD || is_residual(OP)) && p.o2) put(p.o2, a2);
        });
    };
    int i = 0;
    if constexpr (SKEW) {
        uint32_t kept = 0, next_kept = 0;  // OP_DROP: which of a row's elements
        auto first_half = [&](long long t, int i) {
            if constexpr (OP == OP_DROP) {
                next_kept = 0;
#pragma unroll
                for (int k = 0; k < NV; ++k)
                    next_kept |= keep.template bits<VEC, false>(row_of(t), column(k)) << (VEC * k);
            }
            wait(full(i % r.stages), (i / r.stages) & 1);
            load(t, i);
            float ss, se;
            math.sums(p, px, pg, pd, load_w, ss, se);
            warp_sums(ss, se, 32);
            if (wl == 0) {
                red[i % kRed][slot] = make_float2(ss, se);
                mbar_arrive(smem_addr(&sum_bars[i % kRed][group]));
            }
        };
        if (blockIdx.x < r.tiles) first_half(blockIdx.x, 0);
        for (long long t = blockIdx.x; t < r.tiles; t += gridDim.x, ++i) {
            kept = next_kept;
            if (t + gridDim.x < r.tiles) first_half(t + gridDim.x, i + 1);
            wait(smem_addr(&sum_bars[i % kRed][group]), (i / kRed) & 1);
            float ss, se;
            row_sums(i % kRed, ss, se);
            load(t, i);
            outputs(t, ss, se, kept);
            release(i);
        }
    } else {
        for (long long t = blockIdx.x; t < r.tiles; t += gridDim.x, ++i) {
            wait(full(i % r.stages), (i / r.stages) & 1);
            load(t, i);
            release(i);  // the stage is in registers
            if constexpr (OP == OP_DROP && !BWD) {
#pragma unroll
                for (int k = 0; k < NV; ++k)
                    keep.template piece<false>(pg[k], row_of(t), column(k));
            }
            float ss, se;
            math.sums(p, px, pg, pd, load_w, ss, se);
            warp_sums(ss, se, r.tpr < 32 ? r.tpr : 32);
            if (r.tpr > 32) {
                if (wl == 0) red[i % kRed][slot] = make_float2(ss, se);
                named_bar_sync(1 + group, r.tpr);
                row_sums(i % kRed, ss, se);
            }
            outputs(t, ss, se);
        }
    }
    griddep_launch_dependents();
    if (threadIdx.x == 0 && *abort) dev_fail(p.status, KDA_ERR_TIMEOUT);
    if (!BWD || !p.partial) return;
    // dw: the block's groups in group order, in the ring (every copy has been used)
    named_bar_sync(15, r.work);
    if (*abort) return;
    float *sh = (float *)sm;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        float v[VEC];
        floats<VEC>(math.dw[k % (BWD ? NV : 1)], v);
#pragma unroll
        for (int j = 0; j < VEC; ++j)
            if (column(k) + j < p.D) sh[group * p.D + column(k) + j] = v[j];
    }
    named_bar_sync(15, r.work);
    for (int c = threadIdx.x; c < p.D; c += r.work) {
        float s = 0.f;
        for (int g = 0; g < r.rows; ++g) s += sh[g * p.D + c];
        p.partial[(size_t)blockIdx.x * p.D + c] = s;
    }
}

template <int OP, bool BWD, typename T, bool SKEW, bool PAIRS, bool APART>
cudaError_t launch_k(const NormArgs &a, const Ring &r, int blocks, cudaStream_t st) {
    const auto kernel = norm_ring_kernel<OP, BWD, T, SKEW, PAIRS, APART>;
    cudaError_t e = set_max_dynamic_smem((const void *)kernel, kRingBytes);
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, dim3(blocks), dim3(kThreads), r.stages * r.stage_bytes, st, a, r);
}

template <int OP, bool BWD, typename T>
cudaError_t launch_t(const NormArgs &a, const Ring &r, bool pairs, int blocks, cudaStream_t st) {
    if constexpr (sizeof(T) == 2 && (OP == OP_SIGMOID || OP == OP_SILU))
        if (a.strided) return launch_k<OP, BWD, T, false, false, true>(a, r, blocks, st);
    if constexpr (sizeof(T) == 2 && BWD && (OP == OP_SIGMOID || OP == OP_SILU || OP == OP_DROP))
        if (r.skew) return launch_k<OP, BWD, T, true, false, false>(a, r, blocks, st);
    return pairs ? launch_k<OP, BWD, T, false, true, false>(a, r, blocks, st)
                 : launch_k<OP, BWD, T, false, false, false>(a, r, blocks, st);
}

template <int OP, bool BWD>
cudaError_t launch_op(const NormArgs &a, const Ring &r, int size, bool pairs, int blocks,
                      cudaStream_t st) {
    return size == 4 ? launch_t<OP, BWD, float>(a, r, pairs, blocks, st)
                     : launch_t<OP, BWD, __nv_bfloat16>(a, r, pairs, blocks, st);
}

template <bool BWD>
cudaError_t launch_b(const NormArgs &a, const Ring &r, int op, int size, bool pairs, int blocks,
                     cudaStream_t st) {
    switch (op) {
        case OP_NORM: return launch_op<OP_NORM, BWD>(a, r, size, pairs, blocks, st);
        case OP_SIGMOID: return launch_op<OP_SIGMOID, BWD>(a, r, size, pairs, blocks, st);
        case OP_SILU: return launch_op<OP_SILU, BWD>(a, r, size, pairs, blocks, st);
        case OP_DROP: return launch_op<OP_DROP, BWD>(a, r, size, pairs, blocks, st);
    }
    return launch_op<OP_RESIDUAL, BWD>(a, r, size, pairs, blocks, st);
}

}  // namespace

int norm_ring_blocks(const NormArgs &a, int op, bool bwd, int size, bool pairs) {
    const Ring r = ring_for(a, op, bwd, size, pairs);
    const bool gated = op == OP_SIGMOID || op == OP_SILU;
    const int sms = device_sms();
    // fewer than a few tiles per SM: the ring would not fill, and its start costs more
    if (!r.arrays || r.stages < 2 || r.tiles < 4ll * sms) return 0;
    // forward passes with more than a warp per row go as shifted pieces (fp32, 20,011 x
    // 1,001: 49 us, and 55 this way; but BF16 52 and 41), those with a warp this way (BF16,
    // 72,896 x 281: 54, and 79 as shifted pieces)
    if (pairs && !bwd && r.tpr > 32) return 0;
    // fp32 needs half as many threads for the same bytes in flight, and is often faster
    // straight into registers (128 M elements): residual norm forward, 4,096 304 us, and
    // 337 this way, 3,200 303 and 345; backward where all threads have work, 128 396 and
    // 429, 4,096 408 and 444, but 8,192 446 and 428, 2,560 465 and 435, 96 457 and 435;
    // gated norm of 4 x 128, forward 255 and 244, backward with a sigmoid 404 and 428, of
    // 8 x 1,024 with SiLU 452 and 447.
    if (size == 4 && !pairs) {
        const bool full = a.D == r.tpr * 16;
        if (bwd ? full && r.work == kWork && r.tpr <= 256 && op != OP_SILU
                : !gated && (full || r.tpr > 32))
            return 0;
    }
    // Tokens apart: a copy moves a token, and copies of less than 2 KB are too slow (BF16
    // forward, 160,000 x 1 x 128: 28 us without the ring, 79 this way; 40,000 x 8 x 128:
    // 54 and 50; 20,000 x 56 x 128: 182 and 134, backward 278 and 229).  Not for fp32
    // (backward, 10,000 x 32 x 128: 130 and 141) nor rows of more than a warp (forward,
    // 160,000 x 1 x 1,024: 170 and 190).
    if (a.strided && (size != 2 || !gated || r.tpr > 32 || a.heads * (long long)a.D * size < 2048))
        return 0;
    return sms;
}

cudaError_t launch_norm_ring(const NormArgs &a, int op, bool bwd, int size, bool pairs,
                             cudaStream_t st) {
    const Ring r = ring_for(a, op, bwd, size, pairs);
    const int blocks = norm_ring_blocks(a, op, bwd, size, pairs);
    return bwd ? launch_b<true>(a, r, op, size, pairs, blocks, st)
               : launch_b<false>(a, r, op, size, pairs, blocks, st);
}

}  // namespace kda
