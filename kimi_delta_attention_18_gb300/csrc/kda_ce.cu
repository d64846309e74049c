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
#include "kda_gemm_kernel.cuh"

namespace kda {
namespace {

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

// ------------------------------------------------------------------ host side
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
    GemmArgs p = one_product();
    p.M = desc->tokens;
    p.N = desc->vocab;
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
        GemmArgs p = one_product();
        p.status = dev_status;
        p.pairs = l.pairs;
        p.chunk = l.chunk;
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
            GemmArgs q = one_product();
            q.status = dev_status;
            q.pairs = l.pairs;
            q.unit = unit;
            q.chunk = l.chunk;
            q.splits = l.dx_splits;
            q.M = T;
            q.N = q.cols = D;
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
            GemmArgs q = one_product();
            q.status = dev_status;
            q.pairs = l.pairs;
            q.unit = unit;
            q.chunk = l.chunk;
            q.splits = l.dw_splits;
            q.M = cols;
            q.N = q.cols = D;
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
