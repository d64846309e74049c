// The gated feed-forward block: both projections, the activation and their product,
//     a = x Wg^T,  b = x Wu^T,  h = act(a) b,      x [T][D], W [2][F][D] (Wg, then Wu),
// without a and b ever being arrays.  Backward, for d_h:
//     da = d_h b act'(a),  db = d_h act(a),  dx = da Wg + db Wu,  dWg = da^T x,  dWu = db^T x.
//
// Forward: one product whose tiles take rows of Wg and Wu in turn, 32 of each, so that a
// thread of the epilogue has both projections of its channels in registers.  Backward, per
// piece of the channels: the piece's a and b again (4 T D F operations once more; keeping
// them would cost 2 T F elements), da and db in the products' operand type, then the two
// products that read them.  fp32 operands are three BF16 terms each, six products, as in the
// cross entropy, whose kernel this is.
#include "kda_gemm_kernel.cuh"

namespace kda {
namespace {

struct Layout {
    bool f32, pack;
    int planes, pairs, chunk, pitch, piece, pieces, dx_splits, dw_splits;
    size_t xp, wp, dz, acc, dw_acc, total;
};

// Channels whose da and db are held at once: 1 GiB of them, 512 channels at least, in equal
// pieces of whole column tiles.
int piece_cols(const kda_ffn_desc_t *d, int planes) {
    const long long all = (long long)cdiv(d->hidden, BN) * BN;
    long long cols = (1ll << 30) / ((long long)(d->tokens > 0 ? d->tokens : 1) * planes * 4);
    if (cols < 512) cols = 512;
    if (cols < all) cols = cdiv(all, cdiv(all, cols));
    cols = (long long)cdiv(cols, BN) * BN;
    return (int)(cols < all ? cols : all);
}

Layout layout_for(const kda_ffn_desc_t *d, bool backward) {
    Layout l = {};
    const size_t T = d->tokens, F = d->hidden;
    const int D = d->width;
    l.f32 = d->act_dtype == KDA_DTYPE_F32;
    l.planes = l.f32 ? 3 : 1;
    l.pairs = l.f32 ? 6 : 1;
    l.chunk = l.f32 ? kChunkF32 : kChunkBf16;
    // copies with a pitch of whole 128-byte lines: fp32 in terms, and BF16 rows that a
    // tensor map cannot address
    l.pack = l.f32 || D % 8 != 0;
    l.pitch = l.pack ? (D + 63) / 64 * 64 : D;
    if (l.pack) {
        l.xp = round256(T * l.pitch * l.planes * 2);
        l.wp = round256(2 * F * l.pitch * l.planes * 2);
    }
    if (backward) {
        l.piece = piece_cols(d, l.planes);
        l.pieces = cdiv(F, l.piece);
        l.dz = round256(2 * T * l.piece * l.planes * 2);
        const int last = (int)F - (l.pieces - 1) * l.piece;
        l.dx_splits = splits_for(T, D, BN, cdiv(last, BK), 2 * l.pairs);
        l.dw_splits = l.pieces > 1 ? 1 : splits_for(2 * F, D, BN, cdiv(T, BK), l.pairs);
        if (l.pieces > 1 || l.dx_splits > 1) l.acc = round256((size_t)l.dx_splits * T * D * 4);
        if (l.dw_splits > 1) l.dw_acc = round256((size_t)l.dw_splits * 2 * F * D * 4);
    }
    l.total = l.xp + l.wp + l.dz + l.acc + l.dw_acc;
    return l;
}

kda_status_t check(const kda_ffn_desc_t *d) {
    if (!d) return KDA_ERR_INVALID_ARG;
    if (d->tokens < 0 || d->hidden < 1 || d->width < 1) return KDA_ERR_INVALID_ARG;
    if (d->act_dtype != KDA_DTYPE_F32 && d->act_dtype != KDA_DTYPE_BF16) return KDA_ERR_UNSUPPORTED;
    if (d->act != KDA_FFN_SIGMOID && d->act != KDA_FFN_SILU && d->act != KDA_FFN_GELU)
        return KDA_ERR_UNSUPPORTED;
    // tile and coordinate arithmetic is 32-bit
    if (d->tokens > (1 << 24) || d->hidden > (1 << 20) || d->width > (1 << 17))
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

// x and W as the products read them.
cudaError_t run_pack(const kda_ffn_desc_t *d, const Layout &l, const void *x, const void *w,
                     uint8_t *ws, const void *&xp, const void *&wp, cudaStream_t st) {
    xp = l.pack ? ws : x;
    wp = l.pack ? ws + l.xp : w;
    if (!l.pack) return cudaSuccess;
    const long long T = d->tokens, R = 2ll * d->hidden, most = 16ll * device_sms();
    const long long need = ((T + R) * (l.pitch / 8) + 255) / 256;
    const dim3 grid((unsigned)(need < most ? need : most));
    __nv_bfloat16 *to = (__nv_bfloat16 *)ws, *to_w = (__nv_bfloat16 *)(ws + l.xp);
    if (l.f32)
        return launch_dependent(pack_kernel<float>, grid, dim3(256), 0, st, (const float *)x, T, to,
                                (const float *)w, R, to_w, d->width, l.pitch, l.planes, Targets{},
                                (const float *)nullptr, (float *)nullptr);
    return launch_dependent(pack_kernel<__nv_bfloat16>, grid, dim3(256), 0, st,
                            (const __nv_bfloat16 *)x, T, to, (const __nv_bfloat16 *)w, R, to_w,
                            d->width, l.pitch, l.planes, Targets{}, (const float *)nullptr,
                            (float *)nullptr);
}

// Both projections of `cols` channels from the v0-th on, with the epilogue EPI.
template <int EPI>
cudaError_t run_glu(GemmArgs p, const Layout &l, const CUtensorMap &tx, const CUtensorMap &tw,
                    int v0, int cols, int width, cudaStream_t st) {
    p.pairs = l.pairs;
    p.chunk = l.chunk;
    p.planes = l.planes;
    p.cols = cols;
    p.N = 2 * cdiv(cols, 64) * 64;
    p.b_row0 = v0;
    p.k_blocks = cdiv(width, BK);
    if (l.f32) return run_gemm<EPI, false, false, true, false>(p, tx, tw, st);
    return p.k_blocks > kLongStages ? run_gemm<EPI, false, false, true, true>(p, tx, tw, st)
                                    : run_gemm<EPI, false, false, false, true>(p, tx, tw, st);
}

constexpr int kHalfBox = 32;  // rows of W in a box

int size_of(const kda_ffn_desc_t *d) { return d->act_dtype == KDA_DTYPE_BF16 ? 2 : 4; }
bool off(const void *p, int size) { return ((uintptr_t)p & (size - 1)) != 0; }

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

size_t kda_gated_ffn_workspace_size(const kda_ffn_desc_t *desc, int32_t backward) {
    if (check(desc) != KDA_OK || desc->tokens == 0) return 0;
    return layout_for(desc, backward != 0).total;
}

kda_status_t kda_gated_ffn_forward(const kda_ffn_desc_t *desc, const void *x, const void *weight,
                                   void *h, void *workspace, size_t workspace_bytes,
                                   int32_t *dev_status, void *stream) {
    const kda_status_t rc = check(desc);
    if (rc != KDA_OK) return rc;
    if (off(dev_status, 4)) return KDA_ERR_INVALID_ARG;
    if (desc->tokens == 0) return KDA_OK;
    const int size = size_of(desc);
    if (bad16(x) || bad16(weight) || !h || off(h, size)) return KDA_ERR_INVALID_ARG;
    const Layout l = layout_for(desc, false);
    if (l.total > 0 && (!workspace || workspace_bytes < l.total || off(workspace, 16)))
        return KDA_ERR_WORKSPACE;
    cudaStream_t st = (cudaStream_t)stream;
    const void *xp, *wp;
    CUtensorMap tx, tw;
    if (run_pack(desc, l, x, weight, (uint8_t *)workspace, xp, wp, st) != cudaSuccess ||
        !encode(&tx, xp, l.pitch, desc->tokens, l.planes, kMajor) ||
        !encode(&tw, wp, l.pitch, desc->hidden, 2 * l.planes, kHalfBox))
        return KDA_ERR_CUDA;
    GemmArgs p = one_product();
    p.M = desc->tokens;
    p.status = dev_status;
    p.act = desc->act;
    p.out = h;
    p.out_ld = desc->hidden;
    p.vec = desc->hidden % 8 == 0 && !off(h, 16);
    return run_glu<EPI_GLU>(p, l, tx, tw, 0, desc->hidden, desc->width, st) == cudaSuccess
               ? KDA_OK : KDA_ERR_CUDA;
}

kda_status_t kda_gated_ffn_backward(const kda_ffn_desc_t *desc, const void *d_h, const void *x,
                                    const void *weight, void *dx, void *d_weight, void *workspace,
                                    size_t workspace_bytes, int32_t *dev_status, void *stream) {
    const kda_status_t rc = check(desc);
    if (rc != KDA_OK) return rc;
    const int size = size_of(desc);
    cudaStream_t st = (cudaStream_t)stream;
    if (off(dx, size) || off(d_weight, size) || off(dev_status, 4)) return KDA_ERR_INVALID_ARG;
    const int T = desc->tokens, F = desc->hidden, D = desc->width;
    if (T == 0) {
        if (d_weight && cudaMemsetAsync(d_weight, 0, 2ull * F * D * size, st) != cudaSuccess)
            return KDA_ERR_CUDA;
        return KDA_OK;
    }
    if (bad16(x) || bad16(weight) || !d_h || off(d_h, size)) return KDA_ERR_INVALID_ARG;
    if (!dx && !d_weight) return KDA_OK;
    const Layout l = layout_for(desc, true);
    if (!workspace || workspace_bytes < l.total || off(workspace, 16)) return KDA_ERR_WORKSPACE;
    uint8_t *ws = (uint8_t *)workspace;
    __nv_bfloat16 *dz = (__nv_bfloat16 *)(ws + l.xp + l.wp);
    float *acc = (float *)(ws + l.xp + l.wp + l.dz), *dw_acc = acc + l.acc / 4;
    const void *xp, *wp;
    if (run_pack(desc, l, x, weight, ws, xp, wp, st) != cudaSuccess) return KDA_ERR_CUDA;
    CUtensorMap xk, xm, zk, zm, wh, wm;  // K-major and MN-major
    if (!encode(&xk, xp, l.pitch, T, l.planes, kMajor) ||
        !encode(&xm, xp, l.pitch, T, l.planes, kMnMajor) ||
        !encode(&zk, dz, l.piece, T, 2 * l.planes, kMajor) ||
        !encode(&zm, dz, l.piece, T, 2 * l.planes, kMnMajor) ||
        !encode(&wh, wp, l.pitch, F, 2 * l.planes, kHalfBox) ||
        !encode(&wm, wp, l.pitch, F, 2 * l.planes, kMnMajor))
        return KDA_ERR_CUDA;
    for (int k = 0; k < l.pieces; ++k) {
        const int v0 = k * l.piece, cols = F - v0 < l.piece ? F - v0 : l.piece;
        GemmArgs p = one_product();
        p.M = T;
        p.status = dev_status;
        p.act = desc->act;
        p.d_h = (const uint8_t *)d_h + (size_t)v0 * size;
        p.out_ld = F;
        p.vec = F % 8 == 0 && !off(d_h, 16);
        p.dz = dz;
        p.pitch = l.piece;
        if (run_glu<EPI_DGLU>(p, l, xk, wh, v0, cols, D, st) != cudaSuccess) return KDA_ERR_CUDA;
        if (dx) {
            GemmArgs q = one_product();
            q.status = dev_status;
            q.pairs = l.pairs;
            q.chunk = l.chunk;
            q.groups = q.a_group = q.b_group = 2;
            q.splits = l.dx_splits;
            q.M = T;
            q.N = q.cols = D;
            q.k_blocks = cdiv(cols, BK);
            q.bk_row0 = v0;
            q.acc_in = k > 0 ? acc : nullptr;
            if (l.dx_splits == 1 && k == l.pieces - 1) q.out = dx;
            else q.acc_out = acc;
            q.out_bf16 = size == 2;
            q.vec = D % 8 == 0 && !off(dx, 16);
            if (q.splits > q.k_blocks) return KDA_ERR_CUDA;
            if (run_backward<EPI_OUT, false, true>(q, l.f32, zk, wm, st) != cudaSuccess)
                return KDA_ERR_CUDA;
            if (l.dx_splits > 1 && k == l.pieces - 1 &&
                sum_splits(acc, dx, (long long)T * D, l.dx_splits, size == 2, st) != cudaSuccess)
                return KDA_ERR_CUDA;
        }
        if (d_weight) {
            GemmArgs q = one_product();
            q.status = dev_status;
            q.pairs = l.pairs;
            q.chunk = l.chunk;
            q.batches = q.a_group = 2;
            q.splits = l.dw_splits;
            q.M = cols;
            q.N = q.cols = D;
            q.k_blocks = cdiv(T, BK);
            if (l.dw_splits > 1) q.acc_out = dw_acc;
            else q.out = (uint8_t *)d_weight + (size_t)v0 * D * size;
            q.out_batch = (long long)F * D;
            q.out_bf16 = size == 2;
            q.vec = D % 8 == 0 && !off(d_weight, 16);
            if (run_backward<EPI_OUT, true, true>(q, l.f32, zm, xm, st) != cudaSuccess)
                return KDA_ERR_CUDA;
            if (l.dw_splits > 1 && sum_splits(dw_acc, d_weight, 2ll * F * D, l.dw_splits, size == 2,
                                              st) != cudaSuccess)
                return KDA_ERR_CUDA;
        }
    }
    return KDA_OK;
}

}  // extern "C"
