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
#include "kda_f2.cuh"
#include "kda_gemm_kernel.cuh"
#include "kda_vec.cuh"

namespace kda {
namespace {

// Few tokens: the weight's bytes bound the block, and a tile of 128 rows would be mostly empty.
// A warp takes two channels, four rows of W, and their products with every token's x, in fp32
// pairs; where channels are few, up to eight warps share two of them, a slice of D each, and
// their sums are joined in order.
// BF16, one token: 7,168 x 14,336 65.0 us, by tiles 68.5; 1,024 x 2,816 5.3 and 8.4.  Two: 4,096 x
// 4,096 16.4 and 23.3, 2,048 x 5,632 15.0 and 15.4, 4,096 x 10,240 33.6 and 33.4; element by element
// (odd widths) 515 x 1,003 4.7 and 8.2, 1,001 x 2,817 14.4 and 13.5, 2,046 x 5,633 35 and 30.
// fp32: eight tokens 512 x 1,408 16.6 and 17.6, 4,096 x 4,096 66 and 103, 7,168 x 14,336 303 and
// 345 (one to four 124-128).
constexpr int kFewWarps = 8;
bool few(const kda_ffn_desc_t *d) {
    if (d->act_dtype != KDA_DTYPE_BF16) return d->tokens <= 8;
    const long long most = 1ll << (d->width % 8 == 0 ? 24 : 21);  // weights of each projection
    return d->tokens == 1 || (d->tokens == 2 && (long long)d->width * d->hidden <= most);
}

template <typename T, int VEC>
__device__ __forceinline__ void widen(const Piece<T, VEC> &p, f2 (&v)[(VEC + 1) / 2]) {
    float t[VEC];
    p.get(t);
#pragma unroll
    for (int j = 0; j < (VEC + 1) / 2; ++j) v[j] = pk(t[2 * j], VEC == 1 ? 0.f : t[(2 * j + 1) % VEC]);
}

template <typename T, int NT, int VEC>
__global__ void __launch_bounds__(32 * kFewWarps, NT <= 2 ? 4 : 2)
    ffn_few_kernel(const T *x, const T *w, T *h, int tokens, int D, int F, int act, int slices) {
    constexpr int VP = (VEC + 1) / 2, UNROLL = VEC == 1 ? 4 : 2;
    __shared__ float sums[kFewWarps][4 * NT];
    griddep_wait();
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, slice = warp % slices;
    const int f0 = 2 * (blockIdx.x * (kFewWarps / slices) + warp / slices);
    f2 acc[4][NT];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[r][t] = 0;
    if (f0 < F) {
        const int pieces = D / VEC;  // VEC: D is a multiple of it
        const int begin = (int)((long long)pieces * slice / slices),
                  end = (int)((long long)pieces * (slice + 1) / slices);
        const T *rows[4];
#pragma unroll
        for (int r = 0; r < 4; ++r)  // gate, gate, up, up
            rows[r] = w + ((size_t)(r >> 1) * F + min(f0 + (r & 1), F - 1)) * D;
#pragma unroll UNROLL
        for (int i = begin + lane; i < end; i += 32) {
            Piece<T, VEC> pw[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) pw[r].load(rows[r] + (size_t)i * VEC);
            f2 v[4][VP];
#pragma unroll
            for (int r = 0; r < 4; ++r) widen(pw[r], v[r]);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                Piece<T, VEC> px;
                px.load(x + (size_t)min(t, tokens - 1) * D + (size_t)i * VEC);
                f2 u[VP];
                widen(px, u);
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int j = 0; j < VP; ++j) acc[r][t] = fma2(v[r][j], u[j], acc[r][t]);
            }
        }
    }
    float s[4][NT];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const float2 v = un(acc[r][t]);
            s[r][t] = v.x + v.y;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s[r][t] += __shfl_xor_sync(0xffffffffu, s[r][t], o);
        }
    if (slices > 1) {
        if (lane == 0)
#pragma unroll
            for (int i = 0; i < 4 * NT; ++i) sums[warp][i] = s[i / NT][i % NT];
        __syncthreads();
        if (slice > 0) return;
#pragma unroll
        for (int i = 0; i < 4 * NT; ++i) {
            s[i / NT][i % NT] = 0.f;
            for (int k = 0; k < slices; ++k) s[i / NT][i % NT] += sums[warp + k][i];
        }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            if (lane != 2 * t + r || t >= tokens || f0 + r >= F) continue;
            float f, df;
            glu_act(act, s[r][t], f, df);
            act_st(h, (size_t)t * F + f0 + r, f * s[2 + r][t]);
        }
}

template <typename T, int VEC>
cudaError_t launch_few(const void *x, const void *w, void *h, const kda_ffn_desc_t *d, cudaStream_t st) {
    const int F = d->hidden, tasks = (F + 1) / 2, sms = device_sms();
    int slices = 1;  // as many warps as the SMs hold
    while (slices < kFewWarps && (long long)tasks * slices < 32ll * sms &&
           d->width / VEC >= 64 * slices)
        slices *= 2;
    const dim3 grid(cdiv(tasks, kFewWarps / slices)), block(32 * kFewWarps);
    const int n = d->tokens;
    const auto kernel = n == 1   ? ffn_few_kernel<T, 1, VEC>
                        : n == 2 ? ffn_few_kernel<T, 2, VEC>
                        : n <= 4 ? ffn_few_kernel<T, sizeof(T) == 4 ? 4 : 2, VEC>
                                 : ffn_few_kernel<T, sizeof(T) == 4 ? 8 : 2, VEC>;
    return launch_dependent(kernel, grid, block, 0, st, (const T *)x, (const T *)w, (T *)h, n,
                            d->width, F, (int)d->act, slices);
}

struct Layout {
    bool f32, pack, w32;
    int planes, pairs, chunk, pitch, piece, pieces, dx_splits, dw_splits;
    size_t xp, wp, dz, acc, dw_acc, total;
};

// Channels whose da and db are held at once: 1 GiB of them, 512 channels at least, in equal
// pieces of whole column tiles.
int piece_cols(const kda_ffn_desc_t *d, int planes) {
    const long long all = (long long)cdiv(d->hidden, BN) * BN;
    long long cols = (1ll << 30) / ((long long)(d->tokens > 0 ? d->tokens : 1) * planes * 4);
    cols = cols / BN * BN;  // so that the pieces' rounding up stays within it
    if (cols < 512) cols = 512;
    if (cols >= all) return (int)all;
    return cdiv(cdiv(all, cdiv(all, cols)), BN) * BN;
}

Layout layout_for(const kda_ffn_desc_t *d, bool backward) {
    Layout l = {};
    const size_t T = d->tokens, F = d->hidden;
    const int D = d->width;
    l.f32 = d->act_dtype == KDA_DTYPE_F32;
    l.planes = l.f32 ? 3 : 1;
    l.pairs = l.f32 ? 6 : 1;
    // fp32: h and its gradients within 6e-7 of 64 bits (eight stages to an accumulator: 1.1e-6,
    // 2,000 x 2,048 x 3,000 gradient 3 % faster; two: 4e-7, 13 % slower)
    l.chunk = l.f32 ? 4 : kChunkBf16;
    // copies with a pitch of whole 128-byte lines: fp32 in terms, and BF16 rows that a
    // tensor map cannot address
    l.pack = (l.f32 || D % 8 != 0) && (backward || !few(d));
    // fp32, one row of tiles: W is split into its terms on the way (7,168 x 14,336, 9 to 128
    // tokens: 345 us, copied in terms first 707)
    l.w32 = l.f32 && l.pack && !backward && d->tokens <= BM && D % 4 == 0;
    l.pitch = l.pack ? (D + 63) / 64 * 64 : D;
    if (l.pack) {
        l.xp = round256(T * l.pitch * l.planes * 2);
        l.wp = l.w32 ? 0 : round256(2 * F * l.pitch * l.planes * 2);
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
    wp = l.pack && !l.w32 ? ws + l.xp : w;
    if (!l.pack) return cudaSuccess;
    const long long T = d->tokens, R = l.w32 ? 0 : 2ll * d->hidden, most = 16ll * device_sms();
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

// What a round of tiles takes, in the time of a pair's column (1.36 ns a stage of 64).  Measured,
// BF16: a pair's tiles of 256 columns 347 ns a stage, of 192, 128 and 64 286, 285 and 283 (what
// comes from L2 then bounds them); of single CTAs 497, 425, 334 and 282.  The width it leads to is
// within 5 % of the best one from 515 x 1,003 to 7,168 x 14,336, 100 to 1,000 tokens, fp32 too.
int round_cost(bool pair, int bn) { return pair ? (bn > 210 ? bn : 210) : 154 + bn * 5 / 6; }

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
    // Few rows: the width, of pairs or of single CTAs, whose rounds over the SMs take the least
    // (7,168 x 14,336, 256 tokens: 112 pairs' tiles of 256 columns for 76 pairs 88 us, 150 of 192
    // 78; 300 tokens: 118 and 131, single CTAs 143 at best; 4,096 x 10,240, 150 tokens: 53 and 46,
    // 320 pairs' tiles of 64 93).
    const int n = device_sms(), rows = cdiv(p.M, BM);
    if (rows <= 8) {
        long long best = 0;
        for (int bn = BN; bn >= 64; bn -= 64) {
            for (int ctas = n < 2 ? 1 : 2; ctas > 0; --ctas) {
                const long long tiles = (long long)cdiv(rows, ctas) * cdiv(p.N, bn);
                const long long cost = cdiv(tiles, n / ctas) * (long long)round_cost(ctas == 2, bn);
                if (best && cost >= best) continue;
                best = cost;
                p.bn = bn;
                p.ctas = ctas;
            }
        }
    }
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
    if (few(desc)) {
        const bool vec = desc->width % (16 / size) == 0;
        const cudaError_t e =
            size == 4 ? (vec ? launch_few<float, 4>(x, weight, h, desc, st)
                             : launch_few<float, 1>(x, weight, h, desc, st))
                      : (vec ? launch_few<__nv_bfloat16, 8>(x, weight, h, desc, st)
                             : launch_few<__nv_bfloat16, 1>(x, weight, h, desc, st));
        return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
    }
    const void *xp, *wp;
    CUtensorMap tx, tw;
    if (run_pack(desc, l, x, weight, (uint8_t *)workspace, xp, wp, st) != cudaSuccess)
        return KDA_ERR_CUDA;
    GemmArgs p = one_product();
    p.M = desc->tokens;
    p.status = dev_status;
    p.act = desc->act;
    p.out = h;
    p.out_ld = desc->hidden;
    p.vec = desc->hidden % 8 == 0 && !off(h, 16);
    if (l.w32) {
        p.pairs = l.pairs;
        p.cols = desc->hidden;
        p.N = 2 * cdiv(p.cols, 64) * 64;
        p.k_blocks = cdiv(desc->width, kW32Step);
        const W32Operands o = {xp, l.pitch, (const float *)weight, 2ll * p.cols, desc->width};
        return launch_w32(EPI_GLU, p, o, st) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
    }
    if (!encode(&tx, xp, l.pitch, desc->tokens, l.planes, kMajor) ||
        !encode(&tw, wp, l.pitch, desc->hidden, 2 * l.planes, kHalfBox))
        return KDA_ERR_CUDA;
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
