// The norms around a mixer, each with its backward pass.
//
// gated norm: rows x [T][H][D] (one per token and head), gate pre-activations z,
// weight w [D]:   r = 1 / sqrt(mean(x^2) + eps),  n = x r,  y = n w a(z),
// a = sigmoid, silu or 1.  Backward, from x, z and dy alone (nothing is kept from
// the forward pass: x is read anyway, and r is one sum over it):
//     dz = dy n w a'(z),   dw = sum over rows of dy a n,
//     e = dy a w,          dx = r (e - n mean(e n)).
// residual norm: h' = h + s y,  n = h' r w over rows of D.  Backward, from h':
//     dh = dh' + r (e - n mean(e n)) with e = dn w,  dy = s dh,  dw = sum dn n.
//
// Every element is read once and written once: the pass is bound by those bytes.
// A row is held in registers, packed as it was loaded, by `tpr` threads (a power
// of two, part of a warp up to a whole block) with NV 16-byte pieces each, so both sums a
// row needs are one reduction (sum e n = r sum e x needs no r first) and nothing
// is read twice.  dw is summed per thread in fp32 over the block's rows, then per
// block in shared memory, then by a second kernel over the blocks in block order:
// no atomics, the same result every time.  Many rows take kda_norm_ring.cu, but for fp32
// ones that fill their threads.
//
// Measured on GB300: decode's 256 x 56 x 128 BF16 gate 3.6 us and 256 x 7,168 residual
// norm 5.7 us (a launch and one round of loads; their bytes are 1.6 and 2.2 us); fp32,
// 20,011 x 1,001 in shifted pieces 51 us (6.2 TB/s; by single elements 69).
#include <math.h>

#include "kda_norm_rows.cuh"

namespace kda {
namespace {

constexpr int kMaxWidth = 16384;

// dw[c] = sum over blocks of partial[b][c]: 32 columns per block, 32 row slices
// summed in order (slice by slice, then over slices).
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float *partial, float *dw, int blocks,
                                                       int D) {
    __shared__ float sh[32][33];
    griddep_wait();
    griddep_launch_dependents();
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), sl = threadIdx.x >> 5;
    float s = 0.f;
    if (c < D)
        for (int b = sl; b < blocks; b += 32) s += partial[(size_t)b * D + c];
    sh[sl][threadIdx.x & 31] = s;
    __syncthreads();
    if (sl == 0 && c < D) {
        s = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) s += sh[i][threadIdx.x];
        dw[c] = s;
    }
}

// The kernel for these rows and, in a backward pass, its number of blocks (the rows
// of `partial`).
int norm_blocks(const NormArgs &a, int op, bool bwd, int size, int move) {
    const int ring = move != BY_ELEMENT
                         ? norm_ring_blocks(a, op, bwd, size, move == SHIFTED) : 0;
    return ring ? ring : norm_shape(a.D, size, move, a.rows, bwd).blocks;
}

template <bool BWD>
cudaError_t launch_norm(NormArgs a, int op, int size, int move, cudaStream_t st) {
    if (move != BY_ELEMENT && norm_ring_blocks(a, op, BWD, size, move == SHIFTED))
        return launch_norm_ring(a, op, BWD, size, move == SHIFTED, st);
    const Shape s = norm_shape(a.D, size, move, a.rows, BWD);
    a.tpr = s.tpr;
    switch (op) {
        case OP_NORM: return launch_op<OP_NORM, BWD>(a, size, s, st);
        case OP_SIGMOID: return launch_op<OP_SIGMOID, BWD>(a, size, s, st);
        case OP_SILU: return launch_op<OP_SILU, BWD>(a, size, s, st);
        case OP_DROP: return launch_norm_drop(a, BWD, size, s, st);
    }
    return launch_op<OP_RESIDUAL, BWD>(a, size, s, st);
}

int size_of(const kda_norm_desc_t *d) { return d->act_dtype == KDA_DTYPE_BF16 ? 2 : 4; }

kda_status_t check(const kda_norm_desc_t *d) {
    if (!d) return KDA_ERR_INVALID_ARG;
    if (d->tokens < 0 || d->heads < 1 || d->width < 1) return KDA_ERR_INVALID_ARG;
    if (!(d->eps > 0.f) || !isfinite(d->eps)) return KDA_ERR_INVALID_ARG;
    if (d->act_dtype != KDA_DTYPE_F32 && d->act_dtype != KDA_DTYPE_BF16) return KDA_ERR_UNSUPPORTED;
    if (d->gate != KDA_GATE_NONE && d->gate != KDA_GATE_SIGMOID && d->gate != KDA_GATE_SILU)
        return KDA_ERR_UNSUPPORTED;
    if (d->width > kMaxWidth || d->heads > (1 << 20)) return KDA_ERR_UNSUPPORTED;
    const long long row = (long long)d->heads * d->width;
    if (d->tokens > (1ll << 42) / row) return KDA_ERR_UNSUPPORTED;
    if ((d->x_stride != 0 && d->x_stride < row) || (d->gate_stride != 0 && d->gate_stride < row))
        return KDA_ERR_INVALID_ARG;
    if (d->x_stride > (1ll << 40) || d->gate_stride > (1ll << 40)) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

// Pieces if every array's base (the weight's too), width and token stride allow them;
// shifted pieces if the bases do and the arrays are contiguous; -1 if a base is not
// aligned to its element.
int pick_move(const kda_norm_desc_t *d, const float *weight, const void *const *ptrs, int n) {
    const int size = size_of(d), full = 16 / size;
    bool wide = true;
    for (int i = 0; i < n; ++i) {
        if ((uintptr_t)ptrs[i] % size) return -1;
        if ((uintptr_t)ptrs[i] % 16) wide = false;
    }
    if (!wide) return BY_ELEMENT;
    if ((uintptr_t)weight % 16 == 0 && d->width % full == 0 && d->x_stride % full == 0 &&
        d->gate_stride % full == 0)
        return PIECES;
    const long long row = (long long)d->heads * d->width;
    return (d->x_stride == 0 || d->x_stride == row) &&
                   (d->gate_stride == 0 || d->gate_stride == row) && d->width <= kMaxWidth - 16
               ? SHIFTED : BY_ELEMENT;
}

NormArgs make_args(const kda_norm_desc_t *d) {
    NormArgs a = {};
    a.rows = (long long)d->tokens * d->heads;
    const long long row = (long long)d->heads * d->width;
    a.x_stride = d->x_stride ? d->x_stride : row;
    a.gate_stride = d->gate_stride ? d->gate_stride : row;
    a.strided = a.x_stride != row || a.gate_stride != row;
    a.heads = d->heads;
    a.D = d->width;
    a.eps = d->eps;
    a.scale = 1.f;
    a.inv_d = 1.f / (float)d->width;
    return a;
}

// The workspace holds a row of partial sums for every block of any kernel that these
// rows could take.
size_t norm_ws(const kda_norm_desc_t *d) {
    const NormArgs a = make_args(d);
    int most = device_sms();  // the ring's
    for (int move : {BY_ELEMENT, PIECES, SHIFTED}) {
        const int n = norm_shape(d->width, size_of(d), move, a.rows, true).blocks;
        most = n > most ? n : most;
    }
    return ((size_t)most * d->width * sizeof(float) + 255) & ~(size_t)255;
}

kda_status_t backward(const kda_norm_desc_t *d, NormArgs &a, int op, float *dw, int move,
                      void *workspace, size_t workspace_bytes, cudaStream_t st) {
    if (a.rows == 0) {
        if (dw && cudaMemsetAsync(dw, 0, (size_t)d->width * sizeof(float), st) != cudaSuccess)
            return KDA_ERR_CUDA;
        return KDA_OK;
    }
    const int blocks = norm_blocks(a, op, true, size_of(d), move);
    if (dw) {
        const size_t need = (size_t)blocks * d->width * sizeof(float);
        if (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 15u))
            return KDA_ERR_WORKSPACE;
        a.partial = (float *)workspace;
    }
    if (launch_norm<true>(a, op, size_of(d), move, st) != cudaSuccess) return KDA_ERR_CUDA;
    if (dw && launch_dependent(norm_dw_kernel, dim3((d->width + 31) / 32), dim3(1024), 0, st,
                               (const float *)workspace, dw, blocks, d->width) != cudaSuccess)
        return KDA_ERR_CUDA;
    return KDA_OK;
}

bool bad4(const void *p) { return ((uintptr_t)p & 3u) != 0; }

// The residual norm's passes, with y dropped out if `drop`.
kda_status_t residual_forward(const kda_norm_desc_t *desc, const kda_dropout_t *drop, const void *h,
                              const void *y, const float *weight, float scale, void *h_out,
                              void *out, int32_t *dev_status, void *stream) {
    kda_status_t rc = check(desc);
    if (rc != KDA_OK) return rc;
    if (desc->heads != 1 || desc->gate != KDA_GATE_NONE || desc->x_stride || desc->gate_stride ||
        !isfinite(scale))
        return KDA_ERR_INVALID_ARG;
    Drop keep = {};
    float kept = 1.f;
    if (drop && (rc = dropout_args(drop, desc->width, &keep, &kept)) != KDA_OK) return rc;
    if (!isfinite(scale * kept)) return KDA_ERR_INVALID_ARG;
    if (desc->tokens == 0) return KDA_OK;
    if (!h || !out || (!y != !h_out) || bad4(weight) || bad4(dev_status))
        return KDA_ERR_INVALID_ARG;
    const void *ptrs[] = {h, y, h_out, out};
    const int move = pick_move(desc, weight, ptrs, 4);
    if (move < 0) return KDA_ERR_INVALID_ARG;
    NormArgs a = make_args(desc);
    a.x = h; a.gate = y; a.w = weight; a.scale = scale * kept; a.o1 = h_out; a.o2 = out;
    a.status = dev_status;
    a.drop = keep;
    return launch_norm<false>(a, drop ? OP_DROP : OP_RESIDUAL, size_of(desc), move,
                              (cudaStream_t)stream) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status_t residual_backward(const kda_norm_desc_t *desc, const kda_dropout_t *drop,
                               const void *d_out, const void *d_h_out, const void *h_out,
                               const float *weight, float scale, void *dh, void *dy, float *d_weight,
                               void *workspace, size_t workspace_bytes, int32_t *dev_status,
                               void *stream) {
    kda_status_t rc = check(desc);
    if (rc != KDA_OK) return rc;
    if (desc->heads != 1 || desc->gate != KDA_GATE_NONE || desc->x_stride || desc->gate_stride ||
        !isfinite(scale) || bad4(weight) || bad4(d_weight) || bad4(dev_status))
        return KDA_ERR_INVALID_ARG;
    Drop keep = {};
    float kept = 1.f;
    if (drop && (rc = dropout_args(drop, desc->width, &keep, &kept)) != KDA_OK) return rc;
    if (!isfinite(scale * kept)) return KDA_ERR_INVALID_ARG;
    if (desc->tokens > 0 && (!d_out || !h_out || !dh)) return KDA_ERR_INVALID_ARG;
    const void *ptrs[] = {d_out, d_h_out, h_out, dh, dy};
    const int move = pick_move(desc, weight, ptrs, 5);
    if (move < 0) return KDA_ERR_INVALID_ARG;
    NormArgs a = make_args(desc);
    a.x = h_out; a.d_out = d_out; a.d_res = d_h_out; a.w = weight; a.scale = scale * kept;
    a.o1 = dh; a.o2 = dy;
    a.status = dev_status;
    a.drop = keep;
    return backward(desc, a, drop ? OP_DROP : OP_RESIDUAL, d_weight, move, workspace,
                    workspace_bytes, (cudaStream_t)stream);
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

size_t kda_norm_backward_workspace_size(const kda_norm_desc_t *desc) {
    if (check(desc) != KDA_OK) return 0;
    return norm_ws(desc);
}

kda_status_t kda_gated_norm_forward(const kda_norm_desc_t *desc, const void *x, const void *gate,
                                    const float *weight, void *out, int32_t *dev_status,
                                    void *stream) {
    kda_status_t rc = check(desc);
    if (rc != KDA_OK) return rc;
    if (desc->tokens == 0) return KDA_OK;
    if (!x || !out || (!gate != (desc->gate == KDA_GATE_NONE)) || bad4(weight) ||
        bad4(dev_status))
        return KDA_ERR_INVALID_ARG;
    const void *ptrs[] = {x, gate, out};
    const int move = pick_move(desc, weight, ptrs, 3);
    if (move < 0) return KDA_ERR_INVALID_ARG;
    NormArgs a = make_args(desc);
    a.x = x; a.gate = gate; a.w = weight; a.o1 = out;
    a.status = dev_status;
    return launch_norm<false>(a, desc->gate, size_of(desc), move, (cudaStream_t)stream) == cudaSuccess
               ? KDA_OK : KDA_ERR_CUDA;
}

kda_status_t kda_gated_norm_backward(const kda_norm_desc_t *desc, const void *d_out, const void *x,
                                     const void *gate, const float *weight, void *dx, void *d_gate,
                                     float *d_weight, void *workspace, size_t workspace_bytes,
                                     int32_t *dev_status, void *stream) {
    kda_status_t rc = check(desc);
    if (rc != KDA_OK) return rc;
    if (bad4(weight) || bad4(d_weight) || bad4(dev_status)) return KDA_ERR_INVALID_ARG;
    if (desc->tokens > 0 && (!x || !d_out || !dx || (!gate != (desc->gate == KDA_GATE_NONE)) ||
                             (!d_gate != (desc->gate == KDA_GATE_NONE))))
        return KDA_ERR_INVALID_ARG;
    const void *ptrs[] = {x, gate, d_out, dx, d_gate};
    const int move = pick_move(desc, weight, ptrs, 5);
    if (move < 0) return KDA_ERR_INVALID_ARG;
    NormArgs a = make_args(desc);
    a.x = x; a.gate = gate; a.d_out = d_out; a.w = weight; a.o1 = dx; a.o2 = d_gate;
    a.status = dev_status;
    return backward(desc, a, desc->gate, d_weight, move, workspace, workspace_bytes,
                    (cudaStream_t)stream);
}

kda_status_t kda_residual_norm_forward(const kda_norm_desc_t *desc, const void *h, const void *y,
                                       const float *weight, float scale, void *h_out, void *out,
                                       int32_t *dev_status, void *stream) {
    return residual_forward(desc, nullptr, h, y, weight, scale, h_out, out, dev_status, stream);
}

kda_status_t kda_residual_norm_dropout_forward(const kda_norm_desc_t *desc,
                                               const kda_dropout_t *dropout, const void *h,
                                               const void *y, const float *weight, float scale,
                                               void *h_out, void *out, int32_t *dev_status,
                                               void *stream) {
    if (!dropout || (desc && desc->tokens > 0 && !y)) return KDA_ERR_INVALID_ARG;
    return residual_forward(desc, dropout, h, y, weight, scale, h_out, out, dev_status, stream);
}

kda_status_t kda_residual_norm_backward(const kda_norm_desc_t *desc, const void *d_out,
                                        const void *d_h_out, const void *h_out, const float *weight,
                                        float scale, void *dh, void *dy, float *d_weight,
                                        void *workspace, size_t workspace_bytes,
                                        int32_t *dev_status, void *stream) {
    return residual_backward(desc, nullptr, d_out, d_h_out, h_out, weight, scale, dh, dy, d_weight,
                             workspace, workspace_bytes, dev_status, stream);
}

kda_status_t kda_residual_norm_dropout_backward(const kda_norm_desc_t *desc,
                                                const kda_dropout_t *dropout, const void *d_out,
                                                const void *d_h_out, const void *h_out,
                                                const float *weight, float scale, void *dh, void *dy,
                                                float *d_weight, void *workspace,
                                                size_t workspace_bytes, int32_t *dev_status,
                                                void *stream) {
    if (!dropout || (desc && desc->tokens > 0 && !dy)) return KDA_ERR_INVALID_ARG;
    return residual_backward(desc, dropout, d_out, d_h_out, h_out, weight, scale, dh, dy, d_weight,
                             workspace, workspace_bytes, dev_status, stream);
}

}  // extern "C"
