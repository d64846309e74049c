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
// of two, part of a warp up to a whole block) with NV pieces each, so both sums a
// row needs are one reduction (sum e n = r sum e x needs no r first) and nothing
// is read twice.  dw is summed per thread in fp32 over the block's rows, then per
// block in shared memory, then by a second kernel over the blocks in block order:
// no atomics, the same result every time.
#include <math.h>

#include "kda_internal.cuh"
#include "kda_sm100.cuh"
#include "kda_vec.cuh"

namespace kda {
namespace {

using sm100::griddep_launch_dependents;
using sm100::griddep_wait;

constexpr int kMaxWidth = 16384;

struct NormArgs {
    const void *x, *gate, *d_out, *d_res;  // residual: x = h (forward) or h' (backward)
    const float *w;                        // NULL: ones
    void *o1, *o2;      // gated: y | dx, dz      residual: h', n | dh, dy
    float *partial;     // backward: [blocks][D]
    long long rows;
    long long x_stride, gate_stride;  // elements between tokens
    int heads, D, tpr, strided;
    int act;
    float eps, scale, inv_d;
};

__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

// Sums a and b over the tpr threads of this row (every thread gets the result).
__device__ __forceinline__ void row_sum2(float &a, float &b, int tpr, float2 *red) {
    const int w = tpr < 32 ? tpr : 32;
    for (int o = w >> 1; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (tpr > 32) {  // the block holds one row
        const int nw = tpr >> 5;
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(a, b);
        __syncthreads();
        const float2 v = (threadIdx.x & 31) < nw ? red[threadIdx.x & 31] : make_float2(0.f, 0.f);
        a = v.x;
        b = v.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            b += __shfl_xor_sync(0xffffffffu, b, o);
        }
        __syncthreads();
    }
}

// VEC weights from column c on (ones without a weight).
template <int VEC>
__device__ __forceinline__ void load_w(const float *w, int c, float (&v)[VEC]) {
    if (!w) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] = 1.f;
    } else if (VEC == 1) {
        v[0] = w[c];
    } else {
#pragma unroll
        for (int j = 0; j < VEC; j += 4) {
            const float4 q = *(const float4 *)(w + c + j);
            v[j] = q.x;
            v[(j + 1) % VEC] = q.y;
            v[(j + 2) % VEC] = q.z;
            v[(j + 3) % VEC] = q.w;
        }
    }
}

enum { GATED = 0, RESIDUAL = 1 };

template <int KIND, bool BWD, typename T, int VEC, int NV>
__global__ void __launch_bounds__(VEC == 1 && NV > 4 ? 1024 : 512)
    norm_kernel(const __grid_constant__ NormArgs p) {
    extern __shared__ float sh[];
    __shared__ float2 red[32];
    using P = Piece<T, VEC>;
    const int groups = blockDim.x / p.tpr, group = threadIdx.x / p.tpr,
              lane = threadIdx.x - group * p.tpr;
    const T *x = (const T *)p.x, *gate = (const T *)p.gate, *d_out = (const T *)p.d_out,
            *d_res = (const T *)p.d_res;
    T *o1 = (T *)p.o1, *o2 = (T *)p.o2;
    float dw[BWD ? NV * VEC : 1];
#pragma unroll
    for (int i = 0; i < (BWD ? NV * VEC : 1); ++i) dw[i] = 0.f;
    griddep_wait();

    const long long step = (long long)gridDim.x * groups;
    for (long long r0 = (long long)blockIdx.x * groups; r0 < p.rows; r0 += step) {
        const long long row = r0 + group;
        const bool live = row < p.rows;  // all threads take part in the reductions
        const long long base = row * p.D;  // contiguous arrays
        const T *xr = x + base, *gr = gate + base;
        if (KIND == GATED && p.strided) {
            const long long tok = row / p.heads, off = (row - tok * p.heads) * p.D;
            xr = x + tok * p.x_stride + off;
            gr = gate + tok * p.gate_stride + off;
        }
        P px[NV], pg[NV], pd[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + i * p.tpr) * VEC;
            const bool in = live && c < p.D;
            px[i].zero();
            pg[i].zero();
            pd[i].zero();
            if (in) {
                px[i].load(xr + c);
                if (KIND == GATED && p.act) pg[i].load(gr + c);
                if (KIND == RESIDUAL && !BWD && gate) pg[i].load(gate + base + c);
                if (KIND == RESIDUAL && BWD && d_res) pg[i].load(d_res + base + c);
                if (BWD) pd[i].load(d_out + base + c);
            }
        }
        float ss = 0.f, se = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + i * p.tpr) * VEC;
            float v[VEC], g[VEC], d[VEC];
            px[i].get(v);
            pg[i].get(g);
            pd[i].get(d);
            if (KIND == RESIDUAL && !BWD) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) v[j] = fmaf(p.scale, g[j], v[j]);
            }
#pragma unroll
            for (int j = 0; j < VEC; ++j) ss = fmaf(v[j] * p.inv_d, v[j], ss);  // the mean: D x
                                                                                // more range
            if (BWD) {
                float w[VEC];
                load_w<VEC>(c < p.D ? p.w : nullptr, c, w);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    float a = 1.f;
                    if (KIND == GATED && p.act) {
                        a = sigmoid(g[j]);
                        if (p.act == KDA_GATE_SILU) a *= g[j];
                    }
                    se = fmaf(d[j] * a * w[j], v[j], se);
                }
            }
        }
        row_sum2(ss, se, p.tpr, red);
        const float rs = rsqrtf(ss + p.eps);
        const float k = (se * rs) * p.inv_d * rs;  // n mean(e n) = x k
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + i * p.tpr) * VEC;
            if (!live || c >= p.D) continue;
            float v[VEC], g[VEC], d[VEC], a1[VEC], a2[VEC];
            px[i].get(v);
            pg[i].get(g);
            pd[i].get(d);
            float wv[VEC];
            load_w<VEC>(p.w, c, wv);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float w = wv[j];
                if (KIND == GATED) {
                    float a = 1.f, da = 0.f;
                    if (p.act) {
                        const float s = sigmoid(g[j]);
                        a = p.act == KDA_GATE_SILU ? s * g[j] : s;
                        da = p.act == KDA_GATE_SILU ? fmaf(a, 1.f - s, s) : s * (1.f - s);
                    }
                    const float n = v[j] * rs;
                    if (!BWD) {
                        a1[j] = n * w * a;
                    } else {
                        const float e = d[j] * a;
                        dw[i * VEC + j] = fmaf(e, n, dw[i * VEC + j]);
                        a1[j] = rs * fmaf(-k, v[j], e * w);
                        a2[j] = d[j] * n * w * da;
                    }
                } else if (!BWD) {
                    a1[j] = fmaf(p.scale, g[j], v[j]);
                    a2[j] = a1[j] * rs * w;
                } else {
                    const float n = v[j] * rs;
                    dw[i * VEC + j] = fmaf(d[j], n, dw[i * VEC + j]);
                    a1[j] = fmaf(rs, fmaf(-k, v[j], d[j] * w), g[j]);
                    a2[j] = p.scale * a1[j];
                }
            }
            if (o1) P::store(o1 + base + c, a1);
            if (o2 && !(KIND == GATED && !BWD)) P::store(o2 + base + c, a2);
        }
    }
    griddep_launch_dependents();
    if (!BWD || !p.partial) return;
    // dw: the block's groups in group order
    if (groups > 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const int c = (lane + i * p.tpr) * VEC + j;
                if (c < p.D) sh[group * p.D + c] = dw[(i * VEC + j) % (BWD ? NV * VEC : 1)];
            }
        __syncthreads();
        for (int c = threadIdx.x; c < p.D; c += blockDim.x) {
            float s = 0.f;
            for (int g = 0; g < groups; ++g) s += sh[g * p.D + c];
            p.partial[(size_t)blockIdx.x * p.D + c] = s;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const int c = (lane + i * p.tpr) * VEC + j;
                if (c < p.D)
                    p.partial[(size_t)blockIdx.x * p.D + c] = dw[(i * VEC + j) % (BWD ? NV * VEC : 1)];
            }
    }
}

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

struct Shape {
    int vec, nv, tpr, threads, blocks, groups;
};

// A row's pieces over tpr threads.  16-byte pieces when every row of every array
// starts on a 16-byte boundary, single elements otherwise.  Rows of up to 32 x 4
// pieces stay inside a warp (no block barrier); longer rows take a block each with
// four pieces per thread (eight or more only where 512 threads do not reach).
Shape norm_shape(int D, int vec, long long rows) {
    Shape s;
    s.vec = vec;
    const int pieces = (D + vec - 1) / vec;
    int tpr = 8;
    while (tpr < 32 && tpr < pieces) tpr *= 2;
    if (pieces > 32 * 4)
        while (tpr < 512 && tpr * 4 < pieces) tpr *= 2;
    if (vec == 1 && pieces > 512 * 8) tpr = 1024;
    const int nv = (pieces + tpr - 1) / tpr;
    s.nv = nv <= 1 ? 1 : nv <= 2 ? 2 : nv <= 4 ? 4 : nv <= 8 ? 8 : 16;
    s.tpr = tpr;
    s.threads = tpr > 256 ? tpr : 256;
    if (tpr > 32) s.threads = tpr;
    s.groups = s.threads / tpr;
    int dev = 0, sms = 152;
    if (cudaGetDevice(&dev) == cudaSuccess)
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const long long need = (rows + s.groups - 1) / s.groups;
    const long long most = (long long)sms * (2048 / s.threads);
    s.blocks = (int)(need < most ? need : most);
    return s;
}

template <int KIND, bool BWD, typename T, int VEC>
cudaError_t launch_nv(const NormArgs &a, const Shape &s, cudaStream_t st) {
    const size_t smem = BWD && s.groups > 1 ? (size_t)s.groups * a.D * sizeof(float) : 0;
    const dim3 g(s.blocks), b(s.threads);
    switch (s.nv) {  // norm_shape: NV VEC <= 32
        case 1: return launch_dependent(norm_kernel<KIND, BWD, T, VEC, 1>, g, b, smem, st, a);
        case 2: return launch_dependent(norm_kernel<KIND, BWD, T, VEC, 2>, g, b, smem, st, a);
        case 4: return launch_dependent(norm_kernel<KIND, BWD, T, VEC, 4>, g, b, smem, st, a);
    }
    if constexpr (VEC <= 4) {
        if (s.nv == 8)
            return launch_dependent(norm_kernel<KIND, BWD, T, VEC, 8>, g, b, smem, st, a);
    }
    if constexpr (VEC == 1) {
        if (s.nv == 16)
            return launch_dependent(norm_kernel<KIND, BWD, T, VEC, 16>, g, b, smem, st, a);
    }
    return cudaErrorInvalidValue;
}

template <int KIND, bool BWD>
cudaError_t launch_norm(const NormArgs &a, int act_dtype, const Shape &s, cudaStream_t st) {
    if (act_dtype == KDA_DTYPE_F32)
        return s.vec == 1 ? launch_nv<KIND, BWD, float, 1>(a, s, st)
                          : launch_nv<KIND, BWD, float, 4>(a, s, st);
    return s.vec == 1 ? launch_nv<KIND, BWD, __nv_bfloat16, 1>(a, s, st)
                      : launch_nv<KIND, BWD, __nv_bfloat16, 8>(a, s, st);
}

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

// 16-byte pieces if every array's base (the weight's too), width and token stride
// allow them, else single elements; 0 if a base is not aligned to its element.
int pick_vec(const kda_norm_desc_t *d, const float *weight, const void *const *ptrs, int n) {
    const int size = d->act_dtype == KDA_DTYPE_BF16 ? 2 : 4, full = 16 / size;
    bool wide = (uintptr_t)weight % 16 == 0 && d->width % full == 0 && d->x_stride % full == 0 && d->gate_stride % full == 0;
    for (int i = 0; i < n; ++i) {
        if ((uintptr_t)ptrs[i] % size) return 0;
        if ((uintptr_t)ptrs[i] % 16) wide = false;
    }
    return wide ? full : 1;
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
    a.act = d->gate;
    a.eps = d->eps;
    a.scale = 1.f;
    a.inv_d = 1.f / (float)d->width;
    return a;
}

// Blocks any backward shape of these rows can take (the workspace's rows).
size_t norm_ws(const kda_norm_desc_t *d) {
    const long long rows = (long long)d->tokens * d->heads;
    size_t most = 0;
    const int full = d->act_dtype == KDA_DTYPE_BF16 ? 8 : 4;
    for (int vec : {1, full}) {
        const Shape s = norm_shape(d->width, vec, rows);
        if ((size_t)s.blocks > most) most = s.blocks;
    }
    return (most * d->width * sizeof(float) + 255) & ~(size_t)255;
}

template <int KIND>
kda_status_t backward(const kda_norm_desc_t *d, NormArgs &a, float *dw, int vec, void *workspace,
                      size_t workspace_bytes, cudaStream_t st) {
    if (a.rows == 0) {
        if (dw && cudaMemsetAsync(dw, 0, (size_t)d->width * sizeof(float), st) != cudaSuccess)
            return KDA_ERR_CUDA;
        return KDA_OK;
    }
    const Shape s = norm_shape(d->width, vec, a.rows);
    a.tpr = s.tpr;
    if (dw) {
        const size_t need = (size_t)s.blocks * d->width * sizeof(float);
        if (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 15u))
            return KDA_ERR_WORKSPACE;
        a.partial = (float *)workspace;
    }
    if (launch_norm<KIND, true>(a, d->act_dtype, s, st) != cudaSuccess) return KDA_ERR_CUDA;
    if (dw && launch_dependent(norm_dw_kernel, dim3((d->width + 31) / 32), dim3(1024), 0, st,
                               (const float *)workspace, dw, s.blocks, d->width) != cudaSuccess)
        return KDA_ERR_CUDA;
    return KDA_OK;
}

bool bad4(const void *p) { return ((uintptr_t)p & 3u) != 0; }

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

size_t kda_norm_backward_workspace_size(const kda_norm_desc_t *desc) {
    if (check(desc) != KDA_OK) return 0;
    return norm_ws(desc);
}

kda_status_t kda_gated_norm_forward(const kda_norm_desc_t *desc, const void *x, const void *gate,
                                    const float *weight, void *out, void *stream) {
    kda_status_t rc = check(desc);
    if (rc != KDA_OK) return rc;
    if (desc->tokens == 0) return KDA_OK;
    if (!x || !out || (!gate != (desc->gate == KDA_GATE_NONE)) || bad4(weight))
        return KDA_ERR_INVALID_ARG;
    const void *ptrs[] = {x, gate, out};
    const int vec = pick_vec(desc, weight, ptrs, 3);
    if (!vec) return KDA_ERR_INVALID_ARG;
    NormArgs a = make_args(desc);
    a.x = x; a.gate = gate; a.w = weight; a.o1 = out;
    const Shape s = norm_shape(desc->width, vec, a.rows);
    a.tpr = s.tpr;
    return launch_norm<GATED, false>(a, desc->act_dtype, s, (cudaStream_t)stream) == cudaSuccess
               ? KDA_OK : KDA_ERR_CUDA;
}

kda_status_t kda_gated_norm_backward(const kda_norm_desc_t *desc, const void *d_out, const void *x,
                                     const void *gate, const float *weight, void *dx, void *d_gate,
                                     float *d_weight, void *workspace, size_t workspace_bytes,
                                     void *stream) {
    kda_status_t rc = check(desc);
    if (rc != KDA_OK) return rc;
    if (bad4(weight) || bad4(d_weight)) return KDA_ERR_INVALID_ARG;
    if (desc->tokens > 0 && (!x || !d_out || !dx || (!gate != (desc->gate == KDA_GATE_NONE)) ||
                             (!d_gate != (desc->gate == KDA_GATE_NONE))))
        return KDA_ERR_INVALID_ARG;
    const void *ptrs[] = {x, gate, d_out, dx, d_gate};
    const int vec = pick_vec(desc, weight, ptrs, 5);
    if (!vec) return KDA_ERR_INVALID_ARG;
    NormArgs a = make_args(desc);
    a.x = x; a.gate = gate; a.d_out = d_out; a.w = weight; a.o1 = dx; a.o2 = d_gate;
    return backward<GATED>(desc, a, d_weight, vec, workspace, workspace_bytes, (cudaStream_t)stream);
}

kda_status_t kda_residual_norm_forward(const kda_norm_desc_t *desc, const void *h, const void *y,
                                       const float *weight, float scale, void *h_out, void *out,
                                       void *stream) {
    kda_status_t rc = check(desc);
    if (rc != KDA_OK) return rc;
    if (desc->heads != 1 || desc->gate != KDA_GATE_NONE || desc->x_stride || desc->gate_stride ||
        !isfinite(scale))
        return KDA_ERR_INVALID_ARG;
    if (desc->tokens == 0) return KDA_OK;
    if (!h || !out || (!y != !h_out) || bad4(weight)) return KDA_ERR_INVALID_ARG;
    const void *ptrs[] = {h, y, h_out, out};
    const int vec = pick_vec(desc, weight, ptrs, 4);
    if (!vec) return KDA_ERR_INVALID_ARG;
    NormArgs a = make_args(desc);
    a.x = h; a.gate = y; a.w = weight; a.scale = scale; a.o1 = h_out; a.o2 = out;
    const Shape s = norm_shape(desc->width, vec, a.rows);
    a.tpr = s.tpr;
    return launch_norm<RESIDUAL, false>(a, desc->act_dtype, s, (cudaStream_t)stream) == cudaSuccess
               ? KDA_OK : KDA_ERR_CUDA;
}

kda_status_t kda_residual_norm_backward(const kda_norm_desc_t *desc, const void *d_out,
                                        const void *d_h_out, const void *h_out, const float *weight,
                                        float scale, void *dh, void *dy, float *d_weight,
                                        void *workspace, size_t workspace_bytes, void *stream) {
    kda_status_t rc = check(desc);
    if (rc != KDA_OK) return rc;
    if (desc->heads != 1 || desc->gate != KDA_GATE_NONE || desc->x_stride || desc->gate_stride ||
        !isfinite(scale) || bad4(weight) || bad4(d_weight))
        return KDA_ERR_INVALID_ARG;
    if (desc->tokens > 0 && (!d_out || !h_out || !dh)) return KDA_ERR_INVALID_ARG;
    const void *ptrs[] = {d_out, d_h_out, h_out, dh, dy};
    const int vec = pick_vec(desc, weight, ptrs, 5);
    if (!vec) return KDA_ERR_INVALID_ARG;
    NormArgs a = make_args(desc);
    a.x = h_out; a.d_out = d_out; a.d_res = d_h_out; a.w = weight; a.scale = scale;
    a.o1 = dh; a.o2 = dy;
    return backward<RESIDUAL>(desc, a, d_weight, vec, workspace, workspace_bytes,
                              (cudaStream_t)stream);
}

}  // extern "C"
