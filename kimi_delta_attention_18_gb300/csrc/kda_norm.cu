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

#include "kda_norm_math.cuh"
#include "kda_sm100.cuh"

namespace kda {
namespace {

using sm100::griddep_launch_dependents;
using sm100::griddep_wait;

constexpr int kMaxWidth = 16384;

// Sums a and b over the tpr threads of this row (every thread gets the result).
// Rows longer than a warp use `red`, another one in turn so that one barrier does.
__device__ __forceinline__ void row_sum2(float &a, float &b, int tpr, float2 *red) {
    const int w = tpr < 32 ? tpr : 32;
    for (int o = w >> 1; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (tpr > 32) {  // the block holds one row
        const int nw = tpr >> 5, lane = threadIdx.x & 31;
        if (lane == 0) red[threadIdx.x >> 5] = make_float2(a, b);
        __syncthreads();
        const float2 v = lane < nw ? red[lane] : make_float2(0.f, 0.f);
        a = v.x;
        b = v.y;
        for (int o = nw >> 1; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            b += __shfl_xor_sync(0xffffffffu, b, o);
        }
        a = __shfl_sync(0xffffffffu, a, 0);
        b = __shfl_sync(0xffffffffu, b, 0);
    }
}

// VEC weights from column c on (ones without a weight or outside the row).
template <bool SHIFT, int VEC>
__device__ __forceinline__ void weights(const float *w, int c, int D, f2 (&v)[kPairs<VEC>]) {
    float t[VEC];
    if (!w || (!SHIFT && c >= D)) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) t[j] = 1.f;
    } else if (SHIFT || VEC == 1) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) t[j] = c + j >= 0 && c + j < D ? w[c + j] : 1.f;
    } else {
#pragma unroll
        for (int j = 0; j < VEC; j += 4) {
            const float4 q = *(const float4 *)(w + c + j);
            t[j] = q.x;
            t[(j + 1) % VEC] = q.y;
            t[(j + 2) % VEC] = q.z;
            t[(j + 3) % VEC] = q.w;
        }
    }
#pragma unroll
    for (int j = 0; j < kPairs<VEC>; ++j) v[j] = pk(t[2 * j], VEC == 1 ? 1.f : t[(2 * j + 1) % VEC]);
}

// Where registers allow (AHEAD) the next row's pieces are loaded while this row is
// worked on.
template <int OP, bool BWD, typename T, int VEC, int NV, bool SHIFT>
__global__ void __launch_bounds__(VEC == 1 && NV == 16 ? 1024 : 512,
                                  BWD || (VEC == 1 && NV == 16) || VEC * NV > 16 ? 1 : 2)
    norm_kernel(const __grid_constant__ NormArgs p) {
    extern __shared__ float sh[];
    __shared__ float2 red[2][32];
    using P = Piece<T, VEC>;
    constexpr bool AHEAD = BWD && VEC > 1 && NV == 1;
    constexpr int VP = kPairs<VEC>;
    const int groups = blockDim.x / p.tpr, group = threadIdx.x / p.tpr,
              lane = threadIdx.x - group * p.tpr;
    const T *x = (const T *)p.x, *gate = (const T *)p.gate, *d_out = (const T *)p.d_out,
            *d_res = (const T *)p.d_res;
    T *o1 = (T *)p.o1, *o2 = (T *)p.o2;
    const long long step = (long long)gridDim.x * groups;
    const long long first = (long long)blockIdx.x * groups + group;
    // SHIFT: the launch makes step D a multiple of VEC, so the shift stays
    const int c0 = lane * VEC - (SHIFT ? (int)(first * p.D % VEC) : 0);
    auto column = [&](int i) { return c0 + i * p.tpr * VEC; };
    auto load_w = [&](int i, f2 (&w)[VP]) { weights<SHIFT, VEC>(p.w, column(i), p.D, w); };
    RowMath<OP, BWD, T, VEC, NV> math;
    griddep_wait();
    math.begin(load_w);

    P px[NV], pg[NV], pd[NV];
    auto load = [&](long long row, P (&px)[NV], P (&pg)[NV], P (&pd)[NV]) {
        const bool live = row < p.rows;  // all threads take part in the reductions
        const int D = live ? p.D : 0;
        const long long base = row * p.D;  // contiguous arrays
        const T *xr = x + base, *gr = gate + base;
        if (OP != OP_RESIDUAL && p.strided) {
            const long long tok = row / p.heads, off = (row - tok * p.heads) * p.D;
            xr = x + tok * p.x_stride + off;
            gr = gate + tok * p.gate_stride + off;
        }
        if (OP == OP_RESIDUAL) gr = BWD ? d_res + base : gr;
        const bool has_g = OP == OP_SIGMOID || OP == OP_SILU ||
                           (OP == OP_RESIDUAL && (BWD ? d_res != nullptr : gate != nullptr));
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            load_piece<SHIFT, T, VEC>(px[i], xr, column(i), D);
            if (has_g) load_piece<SHIFT, T, VEC>(pg[i], gr, column(i), D);
            else pg[i].zero();
            if (BWD) load_piece<SHIFT, T, VEC>(pd[i], d_out + base, column(i), D);
        }
    };
    if (AHEAD) load(first, px, pg, pd);
    int turn = 0;
    for (long long r0 = (long long)blockIdx.x * groups; r0 < p.rows; r0 += step, turn ^= 1) {
        const long long row = r0 + group;
        P nx[NV], ng[NV], nd[NV];
        if (AHEAD) load(row + step, nx, ng, nd);
        else load(row, px, pg, pd);
        float ss, se;
        math.sums(p, px, pg, pd, load_w, ss, se);
        row_sum2(ss, se, p.tpr, red[turn]);
        math.outputs(p, px, pg, pd, load_w, ss, se, [&](int i, f2 (&a1)[VP], f2 (&a2)[VP]) {
            if (row >= p.rows) return;
            const long long base = row * p.D;
            float t[VEC];
            if (o1) {
                floats<VEC>(a1, t);
                store_piece<SHIFT, T, VEC>(o1 + base, column(i), p.D, t);
            }
            if ((BWD || OP == OP_RESIDUAL) && o2) {
                floats<VEC>(a2, t);
                store_piece<SHIFT, T, VEC>(o2 + base, column(i), p.D, t);
            }
        });
        if (AHEAD) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                px[i] = nx[i];
                pg[i] = ng[i];
                if (BWD) pd[i] = nd[i];
            }
        }
    }
    griddep_launch_dependents();
    if (!BWD || !p.partial) return;
    // dw: the block's groups in group order
    float *to = groups > 1 ? sh + group * p.D : p.partial + (size_t)blockIdx.x * p.D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float t[VEC];
        floats<VEC>(math.dw[i % (BWD ? NV : 1)], t);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const int c = column(i) + j;
            if (c >= 0 && c < p.D) to[c] = t[j];
        }
    }
    if (groups > 1) {
        __syncthreads();
        for (int c = threadIdx.x; c < p.D; c += blockDim.x) {
            float s = 0.f;
            for (int g = 0; g < groups; ++g) s += sh[g * p.D + c];
            p.partial[(size_t)blockIdx.x * p.D + c] = s;
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

// How rows are moved: by elements, in 16-byte pieces, or in 16-byte pieces that are
// aligned in memory although the rows are not (odd widths).
enum { BY_ELEMENT = 0, PIECES = 1, SHIFTED = 2 };

struct Shape {
    int vec, nv, tpr, threads, blocks, groups;
    bool shift;
};

// A row's pieces over tpr threads.  Rows of up to 32 threads x 4 pieces stay inside a
// warp (no block barrier); longer ones take a block each with up to four pieces per
// thread as far as 512 threads reach.  (With two, 7,168 BF16 channels took blocks of
// 512 threads, one per SM: 657 us instead of 505 for the gradient of 40,960 rows.)
Shape norm_shape(int D, int size, int move, long long rows, bool bwd) {
    Shape s;
    s.vec = move == BY_ELEMENT ? 1 : 16 / size;
    s.shift = move == SHIFTED;
    const int pieces = s.shift ? D / s.vec + 2 : (D + s.vec - 1) / s.vec;
    int tpr = 8;
    while (tpr < (s.vec == 1 ? 1024 : 512) && tpr * (tpr < 32 ? 1 : s.vec == 1 ? 16 : 4) < pieces)
        tpr *= 2;
    const int nv = (pieces + tpr - 1) / tpr;
    s.nv = 1;
    while (s.nv < nv) s.nv *= s.vec == 1 ? 4 : 2;
    s.tpr = tpr;
    s.threads = tpr > 32 ? tpr : 256;
    s.groups = s.threads / tpr;
    // A forward pass has a block for each of its row groups; a backward pass as many as
    // are resident, each with the same number of rows, for their dw.
    long long blocks = (rows + s.groups - 1) / s.groups;
    if (bwd) {
        const long long most = (long long)device_sms() * (2048 / s.threads);
        const long long rounds = (blocks + most - 1) / most;
        if (rounds > 1) blocks = (blocks + rounds - 1) / rounds;
    }
    if (blocks > (1 << 30)) blocks = 1 << 30;
    if (s.shift) blocks = (blocks + s.vec - 1) / s.vec * s.vec;  // whole pieces from one of a
    s.blocks = (int)blocks;                                      // thread's rows to its next
    return s;
}

template <int OP, bool BWD, typename T, int VEC, bool SHIFT>
cudaError_t launch_nv(const NormArgs &a, const Shape &s, cudaStream_t st) {
    const size_t smem = BWD && s.groups > 1 ? (size_t)s.groups * a.D * sizeof(float) : 0;
    const dim3 g(s.blocks), b(s.threads);
    if (s.nv == 1)
        return launch_dependent(norm_kernel<OP, BWD, T, VEC, 1, SHIFT>, g, b, smem, st, a);
    if (s.nv == 4)
        return launch_dependent(norm_kernel<OP, BWD, T, VEC, 4, SHIFT>, g, b, smem, st, a);
    if constexpr (VEC == 1) {
        if (s.nv == 16)
            return launch_dependent(norm_kernel<OP, BWD, T, VEC, 16, SHIFT>, g, b, smem, st, a);
    } else {
        if (s.nv == 2)
            return launch_dependent(norm_kernel<OP, BWD, T, VEC, 2, SHIFT>, g, b, smem, st, a);
        if constexpr (VEC == 4) {
            if (s.nv == 8)
                return launch_dependent(norm_kernel<OP, BWD, T, VEC, 8, SHIFT>, g, b, smem, st, a);
        }
    }
    return cudaErrorInvalidValue;
}

template <int OP, bool BWD, typename T>
cudaError_t launch_t(const NormArgs &a, const Shape &s, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    if (s.vec == 1) return launch_nv<OP, BWD, T, 1, false>(a, s, st);
    return s.shift ? launch_nv<OP, BWD, T, V, true>(a, s, st)
                   : launch_nv<OP, BWD, T, V, false>(a, s, st);
}

template <int OP, bool BWD>
cudaError_t launch_op(const NormArgs &a, int size, const Shape &s, cudaStream_t st) {
    return size == 4 ? launch_t<OP, BWD, float>(a, s, st)
                     : launch_t<OP, BWD, __nv_bfloat16>(a, s, st);
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
    kda_status_t rc = check(desc);
    if (rc != KDA_OK) return rc;
    if (desc->heads != 1 || desc->gate != KDA_GATE_NONE || desc->x_stride || desc->gate_stride ||
        !isfinite(scale))
        return KDA_ERR_INVALID_ARG;
    if (desc->tokens == 0) return KDA_OK;
    if (!h || !out || (!y != !h_out) || bad4(weight) || bad4(dev_status))
        return KDA_ERR_INVALID_ARG;
    const void *ptrs[] = {h, y, h_out, out};
    const int move = pick_move(desc, weight, ptrs, 4);
    if (move < 0) return KDA_ERR_INVALID_ARG;
    NormArgs a = make_args(desc);
    a.x = h; a.gate = y; a.w = weight; a.scale = scale; a.o1 = h_out; a.o2 = out;
    a.status = dev_status;
    return launch_norm<false>(a, OP_RESIDUAL, size_of(desc), move, (cudaStream_t)stream) ==
                   cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status_t kda_residual_norm_backward(const kda_norm_desc_t *desc, const void *d_out,
                                        const void *d_h_out, const void *h_out, const float *weight,
                                        float scale, void *dh, void *dy, float *d_weight,
                                        void *workspace, size_t workspace_bytes,
                                        int32_t *dev_status, void *stream) {
    kda_status_t rc = check(desc);
    if (rc != KDA_OK) return rc;
    if (desc->heads != 1 || desc->gate != KDA_GATE_NONE || desc->x_stride || desc->gate_stride ||
        !isfinite(scale) || bad4(weight) || bad4(d_weight) || bad4(dev_status))
        return KDA_ERR_INVALID_ARG;
    if (desc->tokens > 0 && (!d_out || !h_out || !dh)) return KDA_ERR_INVALID_ARG;
    const void *ptrs[] = {d_out, d_h_out, h_out, dh, dy};
    const int move = pick_move(desc, weight, ptrs, 5);
    if (move < 0) return KDA_ERR_INVALID_ARG;
    NormArgs a = make_args(desc);
    a.x = h_out; a.d_out = d_out; a.d_res = d_h_out; a.w = weight; a.scale = scale;
    a.o1 = dh; a.o2 = dy;
    a.status = dev_status;
    return backward(desc, a, OP_RESIDUAL, d_weight, move, workspace, workspace_bytes,
                    (cudaStream_t)stream);
}

}  // extern "C"
