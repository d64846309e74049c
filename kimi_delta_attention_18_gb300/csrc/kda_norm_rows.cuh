// The norms with rows loaded straight into registers: the kernel and its launch.  Every
// instantiation belongs to the file that launches it (kda_norm.cu, and kda_norm_drop.cu with
// dropout).
#pragma once

#include "kda_norm_math.cuh"
#include "kda_sm100.cuh"

namespace kda {

struct Shape {
    int vec, nv, tpr, threads, blocks, groups;
    bool shift;
};
cudaError_t launch_norm_drop(const NormArgs &a, bool bwd, int size, const Shape &s, cudaStream_t st);

namespace {

using sm100::griddep_launch_dependents;
using sm100::griddep_wait;

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
    RowMath<is_residual(OP) ? OP_RESIDUAL : OP, BWD, T, VEC, NV> math;
    griddep_wait();
    math.begin(load_w);
    __shared__ __align__(16) uint32_t keys[OP == OP_DROP ? kKeys : 4];
    if constexpr (OP == OP_DROP) {
        Keep::lay_keys(p.drop, keys, threadIdx.x);
        __syncthreads();
    }
    const Keep keep(OP == OP_DROP ? p.drop : Drop{}, keys);

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
        if (is_residual(OP)) gr = BWD ? d_res + base : gr;
        const bool has_g = OP == OP_SIGMOID || OP == OP_SILU ||
                           (is_residual(OP) && (BWD ? d_res != nullptr : gate != nullptr));
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
        if constexpr (OP == OP_DROP && !BWD) {
#pragma unroll
            for (int i = 0; i < NV; ++i) keep.template piece<SHIFT>(pg[i], row, column(i));
        }
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
            if ((BWD || is_residual(OP)) && o2) {
                floats<VEC>(a2, t);
                if constexpr (OP == OP_DROP && BWD)
                    keep.template floats<SHIFT>(t, row, column(i));
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

// How rows are moved: by elements, in 16-byte pieces, or in 16-byte pieces that are
// aligned in memory although the rows are not (odd widths).
enum { BY_ELEMENT = 0, PIECES = 1, SHIFTED = 2 };

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

}  // namespace
}  // namespace kda
