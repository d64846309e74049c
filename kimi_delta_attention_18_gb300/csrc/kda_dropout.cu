// Dropout by itself: out = x / (1 - p) where the element is kept, else 0, over [T][D].  The
// gradient is the same operation on the output's adjoint.  A thread takes the columns of one
// or two of the generator's blocks of four words, so none is computed twice; kda_philox.cuh
// has the generator and what it costs.
#include <math.h>

#include "kda_philox.cuh"
#include "kda_sm100.cuh"

namespace kda {
namespace {

using sm100::griddep_launch_dependents;
using sm100::griddep_wait;

// VEC columns (a 16-byte piece), or, VEC = 1, four columns element by element.
template <typename T, int VEC>
__global__ void __launch_bounds__(256)
    dropout_kernel(const T *x, T *out, long long rows, int D, const __grid_constant__ Drop drop,
                   float kept) {
    constexpr int COLS = VEC == 1 ? 4 : VEC;
    griddep_wait();
    griddep_launch_dependents();
    __shared__ __align__(16) uint32_t keys[kKeys];
    Keep::lay_keys(drop, keys, threadIdx.x);
    __syncthreads();
    const Keep keep(drop, keys);
    const int per_row = (D + COLS - 1) / COLS;
    const long long total = rows * per_row, step = gridDim.x * 256ll;
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += step) {
        const long long row = total <= 0xffffffffll ? (uint32_t)i / (uint32_t)per_row : i / per_row;
        const int c = (int)(i - row * per_row) * COLS;
        const long long at = row * D + c;
        float v[COLS];
        if constexpr (VEC > 1) {
            Piece<T, VEC> p;
            p.load(x + at);
            p.get(v);
        } else {
#pragma unroll
            for (int j = 0; j < COLS; ++j) v[j] = c + j < D ? act_ld(x, (size_t)(at + j)) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < COLS; ++j) v[j] *= kept;
        keep.template floats<false>(v, row, c);
        if constexpr (VEC > 1) {
            Piece<T, VEC>::store(out + at, v);
        } else {
#pragma unroll
            for (int j = 0; j < COLS; ++j)
                if (c + j < D) act_st(out, (size_t)(at + j), v[j]);
        }
    }
}

template <typename T>
cudaError_t launch(const void *x, void *out, long long rows, int D, const Drop &d, float kept,
                   cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    const bool vec = D % V == 0 && ((uintptr_t)x & 15u) == 0 && ((uintptr_t)out & 15u) == 0;
    const long long need = (rows * ((D + (vec ? V : 4) - 1) / (vec ? V : 4)) + 255) / 256;
    const long long most = 32ll * device_sms();
    const dim3 grid((unsigned)(need < most ? need : most));
    return vec ? launch_dependent(dropout_kernel<T, V>, grid, dim3(256), 0, st, (const T *)x,
                                  (T *)out, rows, D, d, kept)
               : launch_dependent(dropout_kernel<T, 1>, grid, dim3(256), 0, st, (const T *)x,
                                  (T *)out, rows, D, d, kept);
}

}  // namespace

kda_status_t dropout_args(const kda_dropout_t *d, int width, Drop *to, float *kept) {
    if (!d->rng || ((uintptr_t)d->rng & 7u)) return KDA_ERR_INVALID_ARG;
    if (!(d->p >= 0. && d->p < 1.) || d->site < 0 || d->site > 0xffff) return KDA_ERR_INVALID_ARG;
    const double limit = rint(d->p * 4294967296.);
    if (limit > 4294967295.) return KDA_ERR_INVALID_ARG;  // nothing would be kept
    to->rng = (const long long *)d->rng;
    to->limit = (unsigned)limit;
    to->site = (unsigned)d->site;
    to->blocks = (width + 3) / 4;
    *kept = (float)(1. / (1. - limit / 4294967296.));
    return KDA_OK;
}

}  // namespace kda

using namespace kda;

extern "C" kda_status_t kda_dropout(const kda_dropout_t *dropout, int64_t tokens, int32_t width,
                                    int32_t act_dtype, const void *x, void *out, void *stream) {
    if (!dropout || tokens < 0 || width < 1) return KDA_ERR_INVALID_ARG;
    if (act_dtype != KDA_DTYPE_F32 && act_dtype != KDA_DTYPE_BF16) return KDA_ERR_UNSUPPORTED;
    if (width > (1 << 30) || tokens > (1ll << 42) / width) return KDA_ERR_UNSUPPORTED;
    Drop d;
    float kept;
    const kda_status_t rc = dropout_args(dropout, width, &d, &kept);
    if (rc != KDA_OK) return rc;
    if (tokens == 0) return KDA_OK;
    const int size = act_dtype == KDA_DTYPE_BF16 ? 2 : 4;
    if (!x || !out || (uintptr_t)x % size || (uintptr_t)out % size) return KDA_ERR_INVALID_ARG;
    const cudaError_t e =
        size == 2 ? launch<__nv_bfloat16>(x, out, tokens, width, d, kept, (cudaStream_t)stream)
                  : launch<float>(x, out, tokens, width, d, kept, (cudaStream_t)stream);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
