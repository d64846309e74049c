// Rows of activations as pieces of VEC elements: one 16-byte (or, VEC = 1, one
// element) access per piece, kept packed in registers and widened to fp32 on use.
#pragma once

#include "kda_internal.cuh"

namespace kda {

template <typename T, int VEC>
struct Piece;

template <>
struct Piece<float, 4> {
    float4 raw;
    __device__ __forceinline__ void load(const float *p) { raw = *(const float4 *)p; }
    __device__ __forceinline__ void zero() { raw = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float (&v)[4]) const {
        v[0] = raw.x; v[1] = raw.y; v[2] = raw.z; v[3] = raw.w;
    }
    static __device__ __forceinline__ void store(float *p, const float (&v)[4]) {
        *(float4 *)p = make_float4(v[0], v[1], v[2], v[3]);
    }
};

template <>
struct Piece<__nv_bfloat16, 8> {
    uint4 raw;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { raw = *(const uint4 *)p; }
    __device__ __forceinline__ void zero() { raw = make_uint4(0u, 0u, 0u, 0u); }
    // bf16 is the upper half of an fp32: widening is a shift or a mask
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&v)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *(const uint32_t *)&b;
        }
        *(uint4 *)p = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

template <typename T>
struct Piece<T, 1> {
    T raw;
    __device__ __forceinline__ void load(const T *p) { raw = *p; }
    __device__ __forceinline__ void zero() { raw = T(0.f); }
    __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = (float)raw; }
    static __device__ __forceinline__ void store(T *p, const float (&v)[1]) { act_st(p, 0, v[0]); }
};

template <typename T>
constexpr int kFullVec = 16 / (int)sizeof(T);

}  // namespace kda
