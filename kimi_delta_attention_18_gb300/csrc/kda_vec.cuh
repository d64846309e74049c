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
    __device__ __forceinline__ void set(int j, float x) {
        if (j == 0) raw.x = x;
        if (j == 1) raw.y = x;
        if (j == 2) raw.z = x;
        if (j == 3) raw.w = x;
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
    __device__ __forceinline__ void set(int j, __nv_bfloat16 x) {
        const uint32_t b = (uint32_t)__bfloat16_as_ushort(x) << (16 * (j & 1));
        if (j / 2 == 0) raw.x |= b;  // after zero()
        if (j / 2 == 1) raw.y |= b;
        if (j / 2 == 2) raw.z |= b;
        if (j / 2 == 3) raw.w |= b;
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

// Two elements of a row that starts anywhere; the second may be past its end.
template <typename T>
struct Piece<T, 2> {
    T raw[2];
    __device__ __forceinline__ void load(const T *p, bool second) {
        raw[0] = p[0];
        raw[1] = second ? p[1] : T(0.f);
    }
    __device__ __forceinline__ void zero() { raw[0] = raw[1] = T(0.f); }
    __device__ __forceinline__ void get(float (&v)[2]) const {
        v[0] = (float)raw[0];
        v[1] = (float)raw[1];
    }
    static __device__ __forceinline__ void store(T *p, const float (&v)[2], bool second) {
        act_st(p, 0, v[0]);
        if (second) act_st(p, 1, v[1]);
    }
};

template <typename T>
struct Piece<T, 1> {
    T raw;
    __device__ __forceinline__ void load(const T *p) { raw = *p; }
    __device__ __forceinline__ void zero() { raw = T(0.f); }
    __device__ __forceinline__ void set(int, T x) { raw = x; }
    __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = (float)raw; }
    static __device__ __forceinline__ void store(T *p, const float (&v)[1]) { act_st(p, 0, v[0]); }
};

// Columns [c, c + VEC) of a row of D: without SHIFT c is a multiple of VEC and a piece
// is in the row or past it; with it rows start anywhere, pieces are aligned in memory
// (c may be negative) and those at the row's two ends are moved element by element
// (loading them whole and cutting them was 5 % slower).
template <bool SHIFT, typename T, int VEC>
__device__ __forceinline__ void load_piece(Piece<T, VEC> &p, const T *row, int c, int D) {
    if (!SHIFT) {
        if (c < D) p.load(row + c);
        else p.zero();
    } else if (c >= 0 && c + VEC <= D) {
        p.load(row + c);
    } else {
        p.zero();
#pragma unroll
        for (int j = 0; j < VEC; ++j)
            if (c + j >= 0 && c + j < D) p.set(j, row[c + j]);
    }
}
template <bool SHIFT, typename T, int VEC>
__device__ __forceinline__ void store_piece(T *row, int c, int D, const float (&v)[VEC]) {
    if (!SHIFT) {
        if (c < D) Piece<T, VEC>::store(row + c, v);
    } else if (c >= 0 && c + VEC <= D) {
        Piece<T, VEC>::store(row + c, v);
    } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
            if (c + j >= 0 && c + j < D) act_st(row, c + j, v[j]);
    }
}

}  // namespace kda
