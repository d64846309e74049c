// Dropout's random words, from a counter: element (row, column) of a [rows][width] array has
// word column % 4 of Philox 4 x 32 with ten rounds (Salmon, Moraes, Dror and Shaw, "Parallel
// random numbers: as easy as 1, 2, 3", 2011) at the counter
//     (row ceil(width / 4) + column / 4) | site << 48,  offset      (two 64-bit words)
// and the key `seed`; it is kept where that word is at least `limit`.  So a pass over the
// elements in any order, and the backward pass later, finds the same mask, and none is stored.
//
// A round is two 32 x 32 -> 64-bit products and two three-way exclusive ors for four words:
// about 13 instructions an element, a third of what an SM issues in the time that its share
// of a BF16 element's bytes takes.
#pragma once

#include "kda_internal.cuh"
#include "kda_vec.cuh"

namespace kda {

struct Drop {
    const long long *rng;  // seed, offset (device memory: a captured graph reads it anew)
    unsigned limit;        // p 2^32
    unsigned site;
    int blocks;            // ceil(width / 4)
};

// Checks a caller's description; `kept` is 1 / (1 - p), p as the limit has it.
kda_status_t dropout_args(const kda_dropout_t *d, int width, Drop *to, float *kept);

__device__ __forceinline__ uint4 philox(uint4 c, uint32_t k0, uint32_t k1) {
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const unsigned long long p = 0xD2511F53ull * c.x, q = 0xCD9E8D57ull * c.z;
        c = make_uint4((uint32_t)(q >> 32) ^ c.y ^ k0, (uint32_t)q,
                       (uint32_t)(p >> 32) ^ c.w ^ k1, (uint32_t)p);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return c;
}

// The keep mask of one launch.
struct Keep {
    uint32_t k0, k1, o0, o1, limit, site;
    int blocks;
    __device__ __forceinline__ explicit Keep(const Drop &d) {
        const unsigned long long seed = d.rng ? d.rng[0] : 0, offset = d.rng ? d.rng[1] : 0;
        k0 = (uint32_t)seed;
        k1 = (uint32_t)(seed >> 32);
        o0 = (uint32_t)offset;
        o1 = (uint32_t)(offset >> 32);
        limit = d.limit;
        site = d.site << 16;
        blocks = d.blocks;
    }
    // the words of columns 4 b .. 4 b + 3
    __device__ __forceinline__ uint4 words(long long row, int b) const {
        const unsigned long long at = (unsigned long long)row * blocks + b;
        return philox(make_uint4((uint32_t)at, (uint32_t)(at >> 32) | site, o0, o1), k0, k1);
    }
    // Bit j: column c + j is kept.  SHIFT: c is any column (outside the row: any answer),
    // else a multiple of VEC.
    template <int VEC, bool SHIFT>
    __device__ __forceinline__ uint32_t bits(long long row, int c) const {
        constexpr int N = SHIFT ? VEC / 4 + 1 : (VEC + 3) / 4;
        const int first = SHIFT ? c >> 2 : c / 4;
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint4 w = words(row, first + i);
            m |= (w.x >= limit ? 1u : 0u) << (4 * i) | (w.y >= limit ? 2u : 0u) << (4 * i) |
                 (w.z >= limit ? 4u : 0u) << (4 * i) | (w.w >= limit ? 8u : 0u) << (4 * i);
        }
        return SHIFT ? m >> (c & 3) : VEC < 4 ? m >> (c & 3) : m;
    }
};

// A piece's dropped elements become zeros (whatever they were).
__device__ __forceinline__ void keep_piece(Piece<float, 4> &p, uint32_t m) {
    p.raw.x = m & 1 ? p.raw.x : 0.f;
    p.raw.y = m & 2 ? p.raw.y : 0.f;
    p.raw.z = m & 4 ? p.raw.z : 0.f;
    p.raw.w = m & 8 ? p.raw.w : 0.f;
}
__device__ __forceinline__ uint32_t keep_halves(uint32_t w, uint32_t m, int j) {
    return w & ((m >> j & 1 ? 0xffffu : 0u) | (m >> j & 2 ? 0xffff0000u : 0u));
}
__device__ __forceinline__ void keep_piece(Piece<__nv_bfloat16, 8> &p, uint32_t m) {
    p.raw.x = keep_halves(p.raw.x, m, 0);
    p.raw.y = keep_halves(p.raw.y, m, 2);
    p.raw.z = keep_halves(p.raw.z, m, 4);
    p.raw.w = keep_halves(p.raw.w, m, 6);
}
template <typename T>
__device__ __forceinline__ void keep_piece(Piece<T, 2> &p, uint32_t m) {
    if (!(m & 1)) p.raw[0] = T(0.f);
    if (!(m & 2)) p.raw[1] = T(0.f);
}
template <typename T>
__device__ __forceinline__ void keep_piece(Piece<T, 1> &p, uint32_t m) {
    if (!(m & 1)) p.raw = T(0.f);
}
template <int VEC>
__device__ __forceinline__ void keep_floats(float (&v)[VEC], uint32_t m) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = m >> j & 1 ? v[j] : 0.f;
}

}  // namespace kda
