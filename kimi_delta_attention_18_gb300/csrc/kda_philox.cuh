// Dropout's random words, from a counter: element (row, column) of a [rows][width] array has
// word column % 4 of Philox 4 x 32 with ten rounds (Salmon, Moraes, Dror and Shaw, "Parallel
// random numbers: as easy as 1, 2, 3", 2011) at the counter
//     (row ceil(width / 4) + column / 4) | site << 48,  offset      (two 64-bit words)
// and the key `seed`; it is kept where that word is at least `limit`.  So a pass over the
// elements in any order, and the backward pass later, finds the same mask, and none is stored.
//
// For four words a round is two 32 x 32 -> 64-bit products, each four of a scheduler's cycles,
// and two three-way exclusive ors: 10 instructions an element, and 3 to apply the mask, all
// told more than its BF16 bytes take (40,960 x 7,168 by itself 267 us, its bytes 173), about as
// long as fp32's (20,480 x 7,168 178).  The rounds' keys are in shared memory for pieces of
// eight (added up each time: 40,960 x 7,168 BF16 in the norm 603 us, 548 so; but fp32, 20,480 x
// 7,168, 364 added up and 450 from shared memory).
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

constexpr int kKeys = 20;  // of ten rounds, two each

// The keep mask of one launch.  `keys` is shared by the block: lay_keys, then a barrier.
struct Keep {
    const uint32_t *keys;
    uint32_t o0, o1, limit, site;
    int blocks;
    __device__ __forceinline__ Keep(const Drop &d, const uint32_t *keys) : keys(keys) {
        const unsigned long long offset = d.rng ? d.rng[1] : 0;
        o0 = (uint32_t)offset;
        o1 = (uint32_t)(offset >> 32);
        limit = d.limit;
        site = d.site << 16;
        blocks = d.blocks;
    }
    static __device__ __forceinline__ void lay_keys(const Drop &d, uint32_t *keys, int i) {
        if (i >= kKeys) return;
        const unsigned long long seed = d.rng[0];
        keys[i] = i & 1 ? (uint32_t)(seed >> 32) + (uint32_t)(i / 2) * 0xBB67AE85u
                        : (uint32_t)seed + (uint32_t)(i / 2) * 0x9E3779B9u;
    }
    // the words of columns 4 b .. 4 (b + N) - 1
    template <int N>
    __device__ __forceinline__ void words(long long row, int b, uint4 (&c)[N]) const {
        const unsigned long long at = (unsigned long long)row * blocks + b;
        uint4 key = *(const uint4 *)keys;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            c[i] = make_uint4((uint32_t)(at + i), (uint32_t)((at + i) >> 32) | site, o0, o1);
            round(c[i], key.x, key.y);
            round(c[i], key.z, key.w);
        }
#pragma unroll
        for (int k = 4; k < kKeys; k += 4) {
            if (N == 1)  // added up: shared by the calls for a thread's pieces
                key = make_uint4(key.x + 2 * 0x9E3779B9u, key.y + 2 * 0xBB67AE85u,
                                 key.z + 2 * 0x9E3779B9u, key.w + 2 * 0xBB67AE85u);
            else
                key = *(const uint4 *)(keys + k);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                round(c[i], key.x, key.y);
                round(c[i], key.z, key.w);
            }
        }
    }
    static __device__ __forceinline__ void round(uint4 &c, uint32_t k0, uint32_t k1) {
        const unsigned long long p = 0xD2511F53ull * c.x, q = 0xCD9E8D57ull * c.z;
        c = make_uint4((uint32_t)(q >> 32) ^ c.y ^ k0, (uint32_t)q, (uint32_t)(p >> 32) ^ c.w ^ k1,
                       (uint32_t)p);
    }
    // Bit j: column c + j is kept.  SHIFT: c is any column (outside the row: any answer),
    // else a multiple of VEC.
    template <int VEC, bool SHIFT>
    __device__ __forceinline__ uint32_t bits(long long row, int c) const {
        constexpr int N = SHIFT ? VEC / 4 + 1 : (VEC + 3) / 4;
        uint4 w[N];
        words<N>(row, SHIFT ? c >> 2 : c / 4, w);
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
            m |= (w[i].x >= limit ? 1u : 0u) << (4 * i) | (w[i].y >= limit ? 2u : 0u) << (4 * i) |
                 (w[i].z >= limit ? 4u : 0u) << (4 * i) | (w[i].w >= limit ? 8u : 0u) << (4 * i);
        return SHIFT || VEC < 4 ? m >> (c & 3) : m;
    }
    __device__ __forceinline__ uint32_t halves(uint32_t v, uint32_t lo, uint32_t hi) const {
        return v & ((lo >= limit ? 0xffffu : 0u) | (hi >= limit ? 0xffff0000u : 0u));
    }

    // The dropped of a piece's elements, the columns from c on of a row, become zeros (whatever
    // they were).
    template <bool SHIFT, typename T, int VEC>
    __device__ __forceinline__ void piece(Piece<T, VEC> &p, long long row, int c) const {
        if constexpr (!SHIFT && VEC == 8) {
            uint4 w[2];
            words<2>(row, c / 4, w);
            p.raw.x = halves(p.raw.x, w[0].x, w[0].y);
            p.raw.y = halves(p.raw.y, w[0].z, w[0].w);
            p.raw.z = halves(p.raw.z, w[1].x, w[1].y);
            p.raw.w = halves(p.raw.w, w[1].z, w[1].w);
        } else if constexpr (VEC >= 4) {
            float v[VEC];
            p.get(v);
            floats<SHIFT>(v, row, c);
            if constexpr (VEC == 4) {
                p.raw = make_float4(v[0], v[1], v[2], v[3]);
            } else {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    w[k] = __float_as_uint(v[2 * k]) >> 16 | (__float_as_uint(v[2 * k + 1]) & 0xffff0000u);
                p.raw = make_uint4(w[0], w[1], w[2], w[3]);
            }
        } else {
            const uint32_t m = bits<VEC, SHIFT>(row, c);
            if constexpr (VEC == 1) {
                if (!(m & 1)) p.raw = T(0.f);
            } else {
                if (!(m & 1)) p.raw[0] = T(0.f);
                if (!(m & 2)) p.raw[1] = T(0.f);
            }
        }
    }
    template <bool SHIFT, int VEC>
    __device__ __forceinline__ void floats(float (&v)[VEC], long long row, int c) const {
        if constexpr (!SHIFT && VEC >= 4) {
            uint4 w[VEC / 4];
            words<VEC / 4>(row, c / 4, w);
#pragma unroll
            for (int i = 0; i < VEC / 4; ++i) {
                v[4 * i] = w[i].x >= limit ? v[4 * i] : 0.f;
                v[4 * i + 1] = w[i].y >= limit ? v[4 * i + 1] : 0.f;
                v[4 * i + 2] = w[i].z >= limit ? v[4 * i + 2] : 0.f;
                v[4 * i + 3] = w[i].w >= limit ? v[4 * i + 3] : 0.f;
            }
        } else {
            const uint32_t m = bits<VEC, SHIFT>(row, c);
#pragma unroll
            for (int j = 0; j < VEC; ++j) v[j] = m >> j & 1 ? v[j] : 0.f;
        }
    }
};

}  // namespace kda
