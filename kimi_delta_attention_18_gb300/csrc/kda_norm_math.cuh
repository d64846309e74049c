// The arithmetic of the norms around a mixer on one thread's pieces of a row; the
// kernels that move the rows are in kda_norm.cu (rows loaded into registers) and
// kda_norm_ring.cu (rows streamed through shared memory).
//
// Every element is read once and written once, so these passes should be bound by
// their bytes; about 50 instructions per element (the gated gradient written out in
// scalars) were enough to keep it at 5.4 TB/s.  So fp32 arithmetic goes in pairs
// (fma.rn.f32x2 and its like: the results of two scalar operations), and what the
// pass over the sums has computed is kept for the outputs.
#pragma once

#include "kda_internal.cuh"
#include "kda_vec.cuh"

namespace kda {

struct NormArgs {
    const void *x, *gate, *d_out, *d_res;  // residual: x = h (forward) or h' (backward)
    const float *w;                        // NULL: ones
    void *o1, *o2;      // gated: y | dx, dz      residual: h', n | dh, dy
    float *partial;     // backward: [blocks][D]
    int32_t *status;
    long long rows;
    long long x_stride, gate_stride;  // elements between tokens
    int heads, D, tpr, strided;
    float eps, scale, inv_d;
};

enum { OP_NORM = 0, OP_SIGMOID = 1, OP_SILU = 2, OP_RESIDUAL = 3 };  // the first three: kda_gate_t

// Rows streamed through shared memory (from 16-byte bases, enough of them; whole 16-byte
// pieces, at most 8,192 channels, and with a gate in BF16 tokens apart too; or `pairs`:
// contiguous, any width up to 512 forward, 1,024 (BF16) or 2,048 (fp32) backward): its
// number of blocks, 0 where it does not apply, and the launch.
int norm_ring_blocks(const NormArgs &a, int op, bool bwd, int size, bool pairs);
cudaError_t launch_norm_ring(const NormArgs &a, int op, bool bwd, int size, bool pairs,
                             cudaStream_t st);

typedef unsigned long long f2;  // two fp32 values

__device__ __forceinline__ f2 pk(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 un(f2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 both(float a) { return pk(a, a); }

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// 1 / (1 + 2^(-z log2 e)); an overflow to infinity gives 0.
__device__ __forceinline__ f2 sigmoid2(f2 z) {
    const float2 t = un(mul2(z, both(-1.4426950408889634f)));
    const float2 u = un(add2(pk(ex2(t.x), ex2(t.y)), both(1.f)));
    return pk(rcp(u.x), rcp(u.y));
}

template <int VEC>
constexpr int kPairs = (VEC + 1) / 2;

template <typename T, int VEC>
__device__ __forceinline__ void get2(const Piece<T, VEC> &p, f2 (&v)[kPairs<VEC>]) {
    float t[VEC];
    p.get(t);
#pragma unroll
    for (int j = 0; j < kPairs<VEC>; ++j) v[j] = pk(t[2 * j], VEC == 1 ? 0.f : t[(2 * j + 1) % VEC]);
}
template <int VEC>
__device__ __forceinline__ void floats(const f2 (&v)[kPairs<VEC>], float (&t)[VEC]) {
#pragma unroll
    for (int j = 0; j < kPairs<VEC>; ++j) {
        const float2 u = un(v[j]);
        t[2 * j] = u.x;
        if (VEC > 1) t[(2 * j + 1) % VEC] = u.y;
    }
}

// One thread's part of its rows: NV pieces of VEC elements, always the same columns.
// With up to 16 elements (KEEP) it holds their weights and, unless another row's sums
// come before this one's outputs (HOLD false), what the sums' pass computed (the
// gate's sigmoid s, q = d s); otherwise load_w(i, w) is asked again and the gate
// computed again.
template <int OP, bool BWD, typename T, int VEC, int NV, bool HOLD = true>
struct RowMath {
    static constexpr int VP = kPairs<VEC>;
    static constexpr bool KEEP = NV * VEC <= 16, GATED = OP == OP_SIGMOID || OP == OP_SILU;
    static constexpr bool KEEPS = KEEP && HOLD;
    static constexpr int KW = KEEP ? NV : 1, KS = KEEPS && BWD && GATED ? NV : 1;
    using P = Piece<T, VEC>;
    f2 dw[BWD ? NV : 1][VP];
    f2 wk[KW][VP], sk[KS][VP], qk[KS][VP];

    template <typename W>
    __device__ __forceinline__ void begin(W &&load_w) {
        if (BWD) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < VP; ++j) dw[i][j] = 0;
        }
        if (KEEP) {
#pragma unroll
            for (int i = 0; i < NV; ++i) load_w(i, wk[i % KW]);
        }
    }

    // ss: this thread's part of mean(v^2) (the mean, not the sum: D x more range);
    // se: of the sum of e v, e = d a w.
    template <typename W>
    __device__ __forceinline__ void sums(const NormArgs &p, const P (&px)[NV], const P (&pg)[NV],
                                         const P (&pd)[NV], W &&load_w, float &ss, float &se) {
        f2 a2[2] = {0, 0}, b2[2] = {0, 0};
        const f2 inv = both(p.inv_d), scale = both(p.scale);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            f2 v[VP], g[VP], d[VP], w[VP];
            get2<T, VEC>(px[i], v);
            if (GATED ? BWD : OP == OP_RESIDUAL && !BWD) get2<T, VEC>(pg[i], g);
            if (BWD) {
                get2<T, VEC>(pd[i], d);
                if (KEEP) {
#pragma unroll
                    for (int j = 0; j < VP; ++j) w[j] = wk[i % KW][j];
                } else {
                    load_w(i, w);
                }
            }
#pragma unroll
            for (int j = 0; j < VP; ++j) {
                if (OP == OP_RESIDUAL && !BWD) v[j] = fma2(scale, g[j], v[j]);
                a2[j & 1] = fma2(mul2(v[j], inv), v[j], a2[j & 1]);
                if (BWD) {
                    f2 e = d[j];
                    if (GATED) {
                        const f2 s = sigmoid2(g[j]), q = mul2(e, s);
                        if (KEEPS) {
                            sk[i % KS][j] = s;
                            qk[i % KS][j] = q;
                        }
                        e = OP == OP_SILU ? mul2(q, g[j]) : q;
                    }
                    b2[j & 1] = fma2(mul2(e, w[j]), v[j], b2[j & 1]);
                }
            }
        }
        const float2 a = un(add2(a2[0], a2[1])), b = un(add2(b2[0], b2[1]));
        ss = a.x + a.y;
        se = b.x + b.y;
    }

    // From the row's sums: store(i, first, second) for every piece.
    template <typename W, typename S>
    __device__ __forceinline__ void outputs(const NormArgs &p, const P (&px)[NV], const P (&pg)[NV],
                                            const P (&pd)[NV], W &&load_w, float ss, float se,
                                            S &&store) {
        const float r = rsqrtf(ss + p.eps);
        const f2 rs = both(r), scale = both(p.scale);
        const f2 rk = both(-r * ((se * r) * p.inv_d * r));  // r n mean(e n) = -rk x
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            f2 v[VP], g[VP], d[VP], w[VP], o1[VP], o2[VP];
            get2<T, VEC>(px[i], v);
            if (GATED || OP == OP_RESIDUAL) get2<T, VEC>(pg[i], g);
            if (BWD) get2<T, VEC>(pd[i], d);
            if (KEEP) {
#pragma unroll
                for (int j = 0; j < VP; ++j) w[j] = wk[i % KW][j];
            } else {
                load_w(i, w);
            }
#pragma unroll
            for (int j = 0; j < VP; ++j) {
                o2[j] = 0;
                if (OP == OP_RESIDUAL && !BWD) {
                    o1[j] = fma2(scale, g[j], v[j]);
                    o2[j] = mul2(mul2(o1[j], rs), w[j]);
                } else if (!BWD) {
                    o1[j] = mul2(mul2(v[j], rs), w[j]);
                    if (GATED) {
                        const f2 s = sigmoid2(g[j]);
                        o1[j] = mul2(o1[j], OP == OP_SILU ? mul2(s, g[j]) : s);
                    }
                } else {
                    const f2 n = mul2(v[j], rs);
                    f2 e = d[j];
                    if (GATED) {
                        const f2 s = KEEPS ? sk[i % KS][j] : sigmoid2(g[j]);
                        const f2 q = KEEPS ? qk[i % KS][j] : mul2(d[j], s);
                        e = OP == OP_SILU ? mul2(q, g[j]) : q;
                        // a' = s (1 - s), or s + z s (1 - s): d a' = e (1 - s) (+ q)
                        f2 t = fma2(mul2(e, both(-1.f)), s, e);
                        if (OP == OP_SILU) t = add2(t, q);
                        o2[j] = mul2(mul2(n, w[j]), t);
                    }
                    dw[i][j] = fma2(e, n, dw[i][j]);
                    const f2 ew = mul2(e, w[j]);
                    if (OP == OP_RESIDUAL) {
                        o1[j] = fma2(rk, v[j], fma2(ew, rs, g[j]));
                        o2[j] = mul2(scale, o1[j]);
                    } else {
                        o1[j] = fma2(rk, v[j], mul2(ew, rs));
                    }
                }
            }
            store(i, o1, o2);
        }
    }
};

}  // namespace kda
