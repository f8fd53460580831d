// sc_gemm.cuh -- the matrix product of the linear layer: operands, epilogue and
// launcher (sc_gemm.cu).
#pragma once

#include "sc_layers.cuh"

namespace scb {

// One operand of D(m, n) = sum_k A(m, k) B(n, k): a row-major 16-bit matrix
// whose rows start on 16-byte boundaries.  k_major: rows are m (or n), columns
// k; otherwise rows are k, columns m (or n).  fp32 operands come as three bf16
// planes (their leading, middle and last 8 bits of significand).
struct GemmOperand {
    const void *p;
    int64_t ld;            // elements between rows
    bool k_major;
    int planes;            // 1 or 3
    int64_t plane_stride;  // elements between planes
};

// out = act(D + bias) + res; pre = D + bias.  Null pointers are left out.
struct GemmEpilogue {
    const void *bias, *res;
    void *out, *pre;
    int64_t ld_out, ld_res, ld_pre;
    int bias_type, out_type, pre_type, act;
};

// Column sums left to finish: out[c] = sum_i part[i][c], i < n.
struct ColumnSums {
    const float *part;
    void *out;
    int64_t cols;
    int n, type;
};

// What the launch follows on its stream, within the same call.
enum GemmAfter {
    AFTER_ANY,    // anything: starts when all earlier work is done
    AFTER_PASS,   // a pass that makes its operands: sets itself up under it
    BESIDE_GEMM,  // another product of the same passes: runs on the SMs which that one leaves
};

// sums (nullable): finished by a warp that the product leaves idle.  wait_limit >
// 0: the self-test, whose waits for copies all expire after so many cycles.
int launch_gemm(int64_t M, int64_t N, int64_t K, int type16, const GemmOperand &a,
                const GemmOperand &b, const GemmEpilogue &epi, GemmAfter after,
                const ColumnSums *sums, int32_t *dev_status, cudaStream_t stream, int64_t wait_limit = 0);

// ---- activations ------------------------------------------------------------
// 1 / (1 + exp(-x)) times n.  The intrinsics' errors (2 ulp of the quotient, a
// few of exp where the result is far below |n|) stay under 2^-21 |n|.
__device__ __forceinline__ float times_sigmoid(float n, float x) { return __fdividef(n, 1.f + __expf(-x)); }

// sqrt(8 / pi) (z + 0.044715 z^3): gelu_tanh is z sigmoid of it
__device__ __forceinline__ float gelu_tanh_arg(float z) { return 1.59576912f * z * (1.f + 0.044715f * z * z); }

// 2^x, off by 2^-22 of itself (ex2.approx), 0 far below the normal range.
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 1 / x, off by 2^-23 of itself; 0 for an infinity.
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Phi, the normal distribution's function, and e = exp(-z^2 / 2).  The lower
// tail is a product, Phi(-x) = exp(-x^2 / 2) Q(x), and so keeps its relative
// accuracy; above 0, Phi = 1 - Phi(-z).  Q falls from 1/2 to 1 / (x sqrt(2 pi)),
// a polynomial of degree 7 in u = 1 / (1 + x / 4) over 0 <= x <= 13.3, where e
// leaves the normal range (least squares at Chebyshev nodes, weights adjusted
// towards equal ripples of 2^-20 of itself, 2^-25 in Phi).  With fp32 roundings
// Phi is off by 2.2e-7 at most and, below 0, by (z^2 + 14) 2^-24 of itself.
// Two special functions a value (16 a clock and SM) run beside the polynomial's
// packed steps.
__device__ __forceinline__ float2 normal2(float2 z, float2 &e) {
    constexpr float P[8] = {1.706042676e-04f, 9.666055441e-02f,  1.231122538e-01f, -4.171049688e-03f,
                            3.251675665e-01f, -3.054944277e-01f, 3.596809804e-01f, -9.512647241e-02f};
    const float2 a = mul2(mul2(z, z), make_float2(-0.72134752f, -0.72134752f));  // -log2(e) / 2
    e = make_float2(exp2_approx(a.x), exp2_approx(a.y));
    const float2 u = make_float2(rcp_approx(fmaf(fabsf(z.x), 0.25f, 1.f)), rcp_approx(fmaf(fabsf(z.y), 0.25f, 1.f)));
    float2 h = make_float2(P[7], P[7]);
#pragma unroll
    for (int i = 6; i >= 0; --i) h = fma2(h, u, make_float2(P[i], P[i]));
    const float2 q = mul2(e, h), r = fma2(q, make_float2(-1.f, -1.f), make_float2(1.f, 1.f));
    return make_float2(z.x < 0.f ? q.x : r.x, z.y < 0.f ? q.y : r.y);
}

// gelu(z) = z Phi(z), off by at most 6 * 2^-24 |z| and, below 0, by (z^2 + 16)
// 2^-24 of itself.
__device__ __forceinline__ float2 gelu2(float2 z) {
    float2 e;
    return mul2(z, normal2(z, e));
}

// gelu'(z) = Phi(z) + z exp(-z^2 / 2) / sqrt(2 pi); the second term is 0 from
// |z| = 16 on, which keeps infinity * 0 out.
__device__ __forceinline__ float2 gelu_grad2(float2 z) {
    float2 e;
    const float2 n = normal2(z, e);
    const float2 c = make_float2(fminf(fmaxf(z.x, -16.f), 16.f), fminf(fmaxf(z.y, -16.f), 16.f));
    return fma2(mul2(c, make_float2(0.39894228f, 0.39894228f)), e, n);
}

// Activations of one value.
template <int ACT>
__device__ __forceinline__ float act_fn(float z) {
    if constexpr (ACT == SC_ACT_RELU) return z < 0.f ? 0.f : z;  // keeps a NaN
    if constexpr (ACT == SC_ACT_GELU) return gelu2(make_float2(z, z)).x;
    if constexpr (ACT == SC_ACT_GELU_TANH) return times_sigmoid(z, gelu_tanh_arg(z));
    if constexpr (ACT == SC_ACT_SILU) return times_sigmoid(z, z);
    return z;
}

// The terms that vanish at both ends are 0 in fp32 from the bounds below on
// (q (1 - q) of gelu_tanh from |z| = 16, silu's q or 1 - q from 128), which keep
// infinity * 0 out.
template <int ACT>
__device__ __forceinline__ float act_grad(float z) {
    if constexpr (ACT == SC_ACT_RELU) return z > 0.f ? 1.f : (z == z ? 0.f : z);
    if constexpr (ACT == SC_ACT_GELU) return gelu_grad2(make_float2(z, z)).x;
    if constexpr (ACT == SC_ACT_GELU_TANH) {
        const float q = times_sigmoid(1.f, gelu_tanh_arg(z)), c = fminf(fmaxf(z, -16.f), 16.f);
        return q + c * q * (1.f - q) * 1.59576912f * (1.f + 0.134145f * c * c);
    }
    if constexpr (ACT == SC_ACT_SILU) {
        const float q = times_sigmoid(1.f, z), c = fminf(fmaxf(z, -128.f), 128.f);
        return q * (1.f + c * (1.f - q));
    }
    return 1.f;
}

// v times the activation's derivative at z, E values.
template <int ACT, int E>
__device__ __forceinline__ void times_act_grad(float (&v)[E], const float (&z)[E]) {
    if constexpr (ACT == SC_ACT_GELU && E % 2 == 0) {
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const float2 g = mul2(make_float2(v[e], v[e + 1]), gelu_grad2(make_float2(z[e], z[e + 1])));
            v[e] = g.x;
            v[e + 1] = g.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] *= act_grad<ACT>(z[e]);
    }
}

}  // namespace scb
