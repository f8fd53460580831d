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

int launch_gemm(int64_t M, int64_t N, int64_t K, int type16, const GemmOperand &a,
                const GemmOperand &b, const GemmEpilogue &epi, int32_t *dev_status,
                cudaStream_t stream);

// ---- activations ------------------------------------------------------------
// 1 / (1 + exp(-x)) times n.  The intrinsics' errors (2 ulp of the quotient, a
// few of exp where the result is far below |n|) stay under 2^-21 |n|.
__device__ __forceinline__ float times_sigmoid(float n, float x) { return __fdividef(n, 1.f + __expf(-x)); }

// sqrt(8 / pi) (z + 0.044715 z^3): gelu_tanh is z sigmoid of it
__device__ __forceinline__ float gelu_tanh_arg(float z) { return 1.59576912f * z * (1.f + 0.044715f * z * z); }

template <int ACT>
__device__ __forceinline__ float act_fn(float z) {
    if constexpr (ACT == SC_ACT_RELU) return z < 0.f ? 0.f : z;  // keeps a NaN
    if constexpr (ACT == SC_ACT_GELU) return 0.5f * z * (1.f + erff(z * 0.70710678f));
    if constexpr (ACT == SC_ACT_GELU_TANH) return times_sigmoid(z, gelu_tanh_arg(z));
    if constexpr (ACT == SC_ACT_SILU) return times_sigmoid(z, z);
    return z;
}

template <int ACT>
__device__ __forceinline__ float act_grad(float z) {
    if constexpr (ACT == SC_ACT_RELU) return z > 0.f ? 1.f : (z == z ? 0.f : z);
    if constexpr (ACT == SC_ACT_GELU)
        return 0.5f * (1.f + erff(z * 0.70710678f)) + z * 0.39894228f * __expf(-0.5f * z * z);
    if constexpr (ACT == SC_ACT_GELU_TANH) {
        const float q = times_sigmoid(1.f, gelu_tanh_arg(z));
        return q + z * q * (1.f - q) * 1.59576912f * (1.f + 0.134145f * z * z);
    }
    if constexpr (ACT == SC_ACT_SILU) {
        const float q = times_sigmoid(1.f, z);
        return q * (1.f + z * (1.f - q));
    }
    return 1.f;
}

}  // namespace scb
