// sc_layers.cuh -- element types and small device helpers shared by the
// floating-point layers (sc_norm.cu, sc_linear.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "sc_internal.cuh"

namespace scb {

inline bool type_ok(int t) { return t == SC_F32 || t == SC_BF16 || t == SC_F16; }
inline int type_size(int t) { return t == SC_F32 ? 4 : 2; }
inline int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }
inline int64_t div_up(int64_t v, int64_t by) { return (v + by - 1) / by; }
inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }

// Two 16-bit values in one word.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <typename T>
__device__ __forceinline__ void unpack2(uint32_t w, float &a, float &b);
template <>
__device__ __forceinline__ void unpack2<__nv_bfloat16>(uint32_t w, float &a, float &b) {
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xFFFF0000u);
}
template <>
__device__ __forceinline__ void unpack2<__half>(uint32_t w, float &a, float &b) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    a = f.x;
    b = f.y;
}

// E contiguous elements to and from fp32 registers.  E * sizeof(T) is 16 or 32
// bytes on a 16-byte boundary, 8 or 4 bytes on such a boundary, or one element.
template <typename T, int E>
__device__ __forceinline__ void load_vec(const T *p, float (&v)[E]) {
    constexpr int B = E * (int)sizeof(T);
    if constexpr (E == 1) {
        v[0] = to_f(*p);
    } else {
        static_assert(B == 4 || B == 8 || B % 16 == 0, "vector width");
        constexpr int W = B < 16 ? B / 4 : 4;  // 32-bit words per load
        uint32_t raw[B / 4];
#pragma unroll
        for (int i = 0; i < B / 4 / W; ++i) {
            if constexpr (W == 4) {
                const uint4 q = reinterpret_cast<const uint4 *>(p)[i];
                raw[4 * i] = q.x;
                raw[4 * i + 1] = q.y;
                raw[4 * i + 2] = q.z;
                raw[4 * i + 3] = q.w;
            } else if constexpr (W == 2) {
                const uint2 q = reinterpret_cast<const uint2 *>(p)[i];
                raw[2 * i] = q.x;
                raw[2 * i + 1] = q.y;
            } else {
                raw[i] = reinterpret_cast<const uint32_t *>(p)[i];
            }
        }
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < E; ++i) v[i] = __uint_as_float(raw[i]);
        } else {
#pragma unroll
            for (int i = 0; i < E; i += 2) unpack2<T>(raw[i / 2], v[i], v[i + 1]);
        }
    }
}

template <typename T, int E>
__device__ __forceinline__ void store_vec(T *p, const float (&v)[E]) {
    constexpr int B = E * (int)sizeof(T);
    if constexpr (E == 1) {
        *p = from_f<T>(v[0]);
    } else {
        static_assert(B == 4 || B == 8 || B % 16 == 0, "vector width");
        constexpr int W = B < 16 ? B / 4 : 4;
        uint32_t e[B / 4];
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < E; ++i) e[i] = __float_as_uint(v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < E; i += 2) e[i / 2] = pack2<T>(v[i], v[i + 1]);
        }
#pragma unroll
        for (int i = 0; i < B / 4 / W; ++i) {
            if constexpr (W == 4)
                reinterpret_cast<uint4 *>(p)[i] = make_uint4(e[4 * i], e[4 * i + 1], e[4 * i + 2], e[4 * i + 3]);
            else if constexpr (W == 2)
                reinterpret_cast<uint2 *>(p)[i] = make_uint2(e[2 * i], e[2 * i + 1]);
            else
                reinterpret_cast<uint32_t *>(p)[i] = e[i];
        }
    }
}

// The same with the element type known at run time (uniform over the block):
// parameters, which are read far less often than activations.
template <int E>
__device__ __forceinline__ void load_any(const void *p, int type, int64_t i, float (&v)[E]) {
    if (type == SC_F32) load_vec<float, E>(static_cast<const float *>(p) + i, v);
    else if (type == SC_BF16) load_vec<__nv_bfloat16, E>(static_cast<const __nv_bfloat16 *>(p) + i, v);
    else load_vec<__half, E>(static_cast<const __half *>(p) + i, v);
}
__device__ __forceinline__ void store_any(void *p, int type, int64_t i, float v) {
    if (type == SC_F32) static_cast<float *>(p)[i] = v;
    else if (type == SC_BF16) static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
    else static_cast<__half *>(p)[i] = __float2half_rn(v);
}

// Two values at a time (one packed fp32 instruction for both).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Column sums from per-block partial sums (sc_norm.cu): out_k[c] = sum_p
// part[p][k][c], k < n_out, c < cols, in ascending p.  A null out_k is skipped.
int launch_finish_columns(const float *part, int n_part, int n_out, int64_t cols, void *out0,
                          void *out1, int out_type, cudaStream_t stream);

}  // namespace scb
