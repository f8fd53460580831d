// sc_norm.cu -- layer norm and its backward pass.
//
// Forward, per row of D values:   mu = sum x / D,  v = sum (x - mu)^2 / D,
// r = 1 / sqrt(v + eps),  y = (x - mu) r w + b.
// The mean m of fp32 values is off by the roundings of their sum, |mu - m| up to
// 2^-20 |mu|, which is more than r bears where a row varies little about a large
// mean.  With c = x - m (exact there) and t = sum c / D the rest of the mean, v =
// sum c^2 / D - t^2 and y = (c - t) r w + b: one more sum beside that of the
// squares (65792 x 1024 fp32 -> bf16 65.0 -> 66.8 us).  16-bit values that lie
// close together add up exactly in 24 bits, so their mean needs no rest.
// Backward, with h = (x - mu) r, g = dy w, s1 = sum_j g, s2 = sum_j g h:
//   dx = r (g - (s1 + h s2) / D) [+ dx_add],
//   dw_j = sum_i dy_ij h_ij,  db_j = sum_i dy_ij.
// Both are bound by device memory: a row is read once and held in registers.
// Of the copy's 6.45 TB/s: 65792 x 1024 fp32 -> bf16 67 us (93 %), the same
// bf16 -> bf16 55 us (76 %: weight and bias, read per row from L1, are twice its
// bytes); backward of 32896 x 1024 fp32 72 us (87 %).  Small calls are launches:
// 257 x 1024 3.0 us.
#include <initializer_list>
#include <type_traits>

#include "sc_layers.cuh"

namespace scb {
namespace {

// Most blocks (one per SM) that hold column sums in the backward pass, a
// partial row of dweight and dbias each; even, see Pairs.
int bwd_blocks() { return sm_count() + (sm_count() & 1); }

struct NormArgs {
    int64_t rows, cols;
    int64_t ld_x, ld_y, ld_dx, ld_add;
    float eps;
    int w_type;
    const void *x, *w, *b, *add;
    const void *dy;
    void *y;          // forward: y, backward: dx (nullable)
    float *mean, *rstd;
    float *part;      // backward: [gridDim][2][cols] column sums of dy h and dy, or null
};

// Sum over the T threads that share a row (T = 32: one warp; else the whole
// block, T = blockDim.x).  `red` holds one float per warp; two consecutive
// calls must use different buffers (one barrier per call).
template <int T>
__device__ __forceinline__ float row_sum(float v, float *red) {
    v = warp_sum(v);
    if constexpr (T > 32) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int i = 1; i < T / 32; ++i) v += red[i];
    }
    return v;
}

// Two sums at once (BOTH; else of b alone); `red` holds one float2 per warp.
template <int T, bool BOTH>
__device__ __forceinline__ float2 row_sum2(float a, float b, float2 *red) {
    float2 v = make_float2(BOTH ? warp_sum(a) : 0.f, warp_sum(b));
    if constexpr (T > 32) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int i = 1; i < T / 32; ++i) {
            if (BOTH) v.x += red[i].x;
            v.y += red[i].y;
        }
    }
    return v;
}

// s / D from inv = 1 / D with one step of correction, so that a constant row gives
// its value (4099 x 997 takes a third longer with divisions instead).
__device__ __forceinline__ float divided(float s, float D, float inv) {
    const float q = s * inv;
    return isinf(q) ? q : fmaf(fmaf(-q, D, s), inv, q);
}

// The rest t of a row's mean and r, from the sums of c and c^2 (c = x - m).
struct Spread {
    float rest, rstd;
    // an infinite m stays what it is
    __device__ __forceinline__ float mean(float m) const { return isinf(m) ? m : m + rest; }
};
template <bool REST>
__device__ __forceinline__ Spread spread(float s1, float s2, float D, float inv, float eps) {
    const float t = REST ? divided(s1, D, inv) : 0.f;
    if (REST) {
        s2 = fmaf(-s1, t, s2);
        if (s2 < 0.f) s2 = 0.f;  // keeps a NaN
    }
    return {t, 1.f / sqrtf(s2 * inv + eps)};
}

// T threads per row, each holding NC chunks of E columns (chunk c of thread t
// starts at column (c T + t) E), so D <= T NC E; rows and D are aligned for E,
// which is even: the arithmetic runs on two values at a time.
template <typename TX, typename TY, int E, int NC, int T>
__global__ void __launch_bounds__(T < 128 ? 128 : T) ln_fwd_kernel(const NormArgs p) {
    constexpr bool REST = sizeof(TX) == 4;
    constexpr int RPB = T < 128 ? 128 / T : 1;
    __shared__ float red[T / 32];
    __shared__ float2 red2[T / 32];
    const int t = threadIdx.x % T;
    const int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / T;
    if (row >= p.rows) return;  // whole warps (T = 32) only
    const TX *x = static_cast<const TX *>(p.x) + row * p.ld_x;
    float v[NC][E];
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int64_t col = (int64_t)(c * T + t) * E;
        if (col < p.cols) {
            load_vec<TX, E>(x + col, v[c]);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) v[c][e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < E; e += 2) s = add2(s, make_float2(v[c][e], v[c][e + 1]));
    }
    const float inv = 1.f / (float)p.cols;
    const float mu = divided(row_sum<T>(s.x + s.y, red), (float)p.cols, inv);
    const float2 m2 = make_float2(-mu, -mu);
    float2 s2 = s = make_float2(0.f, 0.f);
#pragma unroll
    for (int c = 0; c < NC; ++c)
        if ((int64_t)(c * T + t) * E < p.cols)
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float2 d = add2(make_float2(v[c][e], v[c][e + 1]), m2);
                if (REST) s = add2(s, d);
                s2 = fma2(d, d, s2);
                v[c][e] = d.x;
                v[c][e + 1] = d.y;
            }
    const float2 sums = row_sum2<T, REST>(s.x + s.y, s2.x + s2.y, red2);
    const Spread q = spread<REST>(sums.x, sums.y, (float)p.cols, inv, p.eps);
    const float r = q.rstd;
    if (t == 0) {
        if (p.mean) p.mean[row] = q.mean(mu);
        if (p.rstd) p.rstd[row] = r;
    }
    TY *y = static_cast<TY *>(p.y) + row * p.ld_y;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int64_t col = (int64_t)(c * T + t) * E;
        if (col >= p.cols) continue;
        float w[E], b[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            w[e] = 1.f;
            b[e] = 0.f;
        }
        if (p.w) load_any<E>(p.w, p.w_type, col, w);
        if (p.b) load_any<E>(p.b, p.w_type, col, b);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            float2 d = make_float2(v[c][e], v[c][e + 1]);
            if (REST) d = add2(d, make_float2(-q.rest, -q.rest));
            const float2 o = fma2(mul2(d, make_float2(r, r)), make_float2(w[e], w[e + 1]), make_float2(b[e], b[e + 1]));
            v[c][e] = o.x;
            v[c][e + 1] = o.y;
        }
        store_vec<TY, E>(y + col, v[c]);
    }
}

// Rows too wide for registers: one block per row walks it three times (the
// second and third time from the cache).
template <typename TX, typename TY, int E>
__global__ void __launch_bounds__(512) ln_fwd_wide_kernel(const NormArgs p) {
    constexpr int T = 512;
    constexpr bool REST = sizeof(TX) == 4;
    __shared__ float red[T / 32];
    __shared__ float2 red2[T / 32];
    const int64_t row = blockIdx.x;
    const TX *x = static_cast<const TX *>(p.x) + row * p.ld_x;
    TY *y = static_cast<TY *>(p.y) + row * p.ld_y;
    float v[E];
    float s = 0.f;
    for (int64_t col = (int64_t)threadIdx.x * E; col < p.cols; col += T * E) {
        load_vec<TX, E>(x + col, v);
#pragma unroll
        for (int e = 0; e < E; ++e) s += v[e];
    }
    const float inv = 1.f / (float)p.cols;
    const float mu = divided(row_sum<T>(s, red), (float)p.cols, inv);
    float s2 = 0.f;
    s = 0.f;
    for (int64_t col = (int64_t)threadIdx.x * E; col < p.cols; col += T * E) {
        load_vec<TX, E>(x + col, v);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if (REST) s += v[e] - mu;
            s2 += (v[e] - mu) * (v[e] - mu);
        }
    }
    const float2 sums = row_sum2<T, REST>(s, s2, red2);
    const Spread q = spread<REST>(sums.x, sums.y, (float)p.cols, inv, p.eps);
    const float r = q.rstd;
    if (threadIdx.x == 0) {
        if (p.mean) p.mean[row] = q.mean(mu);
        if (p.rstd) p.rstd[row] = r;
    }
    for (int64_t col = (int64_t)threadIdx.x * E; col < p.cols; col += T * E) {
        load_vec<TX, E>(x + col, v);
        float w[E], b[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            w[e] = 1.f;
            b[e] = 0.f;
        }
        if (p.w) load_any<E>(p.w, p.w_type, col, w);
        if (p.b) load_any<E>(p.b, p.w_type, col, b);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = (v[e] - mu - q.rest) * r * w[e] + b[e];
        store_vec<TY, E>(y + col, v);
    }
}

// ---- rows in registers, any alignment ----------------------------------------
// A group of T threads walks rows, chunk c of thread t covering E columns from
// (c T + t) E - shift on.  With E = 8 or 4 rows are aligned and the shift is 0.
// Rows of an odd stride start on every other 2-element boundary only: with E =
// 2 ("Pairs") the shift is the parity of row * ld, so that every access of two
// elements is aligned; the groups' number is even, so a group's rows all have
// the same shift and its columns stay the same.  Elements outside the row (the
// shifted first pair, a last half pair) are left out.
template <typename T, int E>
__device__ __forceinline__ void load_cols(const T *row, int col, int D, float (&v)[E], float fill) {
    if (col >= 0 && col + E <= D) {
        load_vec<T, E>(row + col, v);
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = col + e >= 0 && col + e < D ? to_f(row[col + e]) : fill;
    }
}
template <typename T, int E>
__device__ __forceinline__ void store_cols(T *row, int col, int D, const float (&v)[E]) {
    if (col >= 0 && col + E <= D) {
        store_vec<T, E>(row + col, v);
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (col + e >= 0 && col + e < D) row[col + e] = from_f<T>(v[e]);
    }
}
// E elements as they lie in memory, so that values loaded ahead take no more
// registers than bytes.
template <typename T, int E>
struct Raw {
    static constexpr int N = (E * (int)sizeof(T) + 3) / 4;
    uint32_t w[N];
    __device__ __forceinline__ void load(const T *row, int col, int D) {
        constexpr int B = E * (int)sizeof(T);
        if (B >= 4 && col >= 0 && col + E <= D) {
            if constexpr (B >= 16) {
#pragma unroll
                for (int i = 0; i < B / 16; ++i) {
                    const uint4 q = reinterpret_cast<const uint4 *>(row + col)[i];
                    w[4 * i] = q.x;
                    w[4 * i + 1] = q.y;
                    w[4 * i + 2] = q.z;
                    w[4 * i + 3] = q.w;
                }
            } else if constexpr (B == 8) {
                const uint2 q = *reinterpret_cast<const uint2 *>(row + col);
                w[0] = q.x;
                w[1] = q.y;
            } else if constexpr (B == 4) {
                w[0] = *reinterpret_cast<const uint32_t *>(row + col);
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = 0;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (col + e < 0 || col + e >= D) continue;
                if constexpr (sizeof(T) == 4) w[e] = __float_as_uint(row[col + e]);
                else w[e / 2] |= (uint32_t) * reinterpret_cast<const uint16_t *>(row + col + e) << (16 * (e & 1));
            }
        }
    }
    __device__ __forceinline__ void get(float (&v)[E]) const {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = __uint_as_float(w[e]);
        } else if constexpr (E == 1) {
            float b;
            unpack2<T>(w[0], v[0], b);
        } else {
#pragma unroll
            for (int e = 0; e < E; e += 2) unpack2<T>(w[e / 2], v[e], v[e + 1]);
        }
    }
};
__device__ __forceinline__ float param(const void *p, int type, int col, int D, float otherwise) {
    float v[1] = {otherwise};
    if (p && col >= 0 && col < D) load_any<1>(p, type, col, v);
    return v[0];
}

// Sums of two values over the T threads of group g; `red` holds two floats per
// warp of the block, consecutive calls use different ones.
template <int T, int NT>
__device__ __forceinline__ void group_sum2(float &a, float &b, float (*red)[2], int g) {
    a = warp_sum(a);
    b = warp_sum(b);
    if constexpr (T > 32) {
        const int w = threadIdx.x >> 5, w0 = g * (T / 32);
        if ((threadIdx.x & 31) == 0) {
            red[w][0] = a;
            red[w][1] = b;
        }
        if constexpr (T == NT) __syncthreads();
        else asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "n"(T) : "memory");
        a = red[w0][0];
        b = red[w0][1];
#pragma unroll
        for (int i = 1; i < T / 32; ++i) {
            a += red[w0 + i][0];
            b += red[w0 + i][1];
        }
    }
}

// Forward of rows that no 16-byte access fits: weight and bias stay in
// registers over a group's rows, and the next row is loaded ahead.  4099 x 997
// bf16 -> fp32 takes 9.3 us, 17 with one element per access.  (Aligned rows are
// faster one by one, above: 4112 x 1024 bf16 5.1 us, 10.0 this way.)
template <typename TX, typename TY, int E, int NC, int T, int NT>
__global__ void __launch_bounds__(NT) ln_fwd_any_kernel(const NormArgs p) {
    constexpr int G = NT / T;
    constexpr bool REST = sizeof(TX) == 4;
    __shared__ float red[2][NT / 32][2];
    const int t = threadIdx.x % T, g = threadIdx.x / T, D = (int)p.cols;
    const int64_t first = (int64_t)blockIdx.x * G + g, step = (int64_t)gridDim.x * G;
    const int shift = E == 2 ? (int)((first * p.ld_x) & 1) : 0;
    float w[NC][E], b[NC][E];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int col = (c * T + t) * E - shift + e;
            w[c][e] = param(p.w, p.w_type, col, D, 1.f);
            b[c][e] = param(p.b, p.w_type, col, D, 0.f);
        }
    const float inv = 1.f / (float)D;
    Raw<TX, E> next[NC];  // the next row, loaded while the current one is worked on
    auto fetch = [&](int64_t row) {
        if (row >= p.rows) return;
#pragma unroll
        for (int c = 0; c < NC; ++c)
            next[c].load(static_cast<const TX *>(p.x) + row * p.ld_x, (c * T + t) * E - shift, D);
    };
    fetch(first);
    for (int64_t row = first; row < p.rows; row += step) {
        float v[NC][E];
        float s = 0.f, unused = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) next[c].get(v[c]);
        fetch(row + step);
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int e = 0; e < E; ++e) s += v[c][e];
        group_sum2<T, NT>(s, unused, red[0], g);
        const float mu = divided(s, (float)D, inv);
        float s2 = 0.f;
        s = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int col = (c * T + t) * E - shift + e;
                v[c][e] -= mu;
                if (col >= 0 && col < D) {
                    if (REST) s += v[c][e];
                    s2 += v[c][e] * v[c][e];
                }
            }
        group_sum2<T, NT>(s, s2, red[1], g);
        const Spread q = spread<REST>(s, s2, (float)D, inv, p.eps);
        const float r = q.rstd;
        if (t == 0) {
            if (p.mean) p.mean[row] = q.mean(mu);
            if (p.rstd) p.rstd[row] = r;
        }
        TY *y = static_cast<TY *>(p.y) + row * p.ld_y;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
#pragma unroll
            for (int e = 0; e < E; ++e) v[c][e] = (v[c][e] - q.rest) * r * w[c][e] + b[c][e];
            store_cols<TY, E>(y, (c * T + t) * E - shift, D, v[c]);
        }
    }
}

// Backward: every thread sums dy h and dy over its group's rows for its own
// columns; the block adds its groups' sums up in shared memory and writes one
// partial row of each (summed over blocks by finish_columns_kernel).  One block
// of 512 threads per SM keeps the partial rows few (444 blocks of 128 threads
// took 19 us for 4112 x 1024 bf16 with dx_add, these 12.3); its groups' rows in
// flight hide the memory's latency.
template <typename TX, typename TY, int E, int NC, int T, int NT>
__global__ void __launch_bounds__(NT, 1) ln_bwd_kernel(const NormArgs p) {
    constexpr int G = NT / T;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // [cols + 2] weights at 1 (a shifted first column is -1); then, for the
    // column sums, [G / 2][2][T * NC * E]
    extern __shared__ __align__(16) float smem[];
    __shared__ float red[2][NT / 32][2];
    const int t = threadIdx.x % T, g = threadIdx.x / T, D = (int)p.cols;
    const int64_t first = (int64_t)blockIdx.x * G + g, step = (int64_t)gridDim.x * G;
    const int shift = E == 2 ? (int)((first * p.ld_x) & 1) : 0;
    float *weight = smem + 4;  // keeps column 0 on a 16-byte boundary
    for (int i = (int)threadIdx.x - 1; i < T * NC * E; i += NT) weight[i] = param(p.w, p.w_type, i, D, 1.f);
    __syncthreads();
    float dw[NC][E], db[NC][E];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int e = 0; e < E; ++e) dw[c][e] = db[c][e] = 0.f;
    const float inv = 1.f / (float)D;
    int par = 0;
    // the next row's values, loaded while the current one is worked on
    Raw<TX, E> nx[NC];
    Raw<TY, E> nd[NC];
    float nmu = 0.f, nr = 0.f;
    auto fetch = [&](int64_t row) {
        if (row >= p.rows) return;
        const TX *x = static_cast<const TX *>(p.x) + row * p.ld_x;
        const TY *dy = static_cast<const TY *>(p.dy) + row * p.ld_y;
        nmu = p.mean[row];
        nr = p.rstd[row];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            nx[c].load(x, (c * T + t) * E - shift, D);
            nd[c].load(dy, (c * T + t) * E - shift, D);
        }
    };
    fetch(first);
    for (int64_t row = first; row < p.rows; row += step) {
        const float mu = nmu, r = nr;
        float h[NC][E], d[NC][E];
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int col = (c * T + t) * E - shift;
            float w[E];
            if constexpr (E >= 4) {
                load_vec<float, E>(weight + col, w);
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) w[e] = weight[col + e];
            }
            nx[c].get(h[c]);
            nd[c].get(d[c]);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                // dy is 0 outside the row, so nothing there counts
                h[c][e] = (h[c][e] - mu) * r;
                dw[c][e] += d[c][e] * h[c][e];
                db[c][e] += d[c][e];
                d[c][e] *= w[e];
                s1 += d[c][e];
                s2 += d[c][e] * h[c][e];
            }
        }
        fetch(row + step);
        if (!p.y) continue;
        group_sum2<T, NT>(s1, s2, red[par], g);
        par ^= 1;
        s1 *= inv;
        s2 *= inv;
        TX *dx = static_cast<TX *>(p.y) + row * p.ld_dx;
        const TX *add = static_cast<const TX *>(p.add) + row * p.ld_add;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int col = (c * T + t) * E - shift;
            float a[E];
#pragma unroll
            for (int e = 0; e < E; ++e) a[e] = 0.f;
            if (p.add) load_cols<TX, E>(add, col, D, a, 0.f);
#pragma unroll
            for (int e = 0; e < E; ++e) a[e] += r * (d[c][e] - (s1 + h[c][e] * s2));
            store_cols<TX, E>(dx, col, D, a);
        }
    }
    if (!p.part) return;
    // Aligned rows: by thread, without bank conflicts.  Pairs: by column, since
    // groups of either shift add up; each column belongs to one thread of a
    // group, and a barrier separates the steps.
    constexpr int W = T * NC * E;
    constexpr bool BY_THREAD = E >= 4;
    float *slices = smem + 4 + W + 4;
    auto at = [&](int c, int e) { return BY_THREAD ? (c * E + e) * T + t : (c * T + t) * E - shift + e; };
    auto inside = [&](int c, int e) { return BY_THREAD || (at(c, e) >= 0 && at(c, e) < D); };
#pragma unroll
    for (int half = G / 2; half >= 1; half /= 2) {
        if (g >= half && g < 2 * half) {
            float *s = slices + (g - half) * 2 * W;
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (inside(c, e)) {
                        s[at(c, e)] = dw[c][e];
                        s[W + at(c, e)] = db[c][e];
                    }
        }
        __syncthreads();
        if (g < half) {
            const float *s = slices + g * 2 * W;
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (inside(c, e)) {
                        dw[c][e] += s[at(c, e)];
                        db[c][e] += s[W + at(c, e)];
                    }
        }
        __syncthreads();
    }
    if (g != 0) return;
    float *out = p.part + (int64_t)blockIdx.x * 2 * D;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int col = (c * T + t) * E - shift;
        if constexpr (BY_THREAD) {
            if (col < D) {  // D is a multiple of E: both rows are aligned
                store_vec<float, E>(out + col, dw[c]);
                store_vec<float, E>(out + D + col, db[c]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (col + e >= 0 && col + e < D) {
                    out[col + e] = dw[c][e];
                    out[D + col + e] = db[c][e];
                }
        }
    }
}

// Backward of rows too wide for registers: dx by one block per row in two
// walks, the column sums by their own kernel.
template <typename TX, typename TY, int E>
__global__ void __launch_bounds__(512) ln_bwd_wide_dx_kernel(const NormArgs p) {
    constexpr int T = 512;
    __shared__ float red[2][T / 32];
    const int64_t row = blockIdx.x;
    const TX *x = static_cast<const TX *>(p.x) + row * p.ld_x;
    const TY *dy = static_cast<const TY *>(p.dy) + row * p.ld_y;
    const float mu = p.mean[row], r = p.rstd[row], inv = 1.f / (float)p.cols;
    float s1 = 0.f, s2 = 0.f;
    float h[E], d[E], w[E];
#pragma unroll
    for (int e = 0; e < E; ++e) w[e] = 1.f;
    for (int64_t col = (int64_t)threadIdx.x * E; col < p.cols; col += T * E) {
        load_vec<TX, E>(x + col, h);
        load_vec<TY, E>(dy + col, d);
        if (p.w) load_any<E>(p.w, p.w_type, col, w);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            s1 += d[e] * w[e];
            s2 += d[e] * w[e] * ((h[e] - mu) * r);
        }
    }
    s1 = row_sum<T>(s1, red[0]) * inv;
    s2 = row_sum<T>(s2, red[1]) * inv;
    TX *dx = static_cast<TX *>(p.y) + row * p.ld_dx;
    const TX *add = static_cast<const TX *>(p.add) + row * p.ld_add;
    for (int64_t col = (int64_t)threadIdx.x * E; col < p.cols; col += T * E) {
        load_vec<TX, E>(x + col, h);
        load_vec<TY, E>(dy + col, d);
        if (p.w) load_any<E>(p.w, p.w_type, col, w);
        float a[E];
#pragma unroll
        for (int e = 0; e < E; ++e) a[e] = 0.f;
        if (p.add) load_vec<TX, E>(add + col, a);
#pragma unroll
        for (int e = 0; e < E; ++e)
            a[e] += r * (d[e] * w[e] - (s1 + (h[e] - mu) * r * s2));
        store_vec<TX, E>(dx + col, a);
    }
}

// One column per lane, 8 rows of a block at a time, a chunk of the rows per
// blockIdx.y: one partial row each.
template <typename TX, typename TY>
__global__ void __launch_bounds__(256) ln_bwd_wide_cols_kernel(const NormArgs p) {
    __shared__ float sw[8][32], sb[8][32];
    const int lane = threadIdx.x & 31, q = threadIdx.x >> 5;
    const int64_t col = (int64_t)blockIdx.x * 32 + lane;
    float dw = 0.f, db = 0.f;
    if (col < p.cols) {
        for (int64_t row = (int64_t)blockIdx.y * 8 + q; row < p.rows; row += (int64_t)gridDim.y * 8) {
            const float d = to_f(static_cast<const TY *>(p.dy)[row * p.ld_y + col]);
            const float x = to_f(static_cast<const TX *>(p.x)[row * p.ld_x + col]);
            dw += d * ((x - p.mean[row]) * p.rstd[row]);
            db += d;
        }
    }
    sw[q][lane] = dw;
    sb[q][lane] = db;
    __syncthreads();
    if (q == 0 && col < p.cols) {
#pragma unroll
        for (int i = 1; i < 8; ++i) {
            dw += sw[i][lane];
            db += sb[i][lane];
        }
        float *out = p.part + (int64_t)blockIdx.y * 2 * p.cols;
        out[col] = dw;
        out[p.cols + col] = db;
    }
}

__global__ void __launch_bounds__(512) finish_columns_kernel(const float *part, int n_part, int n_out,
                                                             int64_t cols, void *out0, void *out1,
                                                             int out_type) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ float s[16][33];
    const int lane = threadIdx.x & 31, q = threadIdx.x >> 5;
    const int64_t i = (int64_t)blockIdx.x * 32 + lane, n = (int64_t)n_out * cols;
    float v = 0.f;
    if (i < n) {
#pragma unroll 8
        for (int k = q; k < n_part; k += 16) v += part[k * n + i];
    }
    s[q][lane] = v;
    __syncthreads();
    if (q == 0 && i < n) {
#pragma unroll
        for (int k = 1; k < 16; ++k) v += s[k][lane];
        void *o = i < cols ? out0 : out1;
        if (o) store_any(o, out_type, i < cols ? i : i - cols, v);
    }
}

template <typename TX, typename TY, int E, int NC, int T>
void fwd(const NormArgs &a, cudaStream_t s) {
    constexpr int NT = T < 128 ? 128 : T;
    ln_fwd_kernel<TX, TY, E, NC, T><<<(unsigned)div_up(a.rows, NT / T), NT, 0, s>>>(a);
}

template <typename TX, typename TY, int E, int T, int NT>
void fwd_any(const NormArgs &a, cudaStream_t s) {
    const int64_t most = 4 * sm_count();
    int64_t blocks = div_up(a.rows, NT / T) < most ? div_up(a.rows, NT / T) : most;
    blocks += blocks & 1;
    ln_fwd_any_kernel<TX, TY, E, 16 / E, T, NT><<<(unsigned)blocks, NT, 0, s>>>(a);
}

// How the rows lie: 16-byte accesses of every row, 2-element accesses (Pairs),
// or neither.
enum Access { VEC, PAIRS, SINGLE };

template <typename TX, typename TY, int ACCESS>
void fwd_rows(const NormArgs &a, cudaStream_t s) {
    // VEC: 8 columns per access (16 bytes of a 16-bit type), 4 where both are
    // fp32, and at most 32 values per thread; otherwise 16 values.
    const int64_t D = a.cols;
    constexpr int E = ACCESS == SINGLE ? 1 : ACCESS == PAIRS ? 2 : sizeof(TX) == 4 && sizeof(TY) == 4 ? 4 : 8;
    if constexpr (ACCESS == VEC) {
        if (D <= 256) return fwd<TX, TY, E, 8 / E, 32>(a, s);
        if (D <= 512) return fwd<TX, TY, E, 16 / E, 32>(a, s);
        if (D <= 1024) return fwd<TX, TY, E, 32 / E, 32>(a, s);
        if (D <= 4096) return fwd<TX, TY, E, 32 / E, 128>(a, s);
        if (D <= 16384) return fwd<TX, TY, E, 32 / E, 512>(a, s);
        ln_fwd_wide_kernel<TX, TY, E><<<(unsigned)a.rows, 512, 0, s>>>(a);
    } else {
        // a shifted row has one column more
        const int64_t W = D + (ACCESS == PAIRS);
        if (W <= 512) return fwd_any<TX, TY, E, 32, 256>(a, s);
        if (W <= 1024) return fwd_any<TX, TY, E, 64, 256>(a, s);
        if (W <= 2048) return fwd_any<TX, TY, E, 128, 256>(a, s);
        if (W <= 4096) return fwd_any<TX, TY, E, 256, 256>(a, s);
        if (W <= 8192) return fwd_any<TX, TY, E, 512, 512>(a, s);
        ln_fwd_wide_kernel<TX, TY, 1><<<(unsigned)a.rows, 512, 0, s>>>(a);
    }
}

template <typename TX, typename TY, int E, int NC, int T>
int bwd(const NormArgs &a, cudaStream_t s) {
    constexpr int NT = 512, G = NT / T, W = T * NC * E;
    int64_t blocks = div_up(a.rows, G);
    blocks += blocks & 1;
    if (blocks > bwd_blocks()) blocks = bwd_blocks();
    const size_t smem = (size_t)(4 + W + 4 + (a.part ? G / 2 * 2 * W : 0)) * sizeof(float);
    const auto kern = ln_bwd_kernel<TX, TY, E, NC, T, NT>;
    if (smem > 40 * 1024) cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    kern<<<(unsigned)blocks, NT, smem, s>>>(a);
    return (int)blocks;
}

// Returns the number of partial rows written.
template <typename TX, typename TY, int ACCESS>
int bwd_rows(const NormArgs &a, cudaStream_t s) {
    constexpr int E = ACCESS == SINGLE ? 1 : ACCESS == PAIRS ? 2 : sizeof(TX) == 4 && sizeof(TY) == 4 ? 4 : 8;
    const int64_t D = a.cols, W = D + (ACCESS == PAIRS);
    if (W <= 256) return bwd<TX, TY, E, 8 / E, 32>(a, s);
    if (W <= 512) return bwd<TX, TY, E, 16 / E, 32>(a, s);
    if (W <= 1024) return bwd<TX, TY, E, 16 / E, 64>(a, s);
    if (W <= 2048) return bwd<TX, TY, E, 16 / E, 128>(a, s);
    if (W <= 4096) return bwd<TX, TY, E, 16 / E, 256>(a, s);
    if (W <= 8192) return bwd<TX, TY, E, 16 / E, 512>(a, s);
    int n = 0;
    if (a.part) {
        const int64_t cb = div_up(D, 32);
        int64_t chunks = div_up(4 * sm_count(), cb);
        if (chunks > div_up(a.rows, 8)) chunks = div_up(a.rows, 8);
        n = (int)(chunks < bwd_blocks() ? chunks : bwd_blocks());
        ln_bwd_wide_cols_kernel<TX, TY><<<dim3((unsigned)cb, (unsigned)n), 256, 0, s>>>(a);
    }
    // the weight is read like the rows here, so it must be aligned like them
    if (a.y && ACCESS == VEC && aligned16(a.w)) ln_bwd_wide_dx_kernel<TX, TY, E><<<(unsigned)a.rows, 512, 0, s>>>(a);
    else if (a.y) ln_bwd_wide_dx_kernel<TX, TY, 1><<<(unsigned)a.rows, 512, 0, s>>>(a);
    return n;
}

template <int A>
using AccessC = std::integral_constant<int, A>;

template <typename F>
int by_types(int xt, int yt, Access access, const F &f) {
    using bf = __nv_bfloat16;
    auto with = [&](auto *x, auto *y) {
        if (access == VEC) return f(x, y, AccessC<VEC>());
        if (access == PAIRS) return f(x, y, AccessC<PAIRS>());
        return f(x, y, AccessC<SINGLE>());
    };
    if (xt == SC_F32 && yt == SC_F32) return with((float *)nullptr, (float *)nullptr);
    if (xt == SC_F32 && yt == SC_BF16) return with((float *)nullptr, (bf *)nullptr);
    if (xt == SC_F32) return with((float *)nullptr, (__half *)nullptr);
    if (xt == SC_BF16 && yt == SC_F32) return with((bf *)nullptr, (float *)nullptr);
    if (xt == SC_BF16) return with((bf *)nullptr, (bf *)nullptr);
    if (yt == SC_F32) return with((__half *)nullptr, (float *)nullptr);
    return with((__half *)nullptr, (__half *)nullptr);
}

int check_desc(const sc_norm_desc *d, const char *who) {
    if (!d) {
        set_error("%s: desc is null", who);
        return SC_ERR_ARG;
    }
    if (d->rows < 0 || d->cols < 1 || d->rows > INT32_MAX || d->cols > INT32_MAX) {
        set_error("%s: rows %lld (0 .. 2^31 - 1), cols %lld (1 .. 2^31 - 1)", who, (long long)d->rows,
                  (long long)d->cols);
        return SC_ERR_ARG;
    }
    if (!type_ok(d->x_type) || !type_ok(d->y_type) || !type_ok(d->w_type)) {
        set_error("%s: element types %d, %d, %d", who, d->x_type, d->y_type, d->w_type);
        return SC_ERR_ARG;
    }
    if (d->x_type != d->y_type && d->x_type != SC_F32 && d->y_type != SC_F32) {
        set_error("%s: two different 16-bit types", who);
        return SC_ERR_UNSUPPORTED;
    }
    return SC_OK;
}

int check_ld(int64_t ld, int64_t cols, const char *who, const char *name) {
    if (ld >= cols) return SC_OK;
    set_error("%s: %s %lld < cols %lld", who, name, (long long)ld, (long long)cols);
    return SC_ERR_ARG;
}

struct Matrix {
    const void *p;
    int64_t ld;
    int type;
};

Access access_of(const sc_norm_desc &d, const void *weight, const void *bias, std::initializer_list<Matrix> ms) {
    const int e = d.x_type == SC_F32 && d.y_type == SC_F32 ? 4 : 8;
    bool vec = d.cols % e == 0 && aligned16(weight) && aligned16(bias), pairs = true;
    for (const Matrix &m : ms) {
        if (!m.p) continue;
        vec = vec && aligned16(m.p) && m.ld % e == 0;
        // pairs begin on the same columns in every matrix
        pairs = pairs && reinterpret_cast<uintptr_t>(m.p) % (2 * type_size(m.type)) == 0 && (m.ld & 1) == (ms.begin()->ld & 1);
    }
    return vec ? VEC : pairs ? PAIRS : SINGLE;
}

int64_t bwd_workspace(const sc_norm_desc &d) {
    const int64_t most = bwd_blocks(), rows = d.rows + (d.rows & 1);
    return round_up((rows < most ? rows : most) * 2 * d.cols * (int64_t)sizeof(float), 256);
}

}  // namespace

int launch_finish_columns(const float *part, int n_part, int n_out, int64_t cols, void *out0,
                          void *out1, int out_type, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];  // begins under the kernel that writes the partial rows
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)div_up(n_out * cols, 32));
    cfg.blockDim = dim3(512);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, finish_columns_kernel, part, n_part, n_out, cols, out0, out1, out_type);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? SC_OK : cuda_fail(e, "column sums");
}

}  // namespace scb

using namespace scb;

extern "C" int sc_layer_norm(const sc_norm_desc *d, const void *x, const void *weight,
                             const void *bias, void *y, float *mean, float *rstd, void *stream) {
    const char *who = "sc_layer_norm";
    clear_error();
    if (int rc = check_desc(d, who)) return rc;
    if (!(d->eps >= 0.0) || isinf(d->eps)) {
        set_error("%s: eps must be finite and >= 0", who);
        return SC_ERR_ARG;
    }
    if (int rc = check_ld(d->ld_x, d->cols, who, "ld_x")) return rc;
    if (int rc = check_ld(d->ld_y, d->cols, who, "ld_y")) return rc;
    if (d->rows == 0) return SC_OK;
    if (!x || !y) {
        set_error("%s: null pointer", who);
        return SC_ERR_ARG;
    }
    NormArgs a = {};
    a.rows = d->rows;
    a.cols = d->cols;
    a.ld_x = d->ld_x;
    a.ld_y = d->ld_y;
    a.eps = (float)d->eps;
    a.w_type = d->w_type;
    a.x = x;
    a.w = weight;
    a.b = bias;
    a.y = y;
    a.mean = mean;
    a.rstd = rstd;
    const Access access = access_of(*d, weight, bias, {{x, d->ld_x, d->x_type}, {y, d->ld_y, d->y_type}});
    const cudaStream_t s = (cudaStream_t)stream;
    by_types(d->x_type, d->y_type, access, [&](auto *tx, auto *ty, auto v) {
        fwd_rows<std::remove_pointer_t<decltype(tx)>, std::remove_pointer_t<decltype(ty)>, decltype(v)::value>(a, s);
        return 0;
    });
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SC_OK : cuda_fail(e, who);
}

extern "C" int64_t sc_layer_norm_workspace_bytes(const sc_norm_desc *d) {
    clear_error();
    if (int rc = check_desc(d, "sc_layer_norm_workspace_bytes")) return -rc;
    return bwd_workspace(*d);
}

extern "C" int sc_layer_norm_backward(const sc_norm_desc *d, const void *dy, const void *x,
                                      const void *weight, const float *mean, const float *rstd,
                                      const void *dx_add, void *dx, void *dweight, void *dbias,
                                      void *stream) {
    const char *who = "sc_layer_norm_backward";
    clear_error();
    if (int rc = check_desc(d, who)) return rc;
    if (int rc = check_ld(d->ld_x, d->cols, who, "ld_x")) return rc;
    if (int rc = check_ld(d->ld_y, d->cols, who, "ld_y")) return rc;
    if (dx)
        if (int rc = check_ld(d->ld_dx, d->cols, who, "ld_dx")) return rc;
    if (dx && dx_add)
        if (int rc = check_ld(d->ld_add, d->cols, who, "ld_add")) return rc;
    const bool sums = dweight || dbias;
    if (d->rows > 0 && (!dy || !x || !mean || !rstd)) {
        set_error("%s: null pointer", who);
        return SC_ERR_ARG;
    }
    if (!dx && !sums) return SC_OK;
    if (sums && d->rows > 0) {
        if (!d->workspace || d->workspace_bytes < bwd_workspace(*d)) {
            set_error("%s: workspace of %lld bytes, %lld needed", who, (long long)d->workspace_bytes,
                      (long long)bwd_workspace(*d));
            return SC_ERR_ARG;
        }
        if (reinterpret_cast<uintptr_t>(d->workspace) & 255u) {
            set_error("%s: workspace is not 256-byte aligned", who);
            return SC_ERR_ARG;
        }
    }
    NormArgs a = {};
    a.rows = d->rows;
    a.cols = d->cols;
    a.ld_x = d->ld_x;
    a.ld_y = d->ld_y;
    a.ld_dx = d->ld_dx;
    a.ld_add = d->ld_add;
    a.w_type = d->w_type;
    a.x = x;
    a.dy = dy;
    a.w = weight;
    a.add = dx ? dx_add : nullptr;
    a.y = dx;
    a.mean = const_cast<float *>(mean);
    a.rstd = const_cast<float *>(rstd);
    a.part = sums ? static_cast<float *>(d->workspace) : nullptr;
    const cudaStream_t s = (cudaStream_t)stream;
    int n_part = 0;
    if (d->rows > 0) {
        const Access access = access_of(*d, nullptr, nullptr,
                                        {{x, d->ld_x, d->x_type}, {dy, d->ld_y, d->y_type},
                                         {dx, d->ld_dx, d->x_type}, {a.add, d->ld_add, d->x_type}});
        n_part = by_types(d->x_type, d->y_type, access, [&](auto *tx, auto *ty, auto v) {
            return bwd_rows<std::remove_pointer_t<decltype(tx)>, std::remove_pointer_t<decltype(ty)>, decltype(v)::value>(a, s);
        });
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return cuda_fail(e, who);
    }
    return sums ? launch_finish_columns(a.part, n_part, 2, d->cols, dweight, dbias, d->w_type, s) : SC_OK;
}
