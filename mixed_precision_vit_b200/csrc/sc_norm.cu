// sc_norm.cu -- layer norm and its backward pass.
//
// Forward, per row of D values:   mu = sum x / D,  v = sum (x - mu)^2 / D,
// r = 1 / sqrt(v + eps),  y = (x - mu) r w + b.
// Backward, with h = (x - mu) r, g = dy w, s1 = sum_j g, s2 = sum_j g h:
//   dx = r (g - (s1 + h s2) / D) [+ dx_add],
//   dw_j = sum_i dy_ij h_ij,  db_j = sum_i dy_ij.
// Both are bound by device memory: a row is read once and held in registers.
#include "sc_layers.cuh"

namespace scb {
namespace {

// Blocks per SM that hold column sums in the backward pass: one partial row of
// dweight and dbias each.
constexpr int BWD_BLOCKS_PER_SM = 3;

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

// T threads per row, each holding NC chunks of E columns (chunk c of thread t
// starts at column (c T + t) E), so D <= T NC E.  VEC: every chunk is inside
// the row and aligned; otherwise E = 1.
template <typename TX, typename TY, int E, int NC, int T>
__global__ void __launch_bounds__(T < 128 ? 128 : T) ln_fwd_kernel(const NormArgs p) {
    constexpr int RPB = T < 128 ? 128 / T : 1;
    __shared__ float red[2][T / 32];
    const int t = threadIdx.x % T;
    const int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / T;
    if (row >= p.rows) return;  // whole warps (T = 32) only
    const TX *x = static_cast<const TX *>(p.x) + row * p.ld_x;
    float v[NC][E];
    float s = 0.f;
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
        for (int e = 0; e < E; ++e) s += v[c][e];
    }
    const float inv = 1.f / (float)p.cols;
    const float mu = row_sum<T>(s, red[0]) * inv;
    s = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
        if ((int64_t)(c * T + t) * E < p.cols)
#pragma unroll
            for (int e = 0; e < E; ++e) s += (v[c][e] - mu) * (v[c][e] - mu);
    const float r = 1.f / sqrtf(row_sum<T>(s, red[1]) * inv + p.eps);
    if (t == 0) {
        if (p.mean) p.mean[row] = mu;
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
        for (int e = 0; e < E; ++e) v[c][e] = (v[c][e] - mu) * r * w[e] + b[e];
        store_vec<TY, E>(y + col, v[c]);
    }
}

// Rows too wide for registers: one block per row walks it three times (the
// second and third time from the cache).
template <typename TX, typename TY, int E>
__global__ void __launch_bounds__(512) ln_fwd_wide_kernel(const NormArgs p) {
    constexpr int T = 512;
    __shared__ float red[2][T / 32];
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
    const float mu = row_sum<T>(s, red[0]) * inv;
    s = 0.f;
    for (int64_t col = (int64_t)threadIdx.x * E; col < p.cols; col += T * E) {
        load_vec<TX, E>(x + col, v);
#pragma unroll
        for (int e = 0; e < E; ++e) s += (v[e] - mu) * (v[e] - mu);
    }
    const float r = 1.f / sqrtf(row_sum<T>(s, red[1]) * inv + p.eps);
    if (threadIdx.x == 0) {
        if (p.mean) p.mean[row] = mu;
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
        for (int e = 0; e < E; ++e) v[e] = (v[e] - mu) * r * w[e] + b[e];
        store_vec<TY, E>(y + col, v);
    }
}

// Backward with the row in registers: T threads per row as in the forward,
// NT / T rows per block at a time; every thread sums dy h and dy over the
// block's rows for its own columns, and the block writes one partial row of
// each (summed over blocks by finish_columns_kernel).
template <typename TX, typename TY, int E, int NC, int T, int NT>
__global__ void __launch_bounds__(NT) ln_bwd_kernel(const NormArgs p) {
    static_assert(T == 32 || T == NT, "a warp or the block per row");
    constexpr int G = NT / T;
    extern __shared__ float slices[];  // T = 32: [G / 2][2][cols] when the column sums are wanted
    __shared__ float red[2][2][T / 32];
    const int t = threadIdx.x % T, g = threadIdx.x / T;
    float dw[NC][E], db[NC][E];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int e = 0; e < E; ++e) dw[c][e] = db[c][e] = 0.f;
    const float inv = 1.f / (float)p.cols;
    int par = 0;
    for (int64_t row = (int64_t)blockIdx.x * G + g; row < p.rows; row += (int64_t)gridDim.x * G) {
        const TX *x = static_cast<const TX *>(p.x) + row * p.ld_x;
        const TY *dy = static_cast<const TY *>(p.dy) + row * p.ld_y;
        const float mu = p.mean[row], r = p.rstd[row];
        float h[NC][E], d[NC][E];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int64_t col = (int64_t)(c * T + t) * E;
            if (col < p.cols) {
                load_vec<TX, E>(x + col, h[c]);
                load_vec<TY, E>(dy + col, d[c]);
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    h[c][e] = mu;
                    d[c][e] = 0.f;
                }
            }
        }
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int64_t col = (int64_t)(c * T + t) * E;
            if (col >= p.cols) continue;
            float w[E];
#pragma unroll
            for (int e = 0; e < E; ++e) w[e] = 1.f;
            if (p.w) load_any<E>(p.w, p.w_type, col, w);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                h[c][e] = (h[c][e] - mu) * r;
                dw[c][e] += d[c][e] * h[c][e];
                db[c][e] += d[c][e];
                d[c][e] *= w[e];
                s1 += d[c][e];
                s2 += d[c][e] * h[c][e];
            }
        }
        if (!p.y) continue;
        if constexpr (T == 32) {
            s1 = warp_sum(s1);
            s2 = warp_sum(s2);
        } else {
            s1 = warp_sum(s1);
            s2 = warp_sum(s2);
            if ((threadIdx.x & 31) == 0) {
                red[par][0][threadIdx.x >> 5] = s1;
                red[par][1][threadIdx.x >> 5] = s2;
            }
            __syncthreads();
            s1 = red[par][0][0];
            s2 = red[par][1][0];
#pragma unroll
            for (int i = 1; i < T / 32; ++i) {
                s1 += red[par][0][i];
                s2 += red[par][1][i];
            }
            par ^= 1;
        }
        s1 *= inv;
        s2 *= inv;
        TX *dx = static_cast<TX *>(p.y) + row * p.ld_dx;
        const TX *add = static_cast<const TX *>(p.add) + row * p.ld_add;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int64_t col = (int64_t)(c * T + t) * E;
            if (col >= p.cols) continue;
            float a[E];
#pragma unroll
            for (int e = 0; e < E; ++e) a[e] = 0.f;
            if (p.add) load_vec<TX, E>(add + col, a);
#pragma unroll
            for (int e = 0; e < E; ++e) a[e] += r * (d[c][e] - (s1 + h[c][e] * s2));
            store_vec<TX, E>(dx + col, a);
        }
    }
    if (!p.part) return;
    float *out = p.part + (int64_t)blockIdx.x * 2 * p.cols;
    if constexpr (G > 1) {
        // halve the warps until one holds the block's sums
#pragma unroll
        for (int half = G / 2; half >= 1; half /= 2) {
            if (g >= half && g < 2 * half) {
                float *s = slices + (int64_t)(g - half) * 2 * p.cols;
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const int64_t col = (int64_t)(c * T + t) * E;
                    if (col >= p.cols) continue;
                    store_vec<float, E>(s + col, dw[c]);
                    store_vec<float, E>(s + p.cols + col, db[c]);
                }
            }
            __syncthreads();
            if (g < half) {
                const float *s = slices + (int64_t)g * 2 * p.cols;
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const int64_t col = (int64_t)(c * T + t) * E;
                    if (col >= p.cols) continue;
                    float a[E], b[E];
                    load_vec<float, E>(s + col, a);
                    load_vec<float, E>(s + p.cols + col, b);
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        dw[c][e] += a[e];
                        db[c][e] += b[e];
                    }
                }
            }
            __syncthreads();
        }
        if (g != 0) return;
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int64_t col = (int64_t)(c * T + t) * E;
        if (col >= p.cols) continue;
        store_vec<float, E>(out + col, dw[c]);
        store_vec<float, E>(out + p.cols + col, db[c]);
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

template <typename TX, typename TY, bool VEC>
void fwd_rows(const NormArgs &a, cudaStream_t s) {
    // 8 columns per access (16 bytes of a 16-bit type), 4 where both are fp32;
    // one where rows are not aligned.  At most 32 values per thread.
    constexpr int E = !VEC ? 1 : (sizeof(TX) == 4 && sizeof(TY) == 4 ? 4 : 8);
    const int64_t D = a.cols;
    if (D <= 256) fwd<TX, TY, E, 8 / E, 32>(a, s);
    else if (D <= 512) fwd<TX, TY, E, 16 / E, 32>(a, s);
    else if (D <= 1024) fwd<TX, TY, E, 32 / E, 32>(a, s);
    else if (D <= 4096) fwd<TX, TY, E, 32 / E, 128>(a, s);
    else if (D <= 16384) fwd<TX, TY, E, 32 / E, 512>(a, s);
    else ln_fwd_wide_kernel<TX, TY, E><<<(unsigned)a.rows, 512, 0, s>>>(a);
}

template <typename TX, typename TY, int E, int NC, int T, int NT>
int bwd(const NormArgs &a, int blocks, cudaStream_t s) {
    const size_t smem = a.part && T < NT ? (size_t)(NT / T / 2) * 2 * a.cols * sizeof(float) : 0;
    ln_bwd_kernel<TX, TY, E, NC, T, NT><<<(unsigned)blocks, NT, smem, s>>>(a);
    return blocks;
}

// Returns the number of partial rows written.
template <typename TX, typename TY, bool VEC>
int bwd_rows(const NormArgs &a, cudaStream_t s) {
    constexpr int E = !VEC ? 1 : (sizeof(TX) == 4 && sizeof(TY) == 4 ? 4 : 8);
    const int64_t D = a.cols;
    const int most = BWD_BLOCKS_PER_SM * sm_count();
    const int b4 = (int)(div_up(a.rows, 4) < most ? div_up(a.rows, 4) : most);
    const int b1 = (int)(a.rows < most ? a.rows : most);
    if (D <= 256) return bwd<TX, TY, E, 8 / E, 32, 128>(a, b4, s);
    if (D <= 1024) return bwd<TX, TY, E, 32 / E, 32, 128>(a, b4, s);
    if (D <= 4096) return bwd<TX, TY, E, 32 / E, 128, 128>(a, b1, s);
    if (D <= 8192) return bwd<TX, TY, E, 16 / E, 512, 512>(a, b1, s);
    int n = 0;
    if (a.part) {
        const int64_t cb = div_up(D, 32);
        int64_t chunks = div_up(4 * sm_count(), cb);
        if (chunks > div_up(a.rows, 8)) chunks = div_up(a.rows, 8);
        n = (int)(chunks < most ? chunks : most);
        ln_bwd_wide_cols_kernel<TX, TY><<<dim3((unsigned)cb, (unsigned)n), 256, 0, s>>>(a);
    }
    if (a.y) ln_bwd_wide_dx_kernel<TX, TY, E><<<(unsigned)a.rows, 512, 0, s>>>(a);
    return n;
}

template <typename F>
int by_types(int xt, int yt, bool vec, const F &f) {
    using bf = __nv_bfloat16;
#define SC_PAIR(a, b, A, B)                          \
    if (xt == a && yt == b) return vec ? f((A *)nullptr, (B *)nullptr, std::true_type()) \
                                       : f((A *)nullptr, (B *)nullptr, std::false_type());
    SC_PAIR(SC_F32, SC_F32, float, float)
    SC_PAIR(SC_F32, SC_BF16, float, bf)
    SC_PAIR(SC_F32, SC_F16, float, __half)
    SC_PAIR(SC_BF16, SC_F32, bf, float)
    SC_PAIR(SC_BF16, SC_BF16, bf, bf)
    SC_PAIR(SC_F16, SC_F32, __half, float)
    SC_PAIR(SC_F16, SC_F16, __half, __half)
#undef SC_PAIR
    return 0;
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

// Columns of one vector access, and whether a matrix allows it on every row.
int vec_of(const sc_norm_desc &d) { return d.x_type == SC_F32 && d.y_type == SC_F32 ? 4 : 8; }
bool vec_ok(const sc_norm_desc &d, const void *p, int64_t ld) {
    return !p || (aligned16(p) && ld % vec_of(d) == 0);
}

int64_t bwd_workspace(const sc_norm_desc &d) {
    const int64_t most = (int64_t)BWD_BLOCKS_PER_SM * sm_count();
    return round_up((d.rows < most ? d.rows : most) * 2 * d.cols * (int64_t)sizeof(float), 256);
}

}  // namespace

int launch_finish_columns(const float *part, int n_part, int n_out, int64_t cols, void *out0,
                          void *out1, int out_type, cudaStream_t stream) {
    finish_columns_kernel<<<(unsigned)div_up(n_out * cols, 32), 512, 0, stream>>>(
        part, n_part, n_out, cols, out0, out1, out_type);
    const cudaError_t e = cudaGetLastError();
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
    const bool vec = d->cols % vec_of(*d) == 0 && vec_ok(*d, x, d->ld_x) && vec_ok(*d, y, d->ld_y) &&
                     vec_ok(*d, weight, 0) && vec_ok(*d, bias, 0);
    const cudaStream_t s = (cudaStream_t)stream;
    by_types(d->x_type, d->y_type, vec, [&](auto *tx, auto *ty, auto v) {
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
        const bool vec = d->cols % vec_of(*d) == 0 && vec_ok(*d, x, d->ld_x) &&
                         vec_ok(*d, dy, d->ld_y) && vec_ok(*d, dx, d->ld_dx) &&
                         vec_ok(*d, a.add, d->ld_add) && vec_ok(*d, weight, 0);
        n_part = by_types(d->x_type, d->y_type, vec, [&](auto *tx, auto *ty, auto v) {
            return bwd_rows<std::remove_pointer_t<decltype(tx)>, std::remove_pointer_t<decltype(ty)>, decltype(v)::value>(a, s);
        });
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return cuda_fail(e, who);
    }
    return sums ? launch_finish_columns(a.part, n_part, 2, d->cols, dweight, dbias, d->w_type, s) : SC_OK;
}
