// sc_linear.cu -- the linear layer (matrix product with bias, activation and
// residual in one call) and its backward pass.
//
//   z = x w^T + bias,  out = act(z) + residual
//   dz = dout act'(z),  dx = dz w,  dw = dz^T x,  dbias_j = sum_i dz_ij
#include "sc_layers.cuh"

namespace scb {
namespace {

// ---- activations ------------------------------------------------------------
__device__ __forceinline__ float act_fn(float z, int act) {
    switch (act) {
        case SC_ACT_RELU: return z > 0.f ? z : (z == z ? 0.f : z);
        case SC_ACT_GELU: return 0.5f * z * (1.f + erff(z * 0.70710678f));
        case SC_ACT_GELU_TANH: return 0.5f * z * (1.f + tanhf(0.79788456f * (z + 0.044715f * z * z * z)));
        case SC_ACT_SILU: return z / (1.f + expf(-z));
        default: return z;
    }
}

__device__ __forceinline__ float act_grad(float z, int act) {
    switch (act) {
        case SC_ACT_RELU: return z > 0.f ? 1.f : (z == z ? 0.f : z);
        case SC_ACT_GELU:
            return 0.5f * (1.f + erff(z * 0.70710678f)) + z * 0.39894228f * expf(-0.5f * z * z);
        case SC_ACT_GELU_TANH: {
            const float t = tanhf(0.79788456f * (z + 0.044715f * z * z * z));
            return 0.5f * (1.f + t) + 0.5f * z * (1.f - t * t) * 0.79788456f * (1.f + 0.134145f * z * z);
        }
        case SC_ACT_SILU: {
            const float q = 1.f / (1.f + expf(-z));
            return q * (1.f + z * (1.f - q));
        }
        default: return 1.f;
    }
}

// ---- gradient of the pre-activation -----------------------------------------
struct PassArgs {
    int64_t rows, cols, ld_in, ld_pre, ld_dst;
    const void *in, *pre;  // pre: null without an activation
    void *dst;             // null: column sums only
    float *part;           // [gridDim.y][cols] column sums, or null
    int act;
};

template <typename TIN, typename T>
__global__ void __launch_bounds__(256) dz_kernel(const PassArgs p) {
    __shared__ float sums[8][32];
    const int lane = threadIdx.x & 31, q = threadIdx.x >> 5;
    const int64_t col = (int64_t)blockIdx.x * 32 + lane;
    float s = 0.f;
    if (col < p.cols) {
        for (int64_t row = (int64_t)blockIdx.y * 8 + q; row < p.rows; row += (int64_t)gridDim.y * 8) {
            float v = to_f(static_cast<const TIN *>(p.in)[row * p.ld_in + col]);
            if (p.pre) v *= act_grad(to_f(static_cast<const T *>(p.pre)[row * p.ld_pre + col]), p.act);
            s += v;
            if (p.dst) static_cast<T *>(p.dst)[row * p.ld_dst + col] = from_f<T>(v);
        }
    }
    if (!p.part) return;
    sums[q][lane] = s;
    __syncthreads();
    if (q == 0 && col < p.cols) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += sums[i][lane];
        p.part[(int64_t)blockIdx.y * p.cols + col] = s;
    }
}

// ---- matrix product ---------------------------------------------------------
struct GemmArgs {
    int64_t M, N, K;
    int64_t am, ak, bn, bk;  // strides of A(m, k) and B(n, k)
    const void *a, *b, *bias, *res;
    void *out, *pre;
    int64_t ld_out, ld_res, ld_pre;
    int bias_type, out_type, act;
};

// D(m, n) = sum_k A(m, k) B(n, k) on the CUDA cores: 64 x 64 tiles, 4 x 4
// outputs per thread, fp32 products and sums.
template <typename T>
__global__ void __launch_bounds__(256) gemm_simt_kernel(const GemmArgs p) {
    __shared__ float sa[16][65], sb[16][65];
    const int64_t m0 = (int64_t)blockIdx.y * 64, n0 = (int64_t)blockIdx.x * 64;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int64_t k0 = 0; k0 < p.K; k0 += 16) {
        for (int i = threadIdx.x; i < 64 * 16; i += 256) {
            const int r = i / 16, k = i % 16;
            const bool kin = k0 + k < p.K;
            sa[k][r] = kin && m0 + r < p.M ? to_f(static_cast<const T *>(p.a)[(m0 + r) * p.am + (k0 + k) * p.ak]) : 0.f;
            sb[k][r] = kin && n0 + r < p.N ? to_f(static_cast<const T *>(p.b)[(n0 + r) * p.bn + (k0 + k) * p.bk]) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 16; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] += sa[k][ty + 16 * i] * sb[k][tx + 16 * j];
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (m >= p.M || n >= p.N) continue;
            float z = acc[i][j];
            float b[1] = {0.f};
            if (p.bias) load_any<1>(p.bias, p.bias_type, n, b);
            z += b[0];
            if (p.pre) static_cast<T *>(p.pre)[m * p.ld_pre + n] = from_f<T>(z);
            float o = act_fn(z, p.act), r[1] = {0.f};
            if (p.res) load_any<1>(p.res, p.out_type, m * p.ld_res + n, r);
            store_any(p.out, p.out_type, m * p.ld_out + n, o + r[0]);
        }
}

int gemm(const GemmArgs &a, int type, cudaStream_t s) {
    const dim3 grid((unsigned)div_up(a.N, 64), (unsigned)div_up(a.M, 64));
    if (type == SC_F32) gemm_simt_kernel<float><<<grid, 256, 0, s>>>(a);
    else if (type == SC_BF16) gemm_simt_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(a);
    else gemm_simt_kernel<__half><<<grid, 256, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SC_OK : cuda_fail(e, "sc_linear: matrix product");
}

// ---- checks and workspace ---------------------------------------------------
int check_desc(const sc_linear_desc *d, const char *who) {
    if (!d) {
        set_error("%s: desc is null", who);
        return SC_ERR_ARG;
    }
    if (d->M < 0 || d->N < 0 || d->K < 1 || d->M > INT32_MAX || d->N > INT32_MAX || d->K > INT32_MAX) {
        set_error("%s: sizes M %lld, N %lld (0 .. 2^31 - 1), K %lld (1 .. 2^31 - 1)", who,
                  (long long)d->M, (long long)d->N, (long long)d->K);
        return SC_ERR_ARG;
    }
    if (!type_ok(d->type) || !type_ok(d->out_type) || (d->out_type != d->type && d->out_type != SC_F32)) {
        set_error("%s: type %d with out_type %d", who, d->type, d->out_type);
        return SC_ERR_ARG;
    }
    if (d->act < SC_ACT_NONE || d->act > SC_ACT_SILU) {
        set_error("%s: activation %d", who, d->act);
        return SC_ERR_ARG;
    }
    if (d->workspace_bytes < 0 || (reinterpret_cast<uintptr_t>(d->workspace) & 255u)) {
        set_error("%s: workspace_bytes < 0, or the workspace is not 256-byte aligned", who);
        return SC_ERR_ARG;
    }
    return SC_OK;
}

int check_matrix(const void *p, int64_t ld, int64_t cols, const char *who, const char *name) {
    if (p && ld < cols) {
        set_error("%s: row stride of %s %lld < %lld columns", who, name, (long long)ld, (long long)cols);
        return SC_ERR_ARG;
    }
    return SC_OK;
}

int check_workspace(const sc_linear_desc &d, int64_t need, const char *who) {
    if (need > 0 && (!d.workspace || d.workspace_bytes < need)) {
        set_error("%s: workspace of %lld bytes, %lld needed", who, (long long)d.workspace_bytes,
                  (long long)need);
        return SC_ERR_ARG;
    }
    return SC_OK;
}

int pass_chunks(int64_t rows, int64_t cols) {
    if (rows < 1 || cols < 1) return 1;
    int64_t c = div_up(8 * (int64_t)sm_count(), div_up(cols, 32));
    if (c > div_up(rows, 8)) c = div_up(rows, 8);
    return (int)(c < 1 ? 1 : c);
}

int64_t dz_bytes(const sc_linear_desc &d) { return round_up(d.M * d.N * type_size(d.type), 256); }
int64_t bwd_workspace(const sc_linear_desc &d) {
    return dz_bytes(d) + round_up((int64_t)pass_chunks(d.M, d.N) * d.N * 4, 256);
}

}  // namespace
}  // namespace scb

using namespace scb;

extern "C" int64_t sc_linear_workspace_bytes(const sc_linear_desc *d, const void *x, const void *w) {
    clear_error();
    if (int rc = check_desc(d, "sc_linear_workspace_bytes")) return -rc;
    return 0;
}

extern "C" int64_t sc_linear_backward_workspace_bytes(const sc_linear_desc *d, const void *dout,
                                                      const void *x, const void *w) {
    clear_error();
    if (int rc = check_desc(d, "sc_linear_backward_workspace_bytes")) return -rc;
    return bwd_workspace(*d);
}

extern "C" int sc_linear(const sc_linear_desc *d, const void *x, const void *w, const void *bias,
                         const void *residual, void *out, void *pre, int32_t *dev_status,
                         void *stream) {
    const char *who = "sc_linear";
    clear_error();
    if (int rc = check_desc(d, who)) return rc;
    if (bias && !type_ok(d->bias_type)) {
        set_error("%s: bias_type %d", who, d->bias_type);
        return SC_ERR_ARG;
    }
    if (d->M == 0 || d->N == 0) return SC_OK;
    if (!x || !w || !out) {
        set_error("%s: null pointer", who);
        return SC_ERR_ARG;
    }
    if (int rc = check_matrix(x, d->ld_x, d->K, who, "x")) return rc;
    if (int rc = check_matrix(w, d->ld_w, d->K, who, "w")) return rc;
    if (int rc = check_matrix(out, d->ld_out, d->N, who, "out")) return rc;
    if (int rc = check_matrix(residual, d->ld_res, d->N, who, "residual")) return rc;
    if (int rc = check_matrix(pre, d->ld_pre, d->N, who, "pre")) return rc;
    GemmArgs a = {};
    a.M = d->M;
    a.N = d->N;
    a.K = d->K;
    a.am = d->ld_x;
    a.ak = 1;
    a.bn = d->ld_w;
    a.bk = 1;
    a.a = x;
    a.b = w;
    a.bias = bias;
    a.res = residual;
    a.out = out;
    a.pre = pre;
    a.ld_out = d->ld_out;
    a.ld_res = d->ld_res;
    a.ld_pre = d->ld_pre;
    a.bias_type = d->bias_type;
    a.out_type = d->out_type;
    a.act = d->act;
    return gemm(a, d->type, (cudaStream_t)stream);
}

extern "C" int sc_linear_backward(const sc_linear_desc *d, const void *dout, const void *x,
                                  const void *w, const void *pre, void *dx, void *dw, void *dbias,
                                  int32_t *dev_status, void *stream) {
    const char *who = "sc_linear_backward";
    clear_error();
    if (int rc = check_desc(d, who)) return rc;
    if ((dw || dbias) && !type_ok(d->grad_type)) {
        set_error("%s: grad_type %d", who, d->grad_type);
        return SC_ERR_ARG;
    }
    if (int rc = check_matrix(dx, d->ld_dx, d->K, who, "dx")) return rc;
    if (int rc = check_matrix(dw, d->ld_dw, d->K, who, "dw")) return rc;
    const cudaStream_t s = (cudaStream_t)stream;
    if (d->act == SC_ACT_NONE) pre = nullptr;
    if (!dx && !dw && !dbias) return SC_OK;
    if (d->M > 0 && d->N > 0) {
        if (!dout || (dx && !w) || (dw && !x) || (d->act != SC_ACT_NONE && !pre)) {
            set_error("%s: null pointer", who);
            return SC_ERR_ARG;
        }
        if (int rc = check_matrix(dout, d->ld_out, d->N, who, "dout")) return rc;
        if (int rc = check_matrix(dx ? w : nullptr, d->ld_w, d->K, who, "w")) return rc;
        if (int rc = check_matrix(dw ? x : nullptr, d->ld_x, d->K, who, "x")) return rc;
        if (int rc = check_matrix(pre, d->ld_pre, d->N, who, "pre")) return rc;
        if (int rc = check_workspace(*d, bwd_workspace(*d), who)) return rc;
    }
    PassArgs p = {};
    p.rows = d->M;
    p.cols = d->N;
    p.ld_in = d->ld_out;
    p.ld_pre = d->ld_pre;
    p.ld_dst = d->N;
    p.in = dout;
    p.pre = pre;
    p.dst = d->workspace;
    p.part = dbias ? reinterpret_cast<float *>(static_cast<char *>(d->workspace) + dz_bytes(*d)) : nullptr;
    p.act = d->act;
    const int chunks = pass_chunks(d->M, d->N);
    if (d->M > 0 && d->N > 0) {
        const dim3 grid((unsigned)div_up(d->N, 32), (unsigned)chunks);
        if (d->type == SC_F32) dz_kernel<float, float><<<grid, 256, 0, s>>>(p);
        else if (d->type == SC_BF16 && d->out_type == SC_F32) dz_kernel<float, __nv_bfloat16><<<grid, 256, 0, s>>>(p);
        else if (d->type == SC_BF16) dz_kernel<__nv_bfloat16, __nv_bfloat16><<<grid, 256, 0, s>>>(p);
        else if (d->out_type == SC_F32) dz_kernel<float, __half><<<grid, 256, 0, s>>>(p);
        else dz_kernel<__half, __half><<<grid, 256, 0, s>>>(p);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return cuda_fail(e, who);
    }
    GemmArgs a = {};
    if (dx && d->M > 0) {
        a.M = d->M;
        a.N = d->K;
        a.K = d->N;
        a.a = p.dst;
        a.am = d->N;
        a.ak = 1;
        a.b = w;
        a.bn = 1;
        a.bk = d->ld_w;
        a.out = dx;
        a.ld_out = d->ld_dx;
        a.out_type = d->type;
        if (int rc = gemm(a, d->type, s)) return rc;
    }
    if (dw && d->N > 0) {
        a.M = d->N;
        a.N = d->K;
        a.K = d->M;
        a.a = p.dst;
        a.am = 1;
        a.ak = d->N;
        a.b = x;
        a.bn = 1;
        a.bk = d->ld_x;
        a.out = dw;
        a.ld_out = d->ld_dw;
        a.out_type = d->grad_type;
        if (int rc = gemm(a, d->type, s)) return rc;
    }
    if (dbias && d->N > 0)
        return launch_finish_columns(p.part, d->M > 0 ? chunks : 0, 1, d->N, dbias, nullptr, d->grad_type, s);
    return SC_OK;
}
