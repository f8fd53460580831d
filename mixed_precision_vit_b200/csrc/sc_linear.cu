// sc_linear.cu -- the linear layer (matrix product with bias, activation and
// residual in one call) and its backward pass.
//
//   z = x w^T + bias,  out = act(z) + residual
//   dz = dout act'(z),  dx = dz w,  dw = dz^T x,  dbias_j = sum_i dz_ij
#include "sc_gemm.cuh"

namespace scb {
namespace {

// ---- passes over an operand -------------------------------------------------
// What the tensor cores cannot read in place goes through one pass into the
// workspace: 16-bit rows that do not start on 16-byte boundaries are copied
// into rows that do, fp32 values are split into three bf16 planes, and the
// backward pass turns dout into dz = dout act'(pre), summing its columns.
struct PassArgs {
    int64_t rows, cols, ld_in, ld_pre, ld_dst, plane;
    const void *in, *pre;  // pre: null without an activation
    void *dst;
    float *part;           // [gridDim.y][cols] column sums, or null
    int act;
};

enum { OUT_NONE = 0, OUT_COPY = 1, OUT_PLANES = 3 };

// x = p1 + p2 + p3 exactly (round to nearest, so |p2| <= 2^-8 |x| and the parts
// change sign freely; towards zero where rounding would overflow).  The parts
// of an infinity or a NaN are itself, 0, 0.
__device__ __forceinline__ void split3(float x, __nv_bfloat16 (&p)[3]) {
    p[0] = __float2bfloat16_rn(x);
    if (isinf(__bfloat162float(p[0])) && isfinite(x)) p[0] = __float2bfloat16_rz(x);
    float r = isfinite(x) ? x - __bfloat162float(p[0]) : 0.f;
    p[1] = __float2bfloat16_rn(r);
    p[2] = __float2bfloat16_rn(r - __bfloat162float(p[1]));
}

// Bound by device memory.  A warp reads E columns per lane of one row at a
// time; 8 warps of a block and gridDim.y blocks share the rows of 32 E columns.
template <typename TIN, typename T, int E, int OUT, int ACT>
__global__ void __launch_bounds__(256) pass_kernel(const PassArgs p) {
    const int lane = threadIdx.x & 31, q = threadIdx.x >> 5;
    const int64_t col = ((int64_t)blockIdx.x * 32 + lane) * E;
    float s[E];
#pragma unroll
    for (int e = 0; e < E; ++e) s[e] = 0.f;
    if (col < p.cols) {
        for (int64_t row = (int64_t)blockIdx.y * 8 + q; row < p.rows; row += (int64_t)gridDim.y * 8) {
            float v[E];
            load_vec<TIN, E>(static_cast<const TIN *>(p.in) + row * p.ld_in + col, v);
            if constexpr (ACT != SC_ACT_NONE) {
                float z[E];
                load_vec<T, E>(static_cast<const T *>(p.pre) + row * p.ld_pre + col, z);
#pragma unroll
                for (int e = 0; e < E; ++e) v[e] *= act_grad<ACT>(z[e]);
            }
#pragma unroll
            for (int e = 0; e < E; ++e) s[e] += v[e];
            if constexpr (OUT == OUT_COPY) {
                store_vec<T, E>(static_cast<T *>(p.dst) + row * p.ld_dst + col, v);
            } else if constexpr (OUT == OUT_PLANES) {
                __nv_bfloat16 *d = static_cast<__nv_bfloat16 *>(p.dst) + row * p.ld_dst + col;
                alignas(16) __nv_bfloat16 o[3][E];
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    __nv_bfloat16 t[3];
                    split3(v[e], t);
#pragma unroll
                    for (int k = 0; k < 3; ++k) o[k][e] = t[k];
                }
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    if constexpr (E == 8) *reinterpret_cast<uint4 *>(d + k * p.plane) = *reinterpret_cast<const uint4 *>(o[k]);
                    else d[k * p.plane] = o[k][0];
                }
            }
        }
    }
    if (!p.part) return;
    __shared__ float sums[8][32 * E];
#pragma unroll
    for (int e = 0; e < E; ++e) sums[q][lane * E + e] = s[e];
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * E; i += 256) {
        const int64_t c = (int64_t)blockIdx.x * 32 * E + i;
        if (c >= p.cols) break;
        float v = sums[0][i];
#pragma unroll
        for (int k = 1; k < 8; ++k) v += sums[k][i];
        p.part[(int64_t)blockIdx.y * p.cols + c] = v;
    }
}

int pass_chunks(int64_t rows, int64_t cols) {
    if (rows < 1 || cols < 1) return 1;
    int64_t c = div_up(8 * (int64_t)sm_count(), div_up(cols, 256));
    if (c > div_up(rows, 8)) c = div_up(rows, 8);
    return (int)c;
}

template <typename TIN, typename T, int OUT, int ACT>
void pass(const PassArgs &p, bool vec, int chunks, cudaStream_t s) {
    if (vec) pass_kernel<TIN, T, 8, OUT, ACT><<<dim3((unsigned)div_up(p.cols, 256), (unsigned)chunks), 256, 0, s>>>(p);
    else pass_kernel<TIN, T, 1, OUT, ACT><<<dim3((unsigned)div_up(p.cols, 32), (unsigned)chunks), 256, 0, s>>>(p);
}

template <typename TIN, typename T, int OUT>
void pass_act(const PassArgs &p, bool vec, int chunks, cudaStream_t s) {
    switch (p.pre ? p.act : SC_ACT_NONE) {
        case SC_ACT_RELU: return pass<TIN, T, OUT, SC_ACT_RELU>(p, vec, chunks, s);
        case SC_ACT_GELU: return pass<TIN, T, OUT, SC_ACT_GELU>(p, vec, chunks, s);
        case SC_ACT_GELU_TANH: return pass<TIN, T, OUT, SC_ACT_GELU_TANH>(p, vec, chunks, s);
        case SC_ACT_SILU: return pass<TIN, T, OUT, SC_ACT_SILU>(p, vec, chunks, s);
        default: return pass<TIN, T, OUT, SC_ACT_NONE>(p, vec, chunks, s);
    }
}

template <typename TIN, typename T, int OUT>
void pass_out(const PassArgs &p, bool vec, int chunks, cudaStream_t s) {
    if (p.dst) pass_act<TIN, T, OUT>(p, vec, chunks, s);
    else pass_act<TIN, T, OUT_NONE>(p, vec, chunks, s);
}

bool rows_ok(const void *p, int64_t ld, int type) { return aligned16(p) && ld * type_size(type) % 16 == 0; }

// One pass; `type` is the operand type, `in_type` what is read.
int launch_pass(const PassArgs &p, int in_type, int type, cudaStream_t s) {
    const bool vec = p.cols % 8 == 0 && rows_ok(p.in, p.ld_in, in_type) && (!p.pre || rows_ok(p.pre, p.ld_pre, type));
    const int chunks = pass_chunks(p.rows, p.cols);
    using bf = __nv_bfloat16;
    if (type == SC_F32) pass_out<float, float, OUT_PLANES>(p, vec, chunks, s);
    else if (type == SC_BF16 && in_type == SC_F32) pass_out<float, bf, OUT_COPY>(p, vec, chunks, s);
    else if (type == SC_BF16) pass_out<bf, bf, OUT_COPY>(p, vec, chunks, s);
    else if (in_type == SC_F32) pass_out<float, __half, OUT_COPY>(p, vec, chunks, s);
    else pass_out<__half, __half, OUT_COPY>(p, vec, chunks, s);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SC_OK : cuda_fail(e, "sc_linear: operand pass");
}

// ---- operands ---------------------------------------------------------------
int tc_type(int type) { return type == SC_F32 ? SC_BF16 : type; }
bool in_place(const void *p, int64_t ld, int type) { return type != SC_F32 && rows_ok(p, ld, type); }
int64_t copy_bytes(int64_t rows, int64_t cols, int type) {
    return round_up((type == SC_F32 ? 3 : 1) * rows * round_up(cols, 8) * 2, 256);
}

// Takes workspace in order of the calls.
struct Scratch {
    char *p;
    void *take(int64_t bytes) {
        void *r = p;
        p += bytes;
        return r;
    }
};

GemmOperand copied(void *p, int64_t rows, int64_t cols, int type) {
    GemmOperand o = {};
    o.p = p;
    o.ld = round_up(cols, 8);
    o.planes = type == SC_F32 ? 3 : 1;
    o.plane_stride = rows * o.ld;
    return o;
}

// The operand as the matrix product reads it: in place, or through a pass.
int operand(const void *p, int64_t rows, int64_t cols, int64_t ld, int type, Scratch &ws, GemmOperand &o, cudaStream_t s) {
    if (in_place(p, ld, type)) {
        o = {};
        o.p = p;
        o.ld = ld;
        o.planes = 1;
        return SC_OK;
    }
    o = copied(ws.take(copy_bytes(rows, cols, type)), rows, cols, type);
    PassArgs a = {};
    a.rows = rows;
    a.cols = cols;
    a.ld_in = ld;
    a.in = p;
    a.dst = const_cast<void *>(o.p);
    a.ld_dst = o.ld;
    a.plane = o.plane_stride;
    return launch_pass(a, type, type, s);
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

int64_t fwd_workspace(const sc_linear_desc &d, const void *x, const void *w) {
    return (in_place(x, d.ld_x, d.type) ? 0 : copy_bytes(d.M, d.K, d.type)) +
           (in_place(w, d.ld_w, d.type) ? 0 : copy_bytes(d.N, d.K, d.type));
}

// dz is dout itself
bool dz_in_place(const sc_linear_desc &d, const void *dout) {
    return d.act == SC_ACT_NONE && d.out_type == d.type && in_place(dout, d.ld_out, d.type);
}

int64_t part_bytes(const sc_linear_desc &d) {
    return round_up((int64_t)pass_chunks(d.M, d.N) * d.N * (int64_t)sizeof(float), 256);
}

int64_t bwd_workspace(const sc_linear_desc &d, const void *dout, const void *x, const void *w) {
    return part_bytes(d) + (dz_in_place(d, dout) ? 0 : copy_bytes(d.M, d.N, d.type)) + fwd_workspace(d, x, w);
}

}  // namespace
}  // namespace scb

using namespace scb;

extern "C" int64_t sc_linear_workspace_bytes(const sc_linear_desc *d, const void *x, const void *w) {
    clear_error();
    if (int rc = check_desc(d, "sc_linear_workspace_bytes")) return -rc;
    return d->M == 0 || d->N == 0 ? 0 : fwd_workspace(*d, x, w);
}

extern "C" int64_t sc_linear_backward_workspace_bytes(const sc_linear_desc *d, const void *dout,
                                                      const void *x, const void *w) {
    clear_error();
    if (int rc = check_desc(d, "sc_linear_backward_workspace_bytes")) return -rc;
    return d->M == 0 || d->N == 0 ? 0 : bwd_workspace(*d, dout, x, w);
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
    if (int rc = check_workspace(*d, fwd_workspace(*d, x, w), who)) return rc;
    const cudaStream_t s = (cudaStream_t)stream;
    Scratch ws = {static_cast<char *>(d->workspace)};
    GemmOperand a, b;
    if (int rc = operand(x, d->M, d->K, d->ld_x, d->type, ws, a, s)) return rc;
    if (int rc = operand(w, d->N, d->K, d->ld_w, d->type, ws, b, s)) return rc;
    a.k_major = b.k_major = true;
    GemmEpilogue e = {};
    e.bias = bias;
    e.res = residual;
    e.out = out;
    e.pre = pre;
    e.ld_out = d->ld_out;
    e.ld_res = d->ld_res;
    e.ld_pre = d->ld_pre;
    e.bias_type = d->bias_type;
    e.out_type = d->out_type;
    e.pre_type = d->type;
    e.act = d->act;
    return launch_gemm(d->M, d->N, d->K, tc_type(d->type), a, b, e, dev_status, s);
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
        if (int rc = check_workspace(*d, bwd_workspace(*d, dout, x, w), who)) return rc;
    } else {
        // an empty sum: zeros
        cudaError_t e = cudaSuccess;
        if (dx && d->M > 0) e = cudaMemset2DAsync(dx, d->ld_dx * type_size(d->type), 0, d->K * type_size(d->type), d->M, s);
        if (e == cudaSuccess && dw && d->N > 0)
            e = cudaMemset2DAsync(dw, d->ld_dw * type_size(d->grad_type), 0, d->K * type_size(d->grad_type), d->N, s);
        if (e == cudaSuccess && dbias && d->N > 0) e = cudaMemsetAsync(dbias, 0, d->N * type_size(d->grad_type), s);
        return e == cudaSuccess ? SC_OK : cuda_fail(e, who);
    }
    Scratch ws = {static_cast<char *>(d->workspace)};
    GemmOperand dz = {};
    PassArgs p = {};
    p.rows = d->M;
    p.cols = d->N;
    p.ld_in = d->ld_out;
    p.ld_pre = d->ld_pre;
    p.in = dout;
    p.pre = pre;
    p.act = d->act;
    float *part = static_cast<float *>(ws.take(part_bytes(*d)));
    p.part = dbias ? part : nullptr;
    if (dz_in_place(*d, dout)) {
        dz.p = dout;
        dz.ld = d->ld_out;
        dz.planes = 1;
    } else {
        dz = copied(ws.take(copy_bytes(d->M, d->N, d->type)), d->M, d->N, d->type);
        if (dx || dw) p.dst = const_cast<void *>(dz.p);
        p.ld_dst = dz.ld;
        p.plane = dz.plane_stride;
    }
    if (p.dst || p.part)
        if (int rc = launch_pass(p, d->out_type, d->type, s)) return rc;
    GemmEpilogue e = {};
    GemmOperand b;
    if (dx) {
        if (int rc = operand(w, d->N, d->K, d->ld_w, d->type, ws, b, s)) return rc;
        dz.k_major = true;
        b.k_major = false;
        e.out = dx;
        e.ld_out = d->ld_dx;
        e.out_type = d->type;
        if (int rc = launch_gemm(d->M, d->K, d->N, tc_type(d->type), dz, b, e, dev_status, s)) return rc;
    }
    if (dw) {
        if (int rc = operand(x, d->M, d->K, d->ld_x, d->type, ws, b, s)) return rc;
        dz.k_major = false;
        b.k_major = false;
        e.out = dw;
        e.ld_out = d->ld_dw;
        e.out_type = d->grad_type;
        if (int rc = launch_gemm(d->N, d->K, d->M, tc_type(d->type), dz, b, e, dev_status, s)) return rc;
    }
    if (dbias) return launch_finish_columns(part, pass_chunks(d->M, d->N), 1, d->N, dbias, nullptr, d->grad_type, s);
    return SC_OK;
}
