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
//
// 16-bit operands: dz is rounded to their type, as a layer's results are, for the
// products (not for the sums).  It is the one rounding besides the results' own:
// fc1's gradients (4112 x 4096 x 1024 bf16, gelu) are off by 2.35e-3 of their norm,
// 1.66e-3 with an unrounded dz.  Two bf16 parts of dz would keep it and run each
// product twice: 29 us become 53 for dx and 52 for dw, 86 about 132 for the call.
// A caller who needs more has fp32 operands.
struct PassJob {
    int64_t rows, cols, ld_in, ld_pre, ld_dst, plane;
    const void *in, *pre;  // pre: null without an activation
    void *dst;             // null: column sums only
    float *part;           // [chunks][cols] column sums, or null
    int vec;               // rows of 8-column pieces on 16-byte boundaries
    int lanes;             // lanes per row (a power of two): 8 columns each
    int chunks;            // blocks that share the rows of one group of columns
    int first_block;
};
// The passes of one call, run by one launch: job 0 may be dz (its own type and
// activation), the others are copies.
constexpr int MAX_JOBS = 3;
struct PassArgs {
    PassJob job[MAX_JOBS];
    int n;
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

// 8 elements from p on with the widest accesses that its address allows (the
// same for every lane of a row): 16 bytes, 4 or 2 elements, or 2 elements after
// a first one.  n < 8: only n exist.
template <typename T>
__device__ __forceinline__ void load8(const T *p, int n, float (&v)[8]) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    if (n < 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? to_f(p[i]) : 0.f;
    } else if ((at & 15) == 0) {
        load_vec<T, 8>(p, v);
    } else if ((at & (4 * sizeof(T) - 1)) == 0) {
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            float t[4];
            load_vec<T, 4>(p + i, t);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[i + k] = t[k];
        }
    } else if ((at & (2 * sizeof(T) - 1)) == 0) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            float t[2];
            load_vec<T, 2>(p + i, t);
            v[i] = t[0];
            v[i + 1] = t[1];
        }
    } else {
        v[0] = to_f(p[0]);
#pragma unroll
        for (int i = 1; i < 7; i += 2) {
            float t[2];
            load_vec<T, 2>(p + i, t);
            v[i] = t[0];
            v[i + 1] = t[1];
        }
        v[7] = to_f(p[7]);
    }
}

constexpr int BLOCK_COLS = 256;  // most columns of a block: 8 per lane

// One block's share of a job: `lanes` lanes take 8 columns each of a row, so a
// warp takes 32 / lanes rows and the block 8 times that.  The copy's rows are
// padded with zeros to a multiple of 8 columns.  Copies are bound by device
// memory; dz of a gelu layer by its instructions (4112 x 4096 bf16: 25 us from
// device memory, 16 at the copy's rate; schedulers 57 % busy).
// VEC: all of it lies on 16-byte boundaries.
template <typename TIN, typename T, int OUT, int ACT, bool VEC>
__device__ __forceinline__ void run_job(const PassJob &p, int block, float (*sums)[BLOCK_COLS]) {
    const int lane = threadIdx.x & 31, q = threadIdx.x >> 5;
    const int64_t col0 = (int64_t)(block / p.chunks) * BLOCK_COLS, col = col0 + (lane & (p.lanes - 1)) * 8;
    const int chunk = block % p.chunks;
    const int per_warp = 32 / p.lanes, per_block = 8 * per_warp;
    const int n = (int)(p.cols - col < 8 ? p.cols - col : 8);
    float s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = 0.f;
    if (n > 0) {
        for (int64_t row = (int64_t)chunk * per_block + q * per_warp + lane / p.lanes; row < p.rows;
             row += (int64_t)p.chunks * per_block) {
            float v[8];
            const TIN *in = static_cast<const TIN *>(p.in) + row * p.ld_in + col;
            if constexpr (VEC) load_vec<TIN, 8>(in, v);
            else load8(in, n, v);
            if constexpr (ACT != SC_ACT_NONE) {
                const T *pre = static_cast<const T *>(p.pre) + row * p.ld_pre + col;
                float z[8];
                if constexpr (VEC) load_vec<T, 8>(pre, z);
                else load8(pre, n, z);
                times_act_grad<ACT, 8>(v, z);
            }
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const float2 t = add2(make_float2(s[e], s[e + 1]), make_float2(v[e], v[e + 1]));
                s[e] = t.x;
                s[e + 1] = t.y;
            }
            if constexpr (OUT == OUT_COPY) {
                store_vec<T, 8>(static_cast<T *>(p.dst) + row * p.ld_dst + col, v);
            } else if constexpr (OUT == OUT_PLANES) {
                __nv_bfloat16 *d = static_cast<__nv_bfloat16 *>(p.dst) + row * p.ld_dst + col;
                float o[3][8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    __nv_bfloat16 t[3];
                    split3(v[e], t);
#pragma unroll
                    for (int k = 0; k < 3; ++k) o[k][e] = __bfloat162float(t[k]);
                }
#pragma unroll
                for (int k = 0; k < 3; ++k) store_vec<__nv_bfloat16, 8>(d + k * p.plane, o[k]);
            }
        }
    }
    if (!p.part) return;
    // the warp's rows, then the block's
    for (int o = 16; o >= p.lanes; o >>= 1)
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] += __shfl_xor_sync(0xffffffffu, s[e], o);
    if (lane < p.lanes) {
#pragma unroll
        for (int e = 0; e < 8; ++e) sums[q][lane * 8 + e] = s[e];
    }
    __syncthreads();
    if ((int)threadIdx.x < p.lanes * 8 && col0 + threadIdx.x < p.cols) {
        float v = sums[0][threadIdx.x];
#pragma unroll
        for (int k = 1; k < 8; ++k) v += sums[k][threadIdx.x];
        p.part[(int64_t)chunk * p.cols + col0 + threadIdx.x] = v;
    }
}

template <typename TIN, typename T, int OUT0, int ACT>
__global__ void __launch_bounds__(256) pass_kernel(const __grid_constant__ PassArgs p) {
    // the matrix product that follows may set itself up now; it waits for this
    // grid's end before it reads
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ float sums[8][BLOCK_COLS];
    constexpr int OUT = sizeof(T) == 4 ? OUT_PLANES : OUT_COPY;
    int j = 0;
    while (j + 1 < p.n && (int)blockIdx.x >= p.job[j + 1].first_block) ++j;
    const PassJob &job = p.job[j];
    const int block = (int)blockIdx.x - job.first_block;
    if (j == 0) {
        if (job.vec) run_job<TIN, T, OUT0, ACT, true>(job, block, sums);
        else run_job<TIN, T, OUT0, ACT, false>(job, block, sums);
    } else {
        if (job.vec) run_job<T, T, OUT, SC_ACT_NONE, true>(job, block, sums);
        else run_job<T, T, OUT, SC_ACT_NONE, false>(job, block, sums);
    }
}

int pass_lanes(int64_t cols) {
    int l = 1;
    while (l < 32 && l * 8 < cols) l *= 2;
    return l;
}

// Blocks that share a group of columns: 8 per SM in all (4 to 8 measure alike
// for dz, fewer are slower for copies), with column sums at most 256, which one
// warp adds up while a product runs.
int pass_chunks(int64_t rows, int64_t cols, bool sums) {
    if (rows < 1 || cols < 1) return 1;
    const int64_t most = div_up(rows, 8 * 32 / pass_lanes(cols));
    int64_t c = div_up(8 * (int64_t)sm_count(), div_up(cols, BLOCK_COLS));
    if (sums && c > 256) c = 256;
    return (int)(c < most ? c : most);
}

template <typename TIN, typename T, int OUT0>
int launch_pass_act(const PassArgs &p, int act, int blocks, cudaStream_t s) {
    switch (act) {
        case SC_ACT_RELU: pass_kernel<TIN, T, OUT0, SC_ACT_RELU><<<blocks, 256, 0, s>>>(p); break;
        case SC_ACT_GELU: pass_kernel<TIN, T, OUT0, SC_ACT_GELU><<<blocks, 256, 0, s>>>(p); break;
        case SC_ACT_GELU_TANH: pass_kernel<TIN, T, OUT0, SC_ACT_GELU_TANH><<<blocks, 256, 0, s>>>(p); break;
        case SC_ACT_SILU: pass_kernel<TIN, T, OUT0, SC_ACT_SILU><<<blocks, 256, 0, s>>>(p); break;
        default: pass_kernel<TIN, T, OUT0, SC_ACT_NONE><<<blocks, 256, 0, s>>>(p); break;
    }
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SC_OK : cuda_fail(e, "sc_linear: operand pass");
}
template <typename TIN, typename T, int OUT>
int launch_pass_out(const PassArgs &p, int act, int blocks, cudaStream_t s) {
    return p.job[0].dst ? launch_pass_act<TIN, T, OUT>(p, act, blocks, s)
                        : launch_pass_act<TIN, T, OUT_NONE>(p, act, blocks, s);
}

bool rows_ok(const void *p, int64_t ld, int type) { return aligned16(p) && ld * type_size(type) % 16 == 0; }

// The passes of a call; `type` is the operand type.
struct Passes {
    PassArgs a = {};
    int act0 = SC_ACT_NONE, in0 = SC_F32;  // of job 0

    void add(const PassJob &j, int in_type, int act, int type) {
        if (a.n == 0) {
            act0 = act;
            in0 = in_type;
        }
        PassJob &o = a.job[a.n++];
        o = j;
        o.vec = j.cols % 8 == 0 && rows_ok(j.in, j.ld_in, in_type) && (!j.pre || rows_ok(j.pre, j.ld_pre, type));
    }
    int launch(int type, cudaStream_t s) {
        if (a.n == 0) return SC_OK;
        int64_t blocks = 0;
        for (int i = 0; i < a.n; ++i) {
            PassJob &j = a.job[i];
            if (blocks > INT32_MAX / 2) break;
            j.lanes = pass_lanes(j.cols);
            j.chunks = pass_chunks(j.rows, j.cols, j.part != nullptr);
            j.first_block = (int)blocks;
            blocks += div_up(j.cols, BLOCK_COLS) * j.chunks;
        }
        if (blocks > INT32_MAX / 2) {
            set_error("sc_linear: the operands are too large");
            return SC_ERR_ARG;
        }
        using bf = __nv_bfloat16;
        const int n = (int)blocks;
        if (type == SC_F32) return launch_pass_out<float, float, OUT_PLANES>(a, act0, n, s);
        if (type == SC_BF16 && in0 == SC_F32) return launch_pass_out<float, bf, OUT_COPY>(a, act0, n, s);
        if (type == SC_BF16) return launch_pass_out<bf, bf, OUT_COPY>(a, act0, n, s);
        if (in0 == SC_F32) return launch_pass_out<float, __half, OUT_COPY>(a, act0, n, s);
        return launch_pass_out<__half, __half, OUT_COPY>(a, act0, n, s);
    }
};

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

// A matrix that the product reads where it is.  One row's stride means nothing,
// so a tensor map, which takes strides below 2^40 bytes, gets another.
GemmOperand placed(const void *p, int64_t rows, int64_t cols, int64_t ld) {
    GemmOperand o = {};
    o.p = p;
    o.ld = rows > 1 ? ld : round_up(cols, 8);
    o.planes = 1;
    return o;
}

GemmOperand copied(void *p, int64_t rows, int64_t cols, int type) {
    GemmOperand o = {};
    o.p = p;
    o.ld = round_up(cols, 8);
    o.planes = type == SC_F32 ? 3 : 1;
    o.plane_stride = rows * o.ld;
    return o;
}

// The operand as the matrix product reads it: in place, or through a pass.
GemmOperand operand(const void *p, int64_t rows, int64_t cols, int64_t ld, int type, bool k_major, Scratch &ws,
                    Passes &passes) {
    GemmOperand o = {};
    if (in_place(p, ld, type)) {
        o = placed(p, rows, cols, ld);
    } else {
        o = copied(ws.take(copy_bytes(rows, cols, type)), rows, cols, type);
        PassJob j = {};
        j.rows = rows;
        j.cols = cols;
        j.ld_in = ld;
        j.in = p;
        j.dst = const_cast<void *>(o.p);
        j.ld_dst = o.ld;
        j.plane = o.plane_stride;
        passes.add(j, type, SC_ACT_NONE, type);
    }
    o.k_major = k_major;
    return o;
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
    // more than any address space holds, and what workspace sizes could not count
    constexpr int64_t MOST = (int64_t)1 << 56;
    if (d->M * d->N > MOST || d->M * d->K > MOST || d->N * d->K > MOST) {
        set_error("%s: a matrix of more than 2^56 elements (M %lld, N %lld, K %lld)", who, (long long)d->M, (long long)d->N,
                  (long long)d->K);
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

// What the copies of x and w take; a null operand is not read.
int64_t fwd_workspace(const sc_linear_desc &d, const void *x, const void *w) {
    return (!x || in_place(x, d.ld_x, d.type) ? 0 : copy_bytes(d.M, d.K, d.type)) +
           (!w || in_place(w, d.ld_w, d.type) ? 0 : copy_bytes(d.N, d.K, d.type));
}

// dz is dout itself
bool dz_in_place(const sc_linear_desc &d, const void *dout) {
    return d.act == SC_ACT_NONE && d.out_type == d.type && in_place(dout, d.ld_out, d.type);
}

int64_t part_bytes(const sc_linear_desc &d) {
    return round_up((int64_t)pass_chunks(d.M, d.N, true) * d.N * (int64_t)sizeof(float), 256);
}

// x: null unless dw is wanted, w: null unless dx is; sums: dbias is wanted.
int64_t bwd_workspace(const sc_linear_desc &d, const void *dout, const void *x, const void *w, bool sums) {
    return (sums ? part_bytes(d) : 0) + ((!x && !w) || dz_in_place(d, dout) ? 0 : copy_bytes(d.M, d.N, d.type)) +
           fwd_workspace(d, x, w);
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
    return d->M == 0 || d->N == 0 ? 0 : bwd_workspace(*d, dout, x, w, true);
}

// wait_limit: see launch_gemm
static int linear(const char *who, const sc_linear_desc *d, const void *x, const void *w, const void *bias,
                  const void *residual, void *out, void *pre, int32_t *dev_status, void *stream, int64_t wait_limit) {
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
    Passes passes;
    const GemmOperand a = operand(x, d->M, d->K, d->ld_x, d->type, true, ws, passes);
    const GemmOperand b = operand(w, d->N, d->K, d->ld_w, d->type, true, ws, passes);
    if (int rc = passes.launch(d->type, s)) return rc;
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
    return launch_gemm(d->M, d->N, d->K, tc_type(d->type), a, b, e, passes.a.n ? AFTER_PASS : AFTER_ANY, nullptr, dev_status, s,
                       wait_limit);
}

extern "C" int sc_linear(const sc_linear_desc *d, const void *x, const void *w, const void *bias,
                         const void *residual, void *out, void *pre, int32_t *dev_status,
                         void *stream) {
    clear_error();
    return linear("sc_linear", d, x, w, bias, residual, out, pre, dev_status, stream, 0);
}

extern "C" int sc_selftest_linear_wait_limit(const sc_linear_desc *d, const void *x, const void *w, void *out, void *pre,
                                             int64_t limit_cycles, int32_t *dev_status, void *stream) {
    const char *who = "sc_selftest_linear_wait_limit";
    clear_error();
    if (!dev_status || limit_cycles < 1 || limit_cycles > (int64_t)1 << 34) {
        set_error("%s: dev_status is null, or limit %lld outside [1, 2^34] cycles", who, (long long)limit_cycles);
        return SC_ERR_ARG;
    }
    return linear(who, d, x, w, nullptr, nullptr, out, pre, dev_status, stream, limit_cycles);
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
        if (int rc = check_workspace(*d, bwd_workspace(*d, dout, dw ? x : nullptr, dx ? w : nullptr, dbias), who)) return rc;
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
    Passes passes;
    ColumnSums sums = {};
    PassJob p = {};
    p.rows = d->M;
    p.cols = d->N;
    p.ld_in = d->ld_out;
    p.ld_pre = d->ld_pre;
    p.in = dout;
    p.pre = pre;
    if (dbias) p.part = static_cast<float *>(ws.take(part_bytes(*d)));
    GemmOperand dz = {};
    if (dz_in_place(*d, dout)) {
        dz = placed(dout, d->M, d->N, d->ld_out);
    } else if (dx || dw) {
        dz = copied(ws.take(copy_bytes(d->M, d->N, d->type)), d->M, d->N, d->type);
        p.dst = const_cast<void *>(dz.p);
        p.ld_dst = dz.ld;
        p.plane = dz.plane_stride;
    }
    if (p.dst || p.part) passes.add(p, d->out_type, d->act, d->type);
    GemmOperand bw = {}, bx = {};
    if (dx) bw = operand(w, d->N, d->K, d->ld_w, d->type, false, ws, passes);
    if (dw) bx = operand(x, d->M, d->K, d->ld_x, d->type, false, ws, passes);
    if (int rc = passes.launch(d->type, s)) return rc;
    if (dbias) {
        sums.part = p.part;
        sums.n = passes.a.job[0].chunks;
        sums.cols = d->N;
        sums.out = dbias;
        sums.type = d->grad_type;
    }
    GemmEpilogue e = {};
    if (dx) {
        dz.k_major = true;
        e.out = dx;
        e.ld_out = d->ld_dx;
        e.out_type = d->type;
        if (int rc = launch_gemm(d->M, d->K, d->N, tc_type(d->type), dz, bw, e, passes.a.n ? AFTER_PASS : AFTER_ANY,
                                 dbias && !dw ? &sums : nullptr, dev_status, s))
            return rc;
    }
    if (dw) {
        dz.k_major = false;
        e.out = dw;
        e.ld_out = d->ld_dw;
        e.out_type = d->grad_type;
        if (int rc = launch_gemm(d->N, d->K, d->M, tc_type(d->type), dz, bx, e,
                                 dx ? BESIDE_GEMM : passes.a.n ? AFTER_PASS : AFTER_ANY, dbias ? &sums : nullptr,
                                 dev_status, s))
            return rc;
    }
    if (dbias && !dx && !dw)
        return launch_finish_columns(sums.part, sums.n, 1, sums.cols, dbias, nullptr, sums.type, s);
    return SC_OK;
}
