// sc_gemm.cu -- host side of the matrix product: tensor maps, tile shapes and
// launches of the kernels in sc_gemm_dev.cuh.
#include "sc_gemm_dev.cuh"
#include <atomic>

namespace scb {
namespace {

using namespace gemm;

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static const EncodeFn fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            f = nullptr;
        }
        return reinterpret_cast<EncodeFn>(f);
    }();
    return fn;
}

bool encode(CUtensorMap *map, int type16, const GemmOperand &o, int64_t rows, int64_t k, int tile_rows) {
    const EncodeFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)(o.k_major ? k : rows), (cuuint64_t)(o.k_major ? rows : k),
                                (cuuint64_t)o.planes};
    const cuuint64_t row_bytes = (cuuint64_t)o.ld * 2;
    const cuuint64_t strides[2] = {row_bytes, o.planes > 1 ? (cuuint64_t)o.plane_stride * 2 : row_bytes};
    const cuuint32_t box[3] = {64, (cuuint32_t)(o.k_major ? tile_rows : GK), 1};
    const cuuint32_t one[3] = {1, 1, 1};
    return fn(map, type16 == SC_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
              const_cast<void *>(o.p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 8 columns per access: rows on 16-byte boundaries
bool vec_rows(const void *p, int64_t ld, int type) { return aligned16(p) && ld * type_size(type) % 16 == 0; }

// early: may start before the previous kernel on the stream has ended (the
// kernel itself waits for it, see GemmAfter).
int launch(GemmFn kern, const GemmArgs &p, int grid, int cluster, bool early, cudaStream_t stream) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, GEMM_SMEM);
    if (e != cudaSuccess) return cuda_fail(e, "matrix product: smem attribute");
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = cluster;
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (early) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(GEMM_THREADS);
    cfg.dynamicSmemBytes = GEMM_SMEM;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = n;
    e = cudaLaunchKernelEx(&cfg, kern, p);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? SC_OK : cuda_fail(e, "matrix product");
}

// A kernel that moves registers between its warps waits for ever if it was
// launched with fewer than the moves add up to, so a build that gave it another
// number is refused (asked once per kernel).
bool keep_regs_ok(GemmFn kern) {
    static std::atomic<GemmFn> known[20];  // two tile widths, two types, five activations
    for (auto &k : known)
        if (k.load(std::memory_order_relaxed) == kern) return true;
    cudaFuncAttributes a;
    if (cudaFuncGetAttributes(&a, kern) != cudaSuccess || a.numRegs != KEEP_REGS) return false;
    for (auto &k : known) {
        GemmFn none = nullptr;
        if (k.compare_exchange_strong(none, kern)) break;
    }
    return true;
}

// Clusters of `parts` CTAs of the split kernel that fit the device at one
// time (asked once per device and size; fewer than SMs / parts, since a
// cluster stays within one GPC).
int split_clusters(int parts) {
    constexpr int DEVICES = 64;
    static std::atomic<int> known[DEVICES][MAX_PARTS + 1];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= DEVICES) return sm_count() / (2 * parts);
    int n = known[dev][parts].load(std::memory_order_relaxed);
    if (n > 0) return n;
    const GemmFn kern = gemm_kernels_none().split;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = parts;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(parts * sm_count()));
    cfg.blockDim = dim3(GEMM_THREADS);
    cfg.dynamicSmemBytes = GEMM_SMEM;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, GEMM_SMEM) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();
        return sm_count() / (2 * parts);
    }
    known[dev][parts].store(n, std::memory_order_relaxed);
    return n;
}

struct Shape {
    int cg, bn, parts;
};

// The tile shape with the least estimated time.  Measured (us, bf16): a stage
// of 64 indexes costs 0.30 in a pair's 256 x 256 tile and 0.24 in a CTA's 128 x
// 128 tile or less (there the issuing threads, not the products, set the pace);
// a launch 6.0 or 5.0 besides; a shared tile costs 0.008 per column for its
// epilogue and 0.005 per column and part for the exchange.  So 4112 x 1024 x 4096 takes 25.5 in pairs
// (68 tiles, one round) and 37.2 in single CTAs (264 tiles, two rounds); 2056 x
// 1024 x 1024 takes 10.6 and 8.5; 257 x 1024 x 4096 takes 13.0 in 4 parts of
// 128 columns and 28 unshared.  A step of fp32 operands (three stages, six
// products) costs 1.75 in a pair, 1.2 in a CTA alone, 1.1 and 1.0 in parts of 128
// and 64 columns: 257 x 1024 x 1024 takes 17.0 in 4 parts of 128, 17.5 in 2 of 64,
// 28.4 unshared, all with their operands' pass; 4112 x 1024 x 1024 48.5 in pairs
// and 56.4 in single CTAs.  Of 20 problems (1 to 514 rows, 512 to 4096 columns and
// indexes, fp32 and bf16) with every shape timed, the rule takes the fastest or one
// within 3 % in 18; 257 x 1024 x 4096 bf16 takes 14.3 in 5 parts, 13.0 in 4; 1 x 1000
// x 1024 fp32 11.1 in 6 of 64 columns, 10.5 in 8 of 128.
Shape choose(int64_t M, int64_t N, int n_k, int planes) {
    const int sms = sm_count();
    auto rounds = [](int64_t tiles, int units) { return (double)div_up(tiles, units < 1 ? 1 : units); };
    const int64_t rows = div_up(M, GM);
    const bool f32 = planes == 3;
    Shape best = {2, 256, 1};
    double least = 6.0 + (f32 ? 1.75 : 0.30) * n_k * rounds(div_up(M, 2 * GM) * div_up(N, 256), sms / 2);
    auto consider = [&](const Shape &s, double t) {
        if (t < least) {
            least = t;
            best = s;
        }
    };
    consider({1, 128, 1}, 5.0 + (f32 ? 1.2 : 0.24) * n_k * rounds(rows * div_up(N, 128), sms));
    for (int bn = 64; bn <= SPLIT_N; bn *= 2) {
        const int64_t tiles = rows * div_up(N, bn);
        const double step = !f32 ? 0.24 : bn == 64 ? 1.0 : 1.1;
        // each part of a shared tile takes two stages or more
        for (int parts = 2; parts <= MAX_PARTS && 2 * parts <= planes * n_k && parts <= n_k && tiles * parts <= sms;
             ++parts)
            // One cluster fewer than fit: a device full of them, or more, does
            // not pay (257 x 1024 x 1024 fp32 in 24 clusters of 5 CTAs: 18.6, of 6
            // 25.7, of 4 16.9; 257 x 768 x 768 in 18 of 6 15.5, of 4 14.2; 257 x
            // 1024 x 1024 bf16 of 5 12.1, of 4 10.1).
            if (tiles < split_clusters(parts))
                consider({1, bn, parts}, 5.0 + 0.008 * bn + 0.005 * bn * parts + step * (double)div_up(n_k, parts));
    }
    return best;
}

}  // namespace

int launch_gemm(int64_t M, int64_t N, int64_t K, int type16, const GemmOperand &a, const GemmOperand &b,
                const GemmEpilogue &epi, GemmAfter after, const ColumnSums *sums, int32_t *dev_status,
                cudaStream_t stream, int64_t wait_limit) {
    GemmArgs p;
    p.planes = a.planes;
    p.n_k = (int)div_up(K, GK);
    const Shape sh = choose(M, N, p.n_k, p.planes);
    // one accumulation, or chunks of it added in fp32
    const int sum = epi.out_type == SC_F32 ? SUM_F32 : p.n_k > LONG_16 ? SUM_16_LONG : SUM_16;
    p.chunk = sum == SUM_16 && sh.parts == 1 ? p.n_k : CHUNK;
    p.lead = p.chunk == CHUNK && p.planes == 1 && p.n_k > 2 * CHUNK ? CHUNK_LEAD : p.chunk;
    // the two accumulators of fp32 operands: twice where two tiles' fit
    p.rest = p.planes == 1 ? 0 : sh.bn <= ACC_COLS / 2 ? ACC_COLS / 2 : ACC_COLS;
    p.acc_two = p.rest < ACC_COLS;
    p.bn = sh.bn;
    p.M = (int)M;
    p.N = (int)N;
    p.a_mn = !a.k_major;
    p.b_mn = !b.k_major;
    p.n_tiles_n = (int)div_up(N, sh.bn);
    const int64_t tiles = div_up(M, sh.cg * GM) * p.n_tiles_n;
    p.n_tiles_m = (int)div_up(M, sh.cg * GM);
    if (tiles > INT32_MAX / 8) {
        set_error("matrix product: %lld x %lld is too large", (long long)M, (long long)N);
        return SC_ERR_ARG;
    }
    p.n_tiles = (int)tiles;
    p.b_stage = sh.bn / sh.cg * GK * 2;
    p.stages = RING_BYTES / (A_STAGE + p.b_stage);
    // the self-test's copies never bring what their barriers expect
    p.stage_tx = (uint32_t)(sh.cg * (A_STAGE + p.b_stage)) + (wait_limit > 0 ? 16 : 0);
    p.wait_limit = wait_limit > 0 ? wait_limit : WAIT_LIMIT_CYCLES;
    if (p.stages > MAX_RING) p.stages = MAX_RING;
    // D fp32; A and B of type16; majorness; N / 8; M / 16
    const uint32_t f = type16 == SC_BF16 ? 1u : 0u;
    p.idesc = (1u << 4) | (f << 7) | (f << 10) | ((uint32_t)p.a_mn << 15) | ((uint32_t)p.b_mn << 16) |
              ((uint32_t)(sh.bn >> 3) << 17) | ((uint32_t)(sh.cg * GM >> 4) << 24);
    p.bias = epi.bias;
    p.res = epi.res;
    p.out = epi.out;
    p.pre = epi.pre;
    p.ld_out = epi.ld_out;
    p.ld_res = epi.ld_res;
    p.ld_pre = epi.ld_pre;
    p.bias_type = epi.bias_type;
    p.out_type = epi.out_type;
    p.pre_type = epi.pre_type;
    p.vec = N % 8 == 0 && vec_rows(epi.out, epi.ld_out, epi.out_type) &&
            (!epi.res || vec_rows(epi.res, epi.ld_res, epi.out_type)) &&
            (!epi.pre || vec_rows(epi.pre, epi.ld_pre, epi.pre_type)) && aligned16(epi.bias);
    p.sums = sums ? *sums : ColumnSums{};
    p.beside = after == BESIDE_GEMM;
    const bool early = after != AFTER_ANY;
    p.dev_status = dev_status;
    if (!encode(&p.ma, type16, a, M, K, GM) || !encode(&p.mb, type16, b, N, K, sh.bn / sh.cg)) {
        set_error("matrix product: the tensor map was rejected");
        return SC_ERR_CUDA;
    }
    GemmKernels k;
    switch (epi.act) {
        case SC_ACT_RELU: k = gemm_kernels_relu(); break;
        case SC_ACT_GELU: k = gemm_kernels_gelu(); break;
        case SC_ACT_GELU_TANH: k = gemm_kernels_gelu_tanh(); break;
        case SC_ACT_SILU: k = gemm_kernels_silu(); break;
        default: k = gemm_kernels_none(); break;
    }
    if (sh.parts > 1) return launch(k.split, p, p.n_tiles * sh.parts, sh.parts, early, stream);
    const int units = sm_count() / sh.cg;
    const GemmFn kern = (sh.cg == 2 ? k.pair : k.single)[sum];
    if (sum != SUM_16 && !keep_regs_ok(kern)) {
        cudaGetLastError();
        set_error("matrix product: the kernel was built with another number of registers than %d", KEEP_REGS);
        return SC_ERR_CUDA;
    }
    return launch(kern, p, sh.cg * (p.n_tiles < units ? p.n_tiles : units), sh.cg, early, stream);
}

}  // namespace scb
