// sc_gemm.cu -- D(m, n) = sum_k A(m, k) B(n, k) on the 5th-generation tensor
// cores (tcgen05.mma.kind::f16, fp32 accumulators in tensor memory), with the
// linear layer's epilogue.
//
// Operand tiles of 64 contraction indexes (128 bytes, 128-byte swizzle) come
// by TMA into a ring of shared-memory stages; rows and columns past the
// matrices' ends read as zeros.  Either operand may have k or its own index
// contiguous (the shared-memory descriptor covers both), so the forward pass
// (x w^T), dz w and dz^T x run the same kernel without transposing anything.
//
// fp32 operands: x = x1 + x2 + x3 exactly, bf16 parts of 8 bits of
// significand, |x2| <= 2^-8 |x|, |x3| <= 2^-16 |x|.  Of the nine products the
// three below 2^-24 |x w| are left out; the others run as six products over
// the planes, the small ones first.
//
// The tensor cores cut an fp32 sum where fp32 arithmetic rounds, so a long sum
// drifts towards zero by about 2^-25 of itself per 16 indexes.  Where the
// result keeps fp32, an accumulator therefore takes CHUNK stages at most, and
// the epilogue warps add the chunks in registers.
//
// Kernels:
//   gemm_kernel<2>  clusters of two CTAs on two SMs, one cta_group::2 MMA of
//                   256 rows x bn columns; persistent over the tiles, two
//                   accumulators, so a tile's epilogue runs under the next
//                   tile's products
//   gemm_kernel<1>  the same with one CTA and 128 rows
//   gemm_split_kernel  few tiles: a cluster of CTAs shares one tile's
//                   contraction and adds the parts over distributed shared
//                   memory, in rank order
// All waits are bounded, as in the count engine: on expiry the kernel records
// SC_DEV_WAIT_LIMIT, waits for its own copies and products, frees tensor
// memory and returns.
#include <cuda.h>

#include <mutex>

#include "sc_gemm.cuh"
#include "sc_tc_dev.cuh"

namespace scb {
namespace {

using namespace tcd;

constexpr int GK = 64;                  // contraction indexes per stage
constexpr int GM = 128;                 // rows per CTA
constexpr int A_STAGE = GM * GK * 2;    // 16 KB
constexpr int EPI_WARPS = 8;            // two per quadrant of tensor-memory lanes
constexpr int EPI_WARP0 = 4;
constexpr int GEMM_THREADS = (EPI_WARP0 + EPI_WARPS) * 32;
constexpr int RING_BYTES = 160 * 1024;  // 5 stages of 32 KB
constexpr int MAX_RING = 8;
constexpr int CHUNK = 16;               // stages (1024 indexes) per accumulation of an fp32 result
// Epilogue staging, per warp: 32 rows x 64 columns of fp32, 16-byte quads
// permuted so that both a lane's row (written) and 8 lanes' row (read) touch
// every bank once.
constexpr int STG_COLS = 64;
constexpr int STG_BYTES = 32 * STG_COLS * 4;
constexpr int ACC_COLS = 256;           // tensor-memory columns per accumulator buffer
constexpr int GN_MAX = 256;            // columns per tile
constexpr int SPLIT_N = 128;            // columns of a tile whose contraction is shared
constexpr int SPLIT_LD = SPLIT_N + 4;
static_assert(GM * SPLIT_LD * 4 <= RING_BYTES, "parts of a shared tile fit the ring");

struct GemmArgs {
    CUtensorMap ma, mb;
    int64_t ld_out, ld_res, ld_pre;
    const void *bias, *res;
    void *out, *pre;
    int32_t *dev_status;
    int M, N;
    int n_k;            // stages of one product
    int n_prod;         // 1, or 6 for fp32 operands
    int chunk;          // stages per accumulation
    int a_mn, b_mn;     // operand has its own index contiguous
    int bn;             // columns per tile
    int n_tiles_n, n_tiles;
    int stages, b_stage, b_box_rows;
    uint32_t idesc;
    int bias_type, out_type, pre_type, act;
    int vec_out, vec_res, vec_pre, vec_bias;  // 8 columns per access
};

struct GemmSync {
    uint64_t full[MAX_RING], empty[MAX_RING];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort_flag;
};

constexpr int GEMM_SMEM = RING_BYTES + EPI_WARPS * STG_BYTES + 1024 + 512;
static_assert(sizeof(GemmSync) <= 512, "barriers");
static_assert(GEMM_SMEM <= 227 * 1024, "shared memory");

// The parts of fp32 operands that product `i` multiplies, small ones first.
__device__ __forceinline__ int plane_a(int i, int n) { return n == 1 ? 0 : (0x001102 >> (4 * i)) & 15; }
__device__ __forceinline__ int plane_b(int i, int n) { return n == 1 ? 0 : (0x010120 >> (4 * i)) & 15; }

// 128-byte swizzled operand: 8-row groups (k_major: of rows, else of k) 1024
// bytes apart; 64-column blocks of the operand's own index 8192 bytes apart.
__device__ __forceinline__ uint64_t swizzled_desc(uint32_t saddr, bool mn) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(mn ? 8192 >> 4 : 1) << 16) |
           ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

template <int CG>
__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t da, uint64_t db, uint32_t idesc, uint32_t acc) {
    if constexpr (CG == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(da), "l"(db), "r"(idesc), "r"(acc)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(da), "l"(db), "r"(idesc), "r"(acc)
            : "memory");
}

// One box into this CTA's shared memory; CG = 2: its bytes count on the
// barrier of the cluster's first CTA (`bar` is a cluster address).  No
// multicast.
template <int CG>
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1, int c2) {
    if constexpr (CG == 2)
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
            "[%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
            "l"(map), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
            "[%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
            "l"(map), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
            : "memory");
}

__device__ __forceinline__ uint32_t cluster_addr(uint32_t saddr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
    return r;
}

// The operand tile of `rows` rows (a multiple of 64 when the operand's own
// index is contiguous) at row r0, contraction index k0.
template <int CG>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap *map, uint32_t bar, bool mn, int rows,
                                          int r0, int k0, int plane) {
    if (!mn) {
        tma_load<CG>(dst, map, bar, k0, r0, plane);
    } else {
        for (int i = 0; i < rows; i += 64) tma_load<CG>(dst + i * 128, map, bar, r0 + i, k0, plane);
    }
}

// Products of one stage: 4 MMAs of 16 contraction indexes.
template <int CG>
__device__ __forceinline__ void stage_mmas(const GemmArgs &p, uint32_t d, uint32_t sa, bool first) {
    const uint32_t sb = sa + A_STAGE;
    const uint32_t ka = p.a_mn ? 2048u : 32u, kb = p.b_mn ? 2048u : 32u;
#pragma unroll
    for (int k = 0; k < GK / 16; ++k)
        mma_f16_ss<CG>(d, swizzled_desc(sa + k * ka, p.a_mn), swizzled_desc(sb + k * kb, p.b_mn), p.idesc,
                       !(first && k == 0));
}

// 8 columns from `col` (a multiple of 8) of a vector or a row at offset o; n of
// them exist.
__device__ __forceinline__ void load8(const void *p, int type, int64_t o, int n, bool vec, float (&v)[8]) {
    if (vec && n == 8) {
        load_any<8>(p, type, o, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float t[1] = {0.f};
            if (i < n) load_any<1>(p, type, o + i, t);
            v[i] = t[0];
        }
    }
}
__device__ __forceinline__ void store8(void *p, int type, int64_t o, int n, bool vec, const float (&v)[8]) {
    if (vec && n == 8) {
        if (type == SC_F32) store_vec<float, 8>(static_cast<float *>(p) + o, v);
        else if (type == SC_BF16) store_vec<__nv_bfloat16, 8>(static_cast<__nv_bfloat16 *>(p) + o, v);
        else store_vec<__half, 8>(static_cast<__half *>(p) + o, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) store_any(p, type, o + i, v[i]);
    }
}

// Epilogue of columns col .. col + 7 of one row; b: their bias.
__device__ __forceinline__ void epilogue8(const GemmArgs &p, float (&v)[8], const float (&b)[8], int64_t row, int col) {
    const int n = min(8, p.N - col);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += b[i];
    if (p.pre) store8(p.pre, p.pre_type, row * p.ld_pre + col, n, p.vec_pre, v);
    if (p.act != SC_ACT_NONE) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = act_fn(v[i], p.act);
    }
    if (p.res) {
        float r[8];
        load8(p.res, p.out_type, row * p.ld_res + col, n, p.vec_res, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += r[i];
    }
    store8(p.out, p.out_type, row * p.ld_out + col, n, p.vec_out, v);
}

template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t *where) {
    if constexpr (CG == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(where)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(where)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
}
template <int CG>
__device__ __forceinline__ void tmem_free(uint32_t base) {
    if constexpr (CG == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(TMEM_COLS) : "memory");
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(TMEM_COLS) : "memory");
}

// CG CTAs per tile of CG * 128 rows.  SPLIT (CG = 1): the CTAs of a cluster
// each take a share of one tile's contraction.  KEEP: accumulations of p.chunk stages added in registers.
template <int CG, bool SPLIT, bool KEEP>
__global__ void __launch_bounds__(GEMM_THREADS, 1) gemm_kernel(const __grid_constant__ GemmArgs p) {
    static_assert(CG == 1 || !SPLIT, "a shared contraction has one CTA per part");
    static_assert(KEEP || !SPLIT, "parts are added in fp32");
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    uint8_t *ring = smem_raw + (base - smem_addr(smem_raw));
    GemmSync &sy = *reinterpret_cast<GemmSync *>(ring + RING_BYTES + EPI_WARPS * STG_BYTES);
    volatile int *abort_flag = &sy.abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = CG == 2 || SPLIT ? (int)cluster_rank() : 0;
    const int first_tile = CG == 2 || SPLIT ? (int)cluster_id() : (int)blockIdx.x;
    const int tile_step = SPLIT ? p.n_tiles : CG == 2 ? (int)cluster_count() : (int)gridDim.x;
    // this CTA's share of the stages of a tile
    const int n_it = p.n_k * p.n_prod;
    int it0 = 0, it1 = n_it;
    if constexpr (SPLIT) {
        const int parts = (int)gridDim.x / p.n_tiles;
        it0 = (int)((int64_t)n_it * rank / parts);
        it1 = (int)((int64_t)n_it * (rank + 1) / parts);
    }

    if (threadIdx.x == 0) {
        for (int s = 0; s < MAX_RING; ++s) {
            mbar_init(&sy.full[s], 1);
            mbar_init(&sy.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sy.acc_full[b], 1);
            mbar_init(&sy.acc_empty[b], CG * EPI_WARPS);
        }
        mbar_init(&sy.drain, 1);
        sy.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) tmem_alloc<CG>(&sy.tmem_base);
    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync();
    tc_fence_after();
    const uint32_t tmem = sy.tmem_base;
    const int stage_bytes = A_STAGE + p.b_stage;
    auto epilogue = [&]() {
        // ================= epilogue =================
        // Warps e and e + 4 share a quadrant of tensor-memory lanes (32 rows)
        // and take half of the columns each.
        const int e = warp - EPI_WARP0, quad = warp & 3;
        const int half = p.bn / 2, c_lo = (e >> 2) * half;
        float *stg = reinterpret_cast<float *>(ring + RING_BYTES + e * STG_BYTES);
        const int lc = lane & 7, lr = lane >> 3;
        // 64 columns of the warp's rows: through shared memory, so that 8 lanes
        // access one row's 64 columns together
        auto stage_quad = [&](int j, float a, float b, float c, float d) {
            const int at = ((j & 1) * 8 + (j >> 1)) ^ (lane & 7);
            *reinterpret_cast<float4 *>(stg + lane * STG_COLS + at * 4) = make_float4(a, b, c, d);
        };
        auto store_staged = [&](int64_t row0, int col) {
            __syncwarp();
            if (col < p.N) {
                float b[8] = {};
                if (p.bias) load8(p.bias, p.bias_type, col, p.N - col < 8 ? p.N - col : 8, p.vec_bias, b);
#pragma unroll(KEEP ? 2 : 4)
                for (int r = lr; r < 32; r += 4) {
                    if (row0 + r >= p.M) break;
                    float o[8];
                    const float *q = stg + r * STG_COLS;
                    *reinterpret_cast<float4 *>(o) = *reinterpret_cast<const float4 *>(q + (lc ^ (r & 7)) * 4);
                    *reinterpret_cast<float4 *>(o + 4) = *reinterpret_cast<const float4 *>(q + (8 + (lc ^ (r & 7))) * 4);
                    epilogue8(p, o, b, row0 + r, col);
                }
            }
            __syncwarp();
        };
        auto release = [&](int buf) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (CG == 2) mbar_arrive_cluster(&sy.acc_empty[buf], 0);
                else mbar_arrive(&sy.acc_empty[buf]);
            }
        };
        uint32_t n = 0;
        for (int t = first_tile; t < p.n_tiles; t += tile_step) {
            const int64_t row0 = (int64_t)(t / p.n_tiles_n) * (CG * GM) + (CG == 2 ? rank * GM : 0) + quad * 32;
            const int n0 = (t % p.n_tiles_n) * p.bn + c_lo;
            const uint32_t lane_acc = tmem + c_lo + ((uint32_t)(quad * 32) << 16);
            if constexpr (KEEP) {
                // add up the chunks: this lane's row, columns c_lo .. c_lo + half
                constexpr int COLS = SPLIT ? SPLIT_N / 2 : GN_MAX / 2;
                float v[COLS] = {};
                for (int i = it0; i < it1; i += p.chunk, ++n) {
                    const int buf = n & 1;
                    if (!wait_warp(&sy.acc_full[buf], (n >> 1) & 1, abort_flag)) return;
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < COLS; c += 32) {
                        if (c < half) {
                            uint32_t r[32];
                            tmem_ld32(lane_acc + buf * ACC_COLS + c, r);
#pragma unroll
                            for (int j = 0; j < 32; ++j) v[c + j] += __uint_as_float(r[j]);
                        }
                    }
                    release(buf);
                }
                if constexpr (SPLIT) {
                    float *part = reinterpret_cast<float *>(ring) + (quad * 32 + lane) * SPLIT_LD + c_lo;
#pragma unroll
                    for (int c = 0; c < COLS; c += 4)
                        if (c < half)
                            *reinterpret_cast<float4 *>(part + c) = make_float4(v[c], v[c + 1], v[c + 2], v[c + 3]);
                } else {
#pragma unroll
                    for (int c = 0; c < COLS; c += STG_COLS) {
                        if (c >= half) break;
#pragma unroll
                        for (int j = 0; j < STG_COLS / 4; ++j)
                            stage_quad(j, v[c + 4 * j], v[c + 4 * j + 1], v[c + 4 * j + 2], v[c + 4 * j + 3]);
                        store_staged(row0, n0 + c + lc * 8);
                    }
                }
            } else {
                const int buf = n & 1;
                if (!wait_warp(&sy.acc_full[buf], (n >> 1) & 1, abort_flag)) return;
                ++n;
                tc_fence_after();
                for (int c = 0; c < half; c += STG_COLS) {
#pragma unroll
                    for (int k = 0; k < STG_COLS; k += 32) {
                        uint32_t r[32];
                        tmem_ld32(lane_acc + buf * ACC_COLS + c + k, r);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            stage_quad(k / 4 + j, __uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1]),
                                       __uint_as_float(r[4 * j + 2]), __uint_as_float(r[4 * j + 3]));
                    }
                    if (c + STG_COLS >= half) release(buf);
                    store_staged(row0, n0 + c + lc * 8);
                }
            }
        }
    };
    // all products and copies done, no arrival on its way to another CTA
    auto finish = [&]() {
        tc_fence_before();
        __syncthreads();
        if (CG == 2 || SPLIT) cluster_sync();
        tc_fence_after();
        if (warp == 2) tmem_free<CG>(tmem);
        if (threadIdx.x == 0 && sy.abort_flag && p.dev_status) atomicOr(p.dev_status, SC_DEV_WAIT_LIMIT);
    };
    // 128 sums per epilogue thread: those warps take registers over from the
    // other four (launched with 168 each: 56 + 2 x 224 = 3 x 168).  The two
    // sides share no code after this.
    if constexpr (KEEP && !SPLIT) {
        if (warp >= EPI_WARP0) {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
            epilogue();
            finish();
            return;
        }
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    }

    if (warp == 0) {
        // ================= TMA producer =================
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int t = first_tile; t < p.n_tiles && ok; t += tile_step) {
                const int m0 = (t / p.n_tiles_n) * (CG * GM) + rank * GM * (CG - 1);
                const int n0 = (t % p.n_tiles_n) * p.bn + (CG == 2 ? rank * (p.bn / 2) : 0);
                for (int i = it0; i < it1; ++i, ++it) {
                    const int s = (int)(it % p.stages);
                    if (!mbar_wait(&sy.empty[s], ((it / p.stages) & 1) ^ 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                    const uint32_t sa = base + s * stage_bytes;
                    uint32_t bar = smem_addr(&sy.full[s]);
                    if (CG == 2) bar = cluster_addr(bar, 0);
                    if (rank == 0 || CG == 1) mbar_expect_tx(&sy.full[s], CG * stage_bytes);
                    const int prod = i / p.n_k, k0 = (i % p.n_k) * GK;
                    load_tile<CG>(sa, &p.ma, bar, p.a_mn, GM, m0, k0, plane_a(prod, p.n_prod));
                    load_tile<CG>(sa + A_STAGE, &p.mb, bar, p.b_mn, p.bn / CG, n0, k0, plane_b(prod, p.n_prod));
                }
            }
            if (ok) {
                // every stage consumed: no copy and no arrival is in flight
                for (uint32_t j = it > (uint32_t)p.stages ? it - p.stages : 0; j < it; ++j)
                    mbar_wait(&sy.empty[j % p.stages], (j / p.stages) & 1, abort_flag);
            }
            if (*abort_flag && (rank == 0 || CG == 1)) {
                // gave up: let the copies that were issued land
                int dummy = 0;
                for (uint32_t j = it > (uint32_t)p.stages ? it - p.stages : 0; j < it; ++j)
                    mbar_wait(&sy.full[j % p.stages], (j / p.stages) & 1, &dummy, WAIT_LIMIT_CYCLES / 16);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ================= MMA issuer =================
        if (lane == 0 && (CG == 1 || rank == 0)) {
            uint32_t it = 0, n = 0;
            bool ok = true;
            for (int t = first_tile; t < p.n_tiles && ok; t += tile_step) {
                for (int i = it0; i < it1 && ok; ++n) {
                    const int buf = n & 1;
                    if (!mbar_wait(&sy.acc_empty[buf], ((n >> 1) & 1) ^ 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t acc = tmem + buf * ACC_COLS;
                    const int end = min(i + p.chunk, it1);
                    for (bool first = true; i < end; ++i, ++it, first = false) {
                        const int s = (int)(it % p.stages);
                        if (!mbar_wait(&sy.full[s], (it / p.stages) & 1, abort_flag)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        stage_mmas<CG>(p, acc, base + s * stage_bytes, first);
                        mma_commit<CG>(&sy.empty[s]);
                    }
                    if (ok) mma_commit<CG>(&sy.acc_full[buf]);
                }
            }
            if (*abort_flag) {  // gave up: let the products that were issued finish
                int dummy = 0;
                mma_commit<1>(&sy.drain);
                mbar_wait(&sy.drain, 0, &dummy, WAIT_LIMIT_CYCLES / 16);
            }
        }
        __syncwarp();
    } else if ((SPLIT || !KEEP) && warp >= EPI_WARP0) {
        epilogue();
    }

    if constexpr (SPLIT) {
        // every part is in its CTA's shared memory: add them up, a share of
        // the rows each
        __syncthreads();
        cluster_sync();
        const int parts = (int)gridDim.x / p.n_tiles;
        const int m0 = (first_tile / p.n_tiles_n) * GM, n0 = (first_tile % p.n_tiles_n) * p.bn;
        const int groups = p.bn / 8;
        if (!*abort_flag) {
            const int r0 = GM * rank / parts, r1 = GM * (rank + 1) / parts;
            for (int i = threadIdx.x; i < (r1 - r0) * groups; i += GEMM_THREADS) {
                const int r = r0 + i / groups, c = (i % groups) * 8;
                if (m0 + r >= p.M || n0 + c >= p.N) continue;
                float v[8] = {};
                const uint32_t mine = base + (uint32_t)(r * SPLIT_LD + c) * 4;
                for (int q = 0; q < parts; ++q) {
                    const uint32_t at = cluster_addr(mine, q);
                    float a[8];
                    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                 : "=f"(a[0]), "=f"(a[1]), "=f"(a[2]), "=f"(a[3])
                                 : "r"(at));
                    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                 : "=f"(a[4]), "=f"(a[5]), "=f"(a[6]), "=f"(a[7])
                                 : "r"(at + 16));
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] += a[j];
                }
                float b[8] = {};
                if (p.bias) load8(p.bias, p.bias_type, n0 + c, p.N - n0 - c < 8 ? p.N - n0 - c : 8, p.vec_bias, b);
                epilogue8(p, v, b, m0 + r, n0 + c);
            }
        }
        __syncwarp();
    }
    finish();
}

// ---- host -------------------------------------------------------------------
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

template <typename K>
int launch(K kern, const GemmArgs &p, int grid, int cluster, cudaStream_t stream) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, GEMM_SMEM);
    if (e != cudaSuccess) return cuda_fail(e, "matrix product: smem attribute");
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(GEMM_THREADS);
    cfg.dynamicSmemBytes = GEMM_SMEM;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, kern, p);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? SC_OK : cuda_fail(e, "matrix product");
}

struct Shape {
    int cg, bn, parts;
};

// Tile shape: 256 x 256 by CTA pairs when that fills the SMs, else 128-row
// tiles, else tiles whose contraction several CTAs share.
Shape choose(int64_t M, int64_t N, int n_it) {
    const int sms = sm_count();
    const int64_t t2 = div_up(M, 256) * div_up(N, 256);
    if (2 * t2 >= sms) return {2, 256, 1};
    const int64_t t1 = div_up(M, 128) * div_up(N, 128);
    int parts = 1;
    while (parts < 8 && t1 * parts * 2 <= sms && n_it >= 4 * parts) parts *= 2;
    return {1, 128, parts};
}

}  // namespace

int launch_gemm(int64_t M, int64_t N, int64_t K, int type16, const GemmOperand &a, const GemmOperand &b,
                const GemmEpilogue &epi, int32_t *dev_status, cudaStream_t stream) {
    GemmArgs p;
    p.n_prod = a.planes == 3 ? 6 : 1;
    p.n_k = (int)div_up(K, GK);
    const Shape sh = choose(M, N, p.n_k * p.n_prod);
    p.chunk = epi.out_type == SC_F32 ? CHUNK : p.n_k * p.n_prod;
    p.bn = sh.bn;
    p.M = (int)M;
    p.N = (int)N;
    p.a_mn = !a.k_major;
    p.b_mn = !b.k_major;
    p.n_tiles_n = (int)div_up(N, sh.bn);
    const int64_t tiles = div_up(M, sh.cg * GM) * p.n_tiles_n;
    if (tiles > INT32_MAX / 8) {
        set_error("matrix product: %lld x %lld is too large", (long long)M, (long long)N);
        return SC_ERR_ARG;
    }
    p.n_tiles = (int)tiles;
    p.b_stage = sh.bn / sh.cg * GK * 2;
    p.stages = RING_BYTES / (A_STAGE + p.b_stage);
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
    p.act = epi.act;
    p.vec_out = vec_rows(epi.out, epi.ld_out, epi.out_type);
    p.vec_res = vec_rows(epi.res, epi.ld_res, epi.out_type);
    p.vec_pre = vec_rows(epi.pre, epi.ld_pre, epi.pre_type);
    p.vec_bias = aligned16(epi.bias);
    p.dev_status = dev_status;
    if (!encode(&p.ma, type16, a, M, K, GM) || !encode(&p.mb, type16, b, N, K, sh.bn / sh.cg)) {
        set_error("matrix product: the tensor map was rejected");
        return SC_ERR_CUDA;
    }
    if (sh.parts > 1) return launch(gemm_kernel<1, true, true>, p, p.n_tiles * sh.parts, sh.parts, stream);
    const int sms = sm_count();
    const bool keep = epi.out_type == SC_F32;
    if (sh.cg == 2) {
        const int pairs = p.n_tiles < sms / 2 ? p.n_tiles : sms / 2;
        return launch(keep ? gemm_kernel<2, false, true> : gemm_kernel<2, false, false>, p, 2 * pairs, 2, stream);
    }
    return launch(keep ? gemm_kernel<1, false, true> : gemm_kernel<1, false, false>, p,
                  p.n_tiles < sms ? p.n_tiles : sms, 1, stream);
}

}  // namespace scb
