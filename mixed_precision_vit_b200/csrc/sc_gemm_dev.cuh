// sc_gemm_dev.cuh -- the kernels of sc_gemm.cu: D(m, n) = sum_k A(m, k) B(n, k)
// on the 5th-generation tensor cores (tcgen05.mma.kind::f16, fp32 accumulators in
// tensor memory), with the linear layer's epilogue.
//
// Operand tiles of 64 contraction indexes (128 bytes, 128-byte swizzle) come
// by TMA into a ring of shared-memory stages; rows and columns past the
// matrices' ends read as zeros.  Either operand may have k or its own index
// contiguous (the shared-memory descriptor covers both), so the forward pass
// (x w^T), dz w and dz^T x run the same kernel without transposing anything.
//
// fp32 operands: x = x1 + x2 + x3 exactly, bf16 parts of 8 bits of
// significand, |x2| <= 2^-8 |x|, |x3| <= 2^-16 |x|.  Of the nine products the
// three below 2^-24 |x w| are left out.  The same part of both operands makes a
// stage, and the other six products run as their stages arrive, so that 64
// indexes take three stages.  (257 x 1024 x 1024 with its pass takes 17.1 us, 2056
// x 1024 x 1024 32; as six products over the parts one after the other, 19.4 and
// 38; with the six operand tiles as stages of their own 21.7 and 38: every stage
// costs the issuing threads its waits.)
//
// The tensor cores cut an fp32 sum where fp32 arithmetic rounds, so a long sum
// drifts towards zero by about 2^-25 of itself per 16 indexes.  Where the
// result keeps fp32, an accumulator therefore takes CHUNK steps at most, and
// the epilogue warps add the chunks in registers.  The first two of a tile, all
// that can run under the stores of the tile before, take CHUNK_LEAD where more
// follow.  (32896 x 1024 x 4096 with an fp32 residual: off by 5.8e-7 of the
// result's norm in 233 us; 4.7e-7 in 239 with 8 throughout, 9.9e-7 in 228 with 16,
// 4.0e-6 in one accumulation; a plain fp32 product is off by 6.1e-7.)  A 16-bit result's rounding hides the
// drift of LONG_16 steps (2^-15, half a step of fp16 is 2^-11); longer sums
// are added up in chunks too (2048 x 2048 x 16384 in one accumulation 90.8 us,
// 2048 x 2048 x 16448 in chunks 93.1).  fp32 operands keep the five small
// products, below 2^-8 of the result, in an accumulator of their own, so that
// only the leading product's drift counts, in chunks of CHUNK throughout (off by
// 4.7e-7 where 16 are off by 1.0e-6; 4112 x 4096 x 1024 takes 157 us, 154 with 16; a plain fp32 product
// is off by 5.7e-7).
//
// Kernels (one template):
//   CG = 2  clusters of two CTAs on two SMs, one cta_group::2 MMA of 256 rows x
//           256 columns, so that each SM stages half of the columns' operand;
//           persistent over the tiles, two accumulators, so that a tile's
//           epilogue runs under the next tile's products
//   CG = 1  the same with one CTA and 128 rows x 128 columns
//   SPLIT   few tiles: a cluster of CTAs shares one tile's contraction and adds
//           the parts over distributed shared memory, in rank order
// Warp 0 issues the copies, warp 1 the products, warp 3 finishes column sums of
// an earlier pass if the caller has any, warps 4 to 11 are the epilogue.
//
// Measured (us, one B200, a replayed graph over two or three sets of inputs after a
// second's rest): 8192^3 bf16 694 (cuBLAS 657); 4112 x 4096 x 1024 30 plain
// (cuBLAS 30), 40 with gelu and the pre-activation kept, where the epilogue sets
// the pace (tensor pipe 51 % busy); 32896 x 1024 x 4096 179 (cuBLAS 181), 197 with
// an fp32 result, 220 with a residual beside it (tensor pipe 74 %).  Products that
// run for longer meet the power limit: the last one takes 266 us replayed and 272
// called for 1.5 s, at 1250 and 1240 MHz.
// All waits are bounded, as in the count engine.  A CTA (a pair, a cluster that
// shares a tile) whose wait expires waits for its own copies and products,
// writes NaN over its tiles, records SC_DEV_WAIT_LIMIT, frees tensor memory and
// returns.
#pragma once
#include <cuda.h>

#include "sc_gemm.cuh"
#include "sc_tc_dev.cuh"

namespace scb {
namespace gemm {

using namespace tcd;

constexpr int GK = 64;                  // contraction indexes per stage
constexpr int GM = 128;                 // rows per CTA
constexpr int A_STAGE = GM * GK * 2;    // 16 KB
constexpr int EPI_WARPS = 8;            // two per quadrant of tensor-memory lanes
constexpr int EPI_WARP0 = 4;
constexpr int GEMM_THREADS = (EPI_WARP0 + EPI_WARPS) * 32;
constexpr int KEEP_REGS = 168;          // registers per thread of a kernel that keeps sums
constexpr int RING_BYTES = 160 * 1024;  // 5 stages of 32 KB
constexpr int MAX_RING = 8;
constexpr int CHUNK = 8;                // steps (512 indexes) per accumulation of an fp32 result
constexpr int CHUNK_LEAD = 12;          // the first two of a tile of more, 16-bit operands
constexpr int LONG_16 = 256;            // most steps of a 16-bit result in one accumulation
// Epilogue staging, per warp: 32 rows x 64 columns of fp32, 16-byte quads
// permuted so that both a lane's row (written) and 8 lanes' row (read) touch
// every bank once.
constexpr int STG_COLS = 64;
// Rows on no 16-byte boundary are staged plainly instead, RAGGED_LD floats to a
// row.
constexpr int RAGGED_LD = STG_COLS + 1;
constexpr int STG_BYTES = 32 * RAGGED_LD * 4;
constexpr int ACC_COLS = 256;           // tensor-memory columns per accumulator buffer
constexpr int GN_MAX = 256;             // columns per tile
constexpr int SPLIT_N = 128;            // columns of a tile whose contraction is shared
constexpr int SPLIT_LD = SPLIT_N + 4;
constexpr int MAX_PARTS = 8;            // the portable cluster size
static_assert(GM * SPLIT_LD * 4 <= RING_BYTES, "parts of a shared tile fit the ring");

struct GemmArgs {
    CUtensorMap ma, mb;
    int64_t ld_out, ld_res, ld_pre;
    const void *bias, *res;
    void *out, *pre;
    int32_t *dev_status;
    int M, N;
    int n_k;            // steps of 64 contraction indexes
    int planes;         // stages per step: 1, or 3 for fp32 operands
    int chunk;          // steps per accumulation,
    int lead;           // of the first two of a tile
    int acc_two;        // 1: two accumulations fit tensor memory, 0: one
    int rest;           // columns from the leading parts' accumulator to the others', fp32 operands
    int a_mn, b_mn;     // operand has its own index contiguous
    int bn;             // columns per tile
    int n_tiles_m, n_tiles_n, n_tiles;
    int stages, b_stage;
    int beside;         // BESIDE_GEMM
    ColumnSums sums;    // part null: none
    uint32_t idesc;
    uint32_t stage_tx;  // bytes that a stage's copies bring, both CTAs' of a pair
    long long wait_limit;
    int bias_type, out_type, pre_type;
    int vec;            // 8 columns per access everywhere
};

struct GemmSync {
    uint64_t full[MAX_RING], empty[MAX_RING];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort_flag;
    uint32_t issued;                   // stages that this CTA's copies were issued for
    uint32_t peer_issued, peer_abort;  // the same of a pair's other CTA, and whether it gave up
};

constexpr int GEMM_SMEM = RING_BYTES + EPI_WARPS * STG_BYTES + 1024 + 512;
static_assert(sizeof(GemmSync) <= 512, "barriers");
static_assert(GEMM_SMEM <= 227 * 1024, "shared memory");

// A slot of the ring of stages and the parity of its current use.
struct Ring {
    int slot;
    uint32_t phase;
    __device__ __forceinline__ void next(int stages) {
        if (++slot == stages) {
            slot = 0;
            phase ^= 1;
        }
    }
    __device__ __forceinline__ void back(int n, int stages) {  // n <= stages
        slot -= n;
        if (slot < 0) {
            slot += stages;
            phase ^= 1;
        }
    }
};

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

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ uint32_t cluster_addr(uint32_t saddr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
    return r;
}

__device__ __forceinline__ void store_cluster(const void *where, uint32_t rank, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr(smem_addr(where), rank)), "r"(v) : "memory");
}
// Takes n bytes off what a barrier still expects.
__device__ __forceinline__ void mbar_complete_tx(uint64_t *bar, uint32_t n) {
    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(n) : "memory");
}

// Row and column of tile t.  Tiles run down GROUP_M row tiles before the next
// column, so that the tiles in work at one time share few rows and columns of
// the operands (they stay in L2 where a whole operand does not).
constexpr int GROUP_M = 16;
__device__ __forceinline__ void tile_at(const GemmArgs &p, int t, int &tm, int &tn) {
    const int per = GROUP_M * p.n_tiles_n, g = t / per, r = t - g * per;
    const int rows = min(GROUP_M, p.n_tiles_m - g * GROUP_M);
    tn = r / rows;
    tm = g * GROUP_M + (r - tn * rows);
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

// Products of A of the stage at sa and B of the stage at sb: 4 MMAs of 16
// contraction indexes.  da, db: the descriptors of a stage at address 0; ka, kb:
// their steps.
template <int CG>
__device__ __forceinline__ void stage_mmas(uint32_t d, uint64_t da, uint64_t db, uint32_t ka, uint32_t kb,
                                           uint32_t idesc, uint32_t sa, uint32_t sb, bool first) {
    // the offsets alone: in a cluster the addresses also hold the CTA's rank
    da += (sa & 0x3FFFFu) >> 4;
    db += ((sb + A_STAGE) & 0x3FFFFu) >> 4;
#pragma unroll
    for (int k = 0; k < GK / 16; ++k) mma_f16_ss<CG>(d, da + k * ka, db + k * kb, idesc, !(first && k == 0));
}

// Epilogue of one element.
template <int ACT>
__device__ __forceinline__ void epilogue1(const GemmArgs &p, float z, float bias, int64_t row, int col) {
    float v[1] = {z + bias};
    if (p.pre) store_any(p.pre, p.pre_type, row * p.ld_pre + col, v[0]);
    v[0] = act_fn<ACT>(v[0]);
    if (p.res) {
        float r[1];
        load_any<1>(p.res, p.out_type, row * p.ld_res + col, r);
        v[0] += r[0];
    }
    store_any(p.out, p.out_type, row * p.ld_out + col, v[0]);
}

// 8 columns of R rows, `step` elements apart, from p on.
template <typename T, int R>
__device__ __forceinline__ void store_rows(void *p, int64_t step, const bool (&in)[R], const float (&v)[R][8]) {
    T *q = static_cast<T *>(p);
#pragma unroll
    for (int r = 0; r < R; ++r, q += step)
        if (in[r]) store_vec<T, 8>(q, v[r]);
}
template <int R>
__device__ __forceinline__ void store_rows_any(void *p, int type, int64_t step, const bool (&in)[R],
                                               const float (&v)[R][8]) {
    if (type == SC_F32) store_rows<float, R>(p, step, in, v);
    else if (type == SC_BF16) store_rows<__nv_bfloat16, R>(p, step, in, v);
    else store_rows<__half, R>(p, step, in, v);
}
__device__ __forceinline__ char *at_element(const void *p, int type, int64_t i) {
    return const_cast<char *>(static_cast<const char *>(p)) + i * (type == SC_F32 ? 4 : 2);
}

// Where a lane's 8 columns of a row lie in the result, and the bytes and
// elements from there to its next rows.
struct RowPtrs {
    char *out, *pre;
    const char *res;
};
__device__ __forceinline__ RowPtrs row_ptrs(const GemmArgs &p, int64_t row, int col) {
    return {at_element(p.out, p.out_type, row * p.ld_out + col), at_element(p.pre, p.pre_type, row * p.ld_pre + col),
            at_element(p.res, p.out_type, row * p.ld_res + col)};
}

// What a kernel knows of the result's type.
enum { OUT_ANY, OUT_F32, OUT_16 };
template <int OUT>
__device__ __forceinline__ bool out_f32(const GemmArgs &p) {
    return OUT == OUT_F32 || (OUT == OUT_ANY && p.out_type == SC_F32);
}

// R rows' 8 columns of the residual, as it lies in memory: loaded ahead of
// their use without taking more registers than bytes.
template <int R, int OUT>
struct Residual {
    static constexpr int Q = OUT == OUT_16 ? 1 : 2;
    uint4 w[R][Q];
    __device__ __forceinline__ void load(const GemmArgs &p, const char *q, int64_t step_bytes, const bool (&in)[R]) {
#pragma unroll
        for (int r = 0; r < R; ++r, q += step_bytes)
            if (in[r]) {
                w[r][0] = reinterpret_cast<const uint4 *>(q)[0];
                if (Q == 2 && out_f32<OUT>(p)) w[r][Q - 1] = reinterpret_cast<const uint4 *>(q)[1];
            }
    }
    template <typename T>
    __device__ __forceinline__ void add(float (&v)[R][8]) const {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint4 l = w[r][0], h = w[r][Q - 1];
            const uint32_t k[8] = {l.x, l.y, l.z, l.w, h.x, h.y, h.z, h.w};
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                float x, y;
                if constexpr (sizeof(T) == 4) {
                    x = __uint_as_float(k[i]);
                    y = __uint_as_float(k[i + 1]);
                } else {
                    unpack2<T>(k[i / 2], x, y);
                }
                const float2 z = add2(make_float2(v[r][i], v[r][i + 1]), make_float2(x, y));
                v[r][i] = z.x;
                v[r][i + 1] = z.y;
            }
        }
    }
    __device__ __forceinline__ void add_to(const GemmArgs &p, float (&v)[R][8]) const {
        if (Q == 2 && out_f32<OUT>(p)) add<float>(v);
        else if (p.out_type == SC_BF16) add<__nv_bfloat16>(v);
        else add<__half>(v);
    }
};

// Epilogue of 8 columns (their bias: b) of R rows from q on, `step` rows apart;
// in: the row exists; a: their residual.  Every step runs over all of them
// before the next one begins: the few warps of an epilogue hide latency by
// independent work, not by each other.
template <int ACT, int OUT, int R>
__device__ __forceinline__ void epilogue_rows(const GemmArgs &p, float (&v)[R][8], const float (&b)[8],
                                              const Residual<R, OUT> &a, const RowPtrs &q, int step, const bool (&in)[R]) {
    if (p.bias) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float2 z = add2(make_float2(v[r][i], v[r][i + 1]), make_float2(b[i], b[i + 1]));
                v[r][i] = z.x;
                v[r][i + 1] = z.y;
            }
    }
    if (p.pre) store_rows_any<R>(q.pre, p.pre_type, step * p.ld_pre, in, v);
    if constexpr (ACT != SC_ACT_NONE) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                if constexpr (ACT == SC_ACT_GELU) {
                    const float2 g = gelu2(make_float2(v[r][i], v[r][i + 1]));
                    v[r][i] = g.x;
                    v[r][i + 1] = g.y;
                } else {
                    v[r][i] = act_fn<ACT>(v[r][i]);
                    v[r][i + 1] = act_fn<ACT>(v[r][i + 1]);
                }
            }
    }
    if (p.res) a.add_to(p, v);
    if (out_f32<OUT>(p)) store_rows<float, R>(q.out, step * p.ld_out, in, v);
    else if (p.out_type == SC_BF16) store_rows<__nv_bfloat16, R>(q.out, step * p.ld_out, in, v);
    else store_rows<__half, R>(q.out, step * p.ld_out, in, v);
}

// 8 elements from q on: one access where they lie on a 16-byte boundary, else
// one each.
template <typename T>
__device__ __forceinline__ void load8_any(const void *q, float (&v)[8]) {
    const T *t = static_cast<const T *>(q);
    if ((reinterpret_cast<uintptr_t>(t) & 15) == 0) {
        load_vec<T, 8>(t, v);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = to_f(t[e]);
    }
}
template <typename T>
__device__ __forceinline__ void store8_any(void *q, const float (&v)[8]) {
    T *t = static_cast<T *>(q);
    if ((reinterpret_cast<uintptr_t>(t) & 15) == 0) {
        store_vec<T, 8>(t, v);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = from_f<T>(v[e]);
    }
}

// Elements lo .. hi - 1 of a 16-byte window of a 16-bit matrix, in the largest
// pieces that fit: the L2 takes one store per piece, and those bound rows on no
// boundary.
template <typename T>
__device__ __forceinline__ void store_run(T *window, const uint32_t (&w)[4], int lo, int hi) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (lo <= 4 * h && hi >= 4 * h + 4) {
            *reinterpret_cast<uint2 *>(window + 4 * h) = make_uint2(w[2 * h], w[2 * h + 1]);
            continue;
        }
#pragma unroll
        for (int k = 2 * h; k < 2 * h + 2; ++k) {
            if (lo <= 2 * k && hi >= 2 * k + 2) {
                *reinterpret_cast<uint32_t *>(window + 2 * k) = w[k];
            } else {
                if (lo <= 2 * k && hi > 2 * k) *reinterpret_cast<uint16_t *>(window + 2 * k) = (uint16_t)w[k];
                if (lo <= 2 * k + 1 && hi > 2 * k + 1) *reinterpret_cast<uint16_t *>(window + 2 * k + 1) = (uint16_t)(w[k] >> 16);
            }
        }
    }
}
// A row's first `head` and last 8 - head columns of 64: v[i] belongs into the
// last ones' window for i < 8 - head, else into the first ones'.
template <typename T>
__device__ __forceinline__ void store_ends(void *row, int head, const float (&v)[8]) {
    T *t = static_cast<T *>(row);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
    store_run(t + 56 + head, w, 0, 8 - head);
    store_run(t + head - 8, w, 8 - head, 8);
}

// The same columns' values, in the order of store_ends, by one access for each
// window that lies in the row: from column -8 on if `before`, up to column 71 if
// `after`; else one by one.  Elements outside the 64 columns are not used.
template <typename T>
__device__ __forceinline__ void load_ends(const void *row, int head, bool before, bool after, float (&v)[8]) {
    const T *t = static_cast<const T *>(row);
    float a[8], b[8];
    if (after) {
        load_vec<T, 8>(t + 56 + head, a);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = i < 8 - head ? to_f(t[56 + head + i]) : 0.f;
    }
    if (before) {
        load_vec<T, 8>(t + head - 8, b);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) b[i] = i >= 8 - head ? to_f(t[i - 8 + head]) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < 8 - head ? a[i] : b[i];
}

// Epilogue of 32 rows x 64 columns whose rows start on no 16-byte boundary.  In
// each row, pieces of 8 columns from its first boundary on take the accesses of
// the aligned case (pre and res as well where they lie alike, as they do in
// equal strides); then each lane finishes one row's up to 14 other elements.
// The staged values already hold the bias, RAGGED_LD floats to a row.
template <int ACT, int OUT>
__device__ __forceinline__ void epilogue_ragged(const GemmArgs &p, const float *stg, int64_t row0, int col0, int lane) {
    constexpr int R = 4;  // rows of a lane at a time
    const int width = min(64, p.N - col0), lc = lane & 7, lr = lane >> 3;
    if (width <= 0) return;
    const int rows = (int)min((int64_t)32, p.M - row0);
    // columns before the row's first 16-byte boundary
    auto head_of = [&](int r) {
        const uintptr_t o = reinterpret_cast<uintptr_t>(at_element(p.out, p.out_type, (row0 + r) * p.ld_out + col0));
        return (int)((0 - o) & 15) >> (out_f32<OUT>(p) ? 2 : 1);
    };
    // a whole row of 16-bit results has none or 8 other elements: its last
    // 8 - head columns and its first head ones
    const bool ends = !out_f32<OUT>(p) && width == 64;
    const int my_head = lane < rows ? min(head_of(lane), width) : 0;
#pragma unroll 1
    for (int r0 = lr; r0 < rows; r0 += 4 * R) {
        float v[R][8], a[R][8];
        int c[R];
        bool in[R];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int r = r0 + 4 * k;
            c[k] = head_of(r) + 8 * lc;
            in[k] = r < rows && c[k] + 8 <= width;
            if (p.res && in[k]) {
                const char *q = at_element(p.res, p.out_type, (row0 + r) * p.ld_res + col0 + c[k]);
                if (out_f32<OUT>(p)) load8_any<float>(q, a[k]);
                else if (p.out_type == SC_BF16) load8_any<__nv_bfloat16>(q, a[k]);
                else load8_any<__half>(q, a[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const float *s = stg + (r0 + 4 * k) * RAGGED_LD + c[k];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[k][e] = in[k] ? s[e] : 0.f;
        }
        if (p.pre) {
#pragma unroll
            for (int k = 0; k < R; ++k)
                if (in[k]) {
                    char *q = at_element(p.pre, p.pre_type, (row0 + r0 + 4 * k) * p.ld_pre + col0 + c[k]);
                    if (p.pre_type == SC_F32) store8_any<float>(q, v[k]);
                    else if (p.pre_type == SC_BF16) store8_any<__nv_bfloat16>(q, v[k]);
                    else store8_any<__half>(q, v[k]);
                }
        }
#pragma unroll
        for (int k = 0; k < R; ++k) {
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                if constexpr (ACT == SC_ACT_GELU) {
                    const float2 g = gelu2(make_float2(v[k][e], v[k][e + 1]));
                    v[k][e] = g.x;
                    v[k][e + 1] = g.y;
                } else {
                    v[k][e] = act_fn<ACT>(v[k][e]);
                    v[k][e + 1] = act_fn<ACT>(v[k][e + 1]);
                }
            }
            if (p.res && in[k]) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[k][e] += a[k][e];
            }
        }
#pragma unroll
        for (int k = 0; k < R; ++k)
            if (in[k]) {
                char *o = at_element(p.out, p.out_type, (row0 + r0 + 4 * k) * p.ld_out + col0 + c[k]);
                if (out_f32<OUT>(p)) store_vec<float, 8>(reinterpret_cast<float *>(o), v[k]);
                else if (p.out_type == SC_BF16) store_vec<__nv_bfloat16, 8>(reinterpret_cast<__nv_bfloat16 *>(o), v[k]);
                else store_vec<__half, 8>(reinterpret_cast<__half *>(o), v[k]);
            }
    }
    if (lane < rows) {
        const int head = my_head, tail = head + (width - head) / 8 * 8;
        const int n = head + width - tail;
        const int64_t row = row0 + lane;
        if (ends) {
            if (head == 0) return;
            float v[8], a[8];
            const char *res = at_element(p.res, p.out_type, row * p.ld_res + col0);
            char *pre = at_element(p.pre, p.pre_type, row * p.ld_pre + col0);
            char *out = at_element(p.out, p.out_type, row * p.ld_out + col0);
            if (p.res && ((reinterpret_cast<uintptr_t>(res) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0) {
                const bool before = col0 > 0, after = col0 + 64 + head <= p.N;
                if (p.out_type == SC_BF16) load_ends<__nv_bfloat16>(res, head, before, after, a);
                else load_ends<__half>(res, head, before, after, a);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float t[1] = {0.f};
                    if (p.res) load_any<1>(res, p.out_type, i < 8 - head ? 56 + head + i : i - 8 + head, t);
                    a[i] = t[0];
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = stg[lane * RAGGED_LD + (i < 8 - head ? 56 + head + i : i - 8 + head)];
            if (p.pre) {
                if (((reinterpret_cast<uintptr_t>(pre) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0 && p.pre_type != SC_F32) {
                    if (p.pre_type == SC_BF16) store_ends<__nv_bfloat16>(pre, head, v);
                    else store_ends<__half>(pre, head, v);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) store_any(pre, p.pre_type, i < 8 - head ? 56 + head + i : i - 8 + head, v[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = act_fn<ACT>(v[i]) + a[i];
            if (p.out_type == SC_BF16) store_ends<__nv_bfloat16>(out, head, v);
            else store_ends<__half>(out, head, v);
            return;
        }
#pragma unroll 1
        for (int i0 = 0; i0 < n; i0 += 8) {
            float v[8], a[8];
            int c[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = min(i0 + e, n - 1);  // the last one again where none is left
                c[e] = i < head ? i : tail + i - head;
                v[e] = stg[lane * RAGGED_LD + c[e]];
                float t[1] = {0.f};
                if (p.res) load_any<1>(p.res, p.out_type, row * p.ld_res + col0 + c[e], t);
                a[e] = t[0];
            }
            if (p.pre) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (i0 + e < n) store_any(p.pre, p.pre_type, row * p.ld_pre + col0 + c[e], v[e]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (i0 + e < n) store_any(p.out, p.out_type, row * p.ld_out + col0 + c[e], act_fn<ACT>(v[e]) + a[e]);
        }
    }
}

// tcgen05.ld without its wait; the registers are valid after tmem_wait_ld.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
          "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]),
          "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]),
          "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&v)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(v[i]));  // no use before the wait
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
// each take a share of one tile's contraction.  KEEP: the epilogue adds up
// accumulations of p.chunk steps in registers (fp32 results, parts, long sums).
// (OUT_ANY for the last two: 32896 x 1024 x 4096 with an fp32 residual and
// result 273 -> 286 us.)
template <int CG, bool SPLIT, bool KEEP, int OUT, int ACT>
__global__ void __launch_bounds__(GEMM_THREADS, 1) gemm_kernel(const __grid_constant__ GemmArgs p) {
    static_assert(CG == 1 || !SPLIT, "a shared contraction has one CTA per part");
    static_assert(KEEP ? SPLIT == (OUT == OUT_ANY) : OUT == OUT_16 && !SPLIT, "parts and fp32 results are added in fp32");
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    uint8_t *ring = smem_raw + (base - smem_addr(smem_raw));
    GemmSync &sy = *reinterpret_cast<GemmSync *>(ring + RING_BYTES + EPI_WARPS * STG_BYTES);
    volatile int *abort_flag = &sy.abort_flag;
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = CG == 2 || SPLIT ? (int)cluster_rank() : 0;
    const int first_tile = CG == 2 || SPLIT ? (int)cluster_id() : (int)blockIdx.x;
    const int tile_step = SPLIT ? p.n_tiles : CG == 2 ? (int)cluster_count() : (int)gridDim.x;
    // this CTA's share of the steps of a tile
    int it0 = 0, it1 = p.n_k;
    if constexpr (SPLIT) {
        const int parts = (int)gridDim.x / p.n_tiles;
        it0 = (int)((int64_t)p.n_k * rank / parts);
        it1 = (int)((int64_t)p.n_k * (rank + 1) / parts);
    }
    // the end of the accumulation that begins at step i
    auto chunk_end = [&](int i) { return min(i + (!SPLIT && i < 2 * p.lead ? p.lead : p.chunk), it1); };

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
        sy.issued = sy.peer_issued = sy.peer_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) tmem_alloc<CG>(&sy.tmem_base);
    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync();
    tc_fence_after();
    const uint32_t tmem = sy.tmem_base;
    // Nothing above touches the operands.  A product beside another one needs
    // no wait here: that one has begun, so the passes before it are done.
    if (!p.beside) asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int stage_bytes = A_STAGE + p.b_stage;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, p.wait_limit));
    };
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
        float ragged_bias[2] = {0.f, 0.f};  // of columns lane and lane + 32 of the 64 to be staged
        auto load_ragged_bias = [&](int col0) {
            if (p.vec || !p.bias) return;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float t[1] = {0.f};
                if (col0 + lane + 32 * k < p.N) load_any<1>(p.bias, p.bias_type, col0 + lane + 32 * k, t);
                ragged_bias[k] = t[0];
            }
        };
        // the lane's row of 64 columns, value(i) each
        auto stage = [&](auto value) {
            if (p.vec) {
#pragma unroll
                for (int j = 0; j < STG_COLS / 4; ++j) {
                    const int at = ((j & 1) * 8 + (j >> 1)) ^ (lane & 7);
                    *reinterpret_cast<float4 *>(stg + lane * STG_COLS + at * 4) =
                        make_float4(value(4 * j), value(4 * j + 1), value(4 * j + 2), value(4 * j + 3));
                }
            } else {
#pragma unroll
                for (int i = 0; i < STG_COLS; ++i)
                    stg[lane * RAGGED_LD + i] = value(i) + __shfl_sync(0xffffffffu, ragged_bias[i >> 5], i & 31);
            }
        };
        constexpr int R = 4;  // rows of a lane at a time: lr + 4 k
        // 16-bit residuals are loaded one step ahead; fp32 ones (and the sums
        // beside them) would take too many registers
        constexpr bool AHEAD = !KEEP;
        Residual<R, OUT> ahead;
        const int64_t res_row = p.ld_res * (p.out_type == SC_F32 ? 4 : 2);
        auto rows_in = [&](int64_t row, bool (&in)[R]) {
#pragma unroll
            for (int k = 0; k < R; ++k) in[k] = row + 4 * k < p.M;
        };
        // the residual of the lane's first rows of the 64 columns from col0 on
        auto fetch_first = [&](int64_t row0, int col0) {
            if (AHEAD && p.vec && p.res && col0 + lc * 8 < p.N) {
                bool in[R];
                rows_in(row0 + lr, in);
                ahead.load(p, row_ptrs(p, row0 + lr, col0 + lc * 8).res, 4 * res_row, in);
            }
        };
        // more: another 64 columns follow
        auto store_staged = [&](int64_t row0, int col0, const float (&b)[8], bool more) {
            __syncwarp();
            if (p.vec) {
                const int col = col0 + lc * 8;
                if (col < p.N) {
                    RowPtrs q = row_ptrs(p, row0 + lr, col);
                    const int64_t out_step = 4 * R * p.ld_out * (p.out_type == SC_F32 ? 4 : 2);
                    const int64_t pre_step = 4 * R * p.ld_pre * (p.pre_type == SC_F32 ? 4 : 2);
                    // the same quads for rows r and r + 8
                    const float *s0 = stg + lr * STG_COLS + (lc ^ lr) * 4, *s1 = stg + (lr + 4) * STG_COLS + (lc ^ (lr + 4)) * 4;
#pragma unroll 1
                    for (int r = lr; r < 32; r += 4 * R) {
                        float o[R][8];
                        bool in[R];
                        rows_in(row0 + r, in);
#pragma unroll
                        for (int k = 0; k < R; ++k) {
                            const float *f = (k & 1 ? s1 : s0) + (k >> 1) * 8 * STG_COLS;
                            const float4 x = *reinterpret_cast<const float4 *>(f);
                            const float4 y = *reinterpret_cast<const float4 *>(f + 32);
                            o[k][0] = x.x; o[k][1] = x.y; o[k][2] = x.z; o[k][3] = x.w;
                            o[k][4] = y.x; o[k][5] = y.y; o[k][6] = y.z; o[k][7] = y.w;
                        }
                        Residual<R, OUT> a;
                        if (p.res) {
                            if (AHEAD) {
                                a = ahead;
                                q.res += 4 * R * res_row;
                                if (r + 4 * R < 32) {
                                    bool next[R];
                                    rows_in(row0 + r + 4 * R, next);
                                    ahead.load(p, q.res, 4 * res_row, next);
                                } else if (more) {
                                    fetch_first(row0, col0 + STG_COLS);
                                }
                            } else {
                                a.load(p, q.res, 4 * res_row, in);
                                q.res += 4 * R * res_row;
                            }
                        }
                        epilogue_rows<ACT, OUT, R>(p, o, b, a, q, 4, in);
                        s0 += 4 * R * STG_COLS;
                        s1 += 4 * R * STG_COLS;
                        q.out += out_step;
                        q.pre += pre_step;
                    }
                }
            } else {
                epilogue_ragged<ACT, OUT>(p, stg, row0, col0, lane);
            }
            __syncwarp();
        };
        auto load_bias = [&](int col0, float (&b)[8]) {
            if (p.vec && p.bias && col0 + lc * 8 < p.N) load_any<8>(p.bias, p.bias_type, col0 + lc * 8, b);
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
            int tm, tn;
            tile_at(p, t, tm, tn);
            const int64_t row0 = (int64_t)tm * (CG * GM) + (CG == 2 ? rank * GM : 0) + quad * 32;
            const int n0 = tn * p.bn + c_lo;
            if (!SPLIT && p.res) {
                // the residual's part of this tile into L2, under the products
                const int cb = 128 / (p.out_type == SC_F32 ? 4 : 2), size = p.out_type == SC_F32 ? 4 : 2;
                const int cols = min(half, p.N - n0);
                if (row0 + lane < p.M)
                    for (int c = 0; c < cols; c += cb)
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char *>(p.res) +
                                                                     ((row0 + lane) * p.ld_res + n0 + c) * size));
            }
            if (!SPLIT) fetch_first(row0, n0);
            const uint32_t lane_acc = tmem + c_lo + ((uint32_t)(quad * 32) << 16);
            if constexpr (KEEP) {
                // add up the chunks: this lane's row, columns c_lo .. c_lo + half
                constexpr int COLS = SPLIT ? SPLIT_N / 2 : GN_MAX / 2;
                float v[COLS] = {};
                for (int i = it0; i < it1; i = chunk_end(i), ++n) {
                    const int buf = n & p.acc_two;
                    if (!wait(&sy.acc_full[buf], (n >> p.acc_two) & 1)) return;
                    tc_fence_after();
                    uint32_t acc = lane_acc + buf * ACC_COLS + p.rest;
                    for (int left = p.rest;; left = 0, acc -= p.rest) {  // the rest first
#pragma unroll
                        for (int c = 0; c < COLS; c += 32) {
                            if (c < half) {
                                uint32_t r[32];
                                tmem_ld32(acc + c, r);
#pragma unroll
                                for (int j = 0; j < 32; ++j) v[c + j] += __uint_as_float(r[j]);
                            }
                        }
                        if (!left) break;
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
                        float b[8] = {};
                        load_bias(n0 + c, b);
                        load_ragged_bias(n0 + c);
                        stage([&](int i) { return v[c + i]; });
                        store_staged(row0, n0 + c, b, c + STG_COLS < half);
                    }
                }
            } else {
                const int buf = n & p.acc_two;
                if (!wait(&sy.acc_full[buf], (n >> p.acc_two) & 1)) return;
                ++n;
                tc_fence_after();
                for (int c = 0; c < half; c += STG_COLS) {
                    float b[8] = {};
                    load_bias(n0 + c, b);
                    load_ragged_bias(n0 + c);
                    uint32_t r[2][32];
                    tmem_ld32_async(lane_acc + buf * ACC_COLS + c, r[0]);
                    tmem_ld32_async(lane_acc + buf * ACC_COLS + c + 32, r[1]);
                    tmem_wait_ld(r[0]);
                    tmem_wait_ld(r[1]);
                    // 16-bit results of fp32 operands are weight gradients: no activation
                    if (ACT == SC_ACT_NONE && p.rest) {
#pragma unroll
                        for (int h = 0; h < 64; h += 8) {
                            uint32_t q[8];
                            tmem_ld8(lane_acc + buf * ACC_COLS + p.rest + c + h, q);
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                uint32_t &x = r[h >> 5][(h & 31) + j];
                                x = __float_as_uint(__uint_as_float(x) + __uint_as_float(q[j]));
                            }
                        }
                    }
                    stage([&](int i) { return __uint_as_float(r[i >> 5][i & 31]); });
                    if (c + STG_COLS >= half) release(buf);
                    store_staged(row0, n0 + c, b, c + STG_COLS < half);
                }
            }
        }
    };
    // After a wait that expired: this CTA's (a pair's) products finish and its
    // copies land, each waited for with a limit again.  All threads call it, of
    // both CTAs of a pair, with no product or copy left to issue.
    auto settle = [&]() {
        int unused = 0;
        const long long limit = p.wait_limit / 16;
        if (warp == 1) {
            if ((CG == 1 || rank == 0) && elect_one()) mma_commit<CG>(&sy.drain);  // arrives in both CTAs
            mbar_wait(&sy.drain, 0, &unused, limit);
        } else if (threadIdx.x == 0 && rank * (CG - 1) == 0) {
            // A pair's copies all count on this CTA's barriers, which expect
            // both halves of the stages that this CTA armed: what only one of
            // the two issued is put right first.
            const uint32_t mine = sy.issued, other = CG == 2 ? sy.peer_issued : mine;
            const uint32_t end = max(mine, other), n = p.stages;
            for (uint32_t j = end < n ? 0 : end - n; j < end; ++j) {
                uint64_t *bar = &sy.full[j % n];
                if (j >= mine) mbar_expect_tx(bar, stage_bytes);
                else if (j >= other) mbar_complete_tx(bar, stage_bytes);
                unused = 0;
                mbar_wait(bar, (j / n) & 1, &unused, limit);
            }
        }
        __syncwarp();
        __syncthreads();
    };
    // all products and copies done, no arrival on its way to another CTA
    auto finish = [&]() {
        tc_fence_before();
        __syncthreads();
        if (CG == 2 && threadIdx.x == 0) {
            if (rank == 1) store_cluster(&sy.peer_issued, 0, sy.issued);
            if (*abort_flag) store_cluster(&sy.peer_abort, rank ^ 1, 1);
        }
        __syncwarp();
        if (CG == 2 || SPLIT) cluster_sync();
        tc_fence_after();
        if (__builtin_expect(*abort_flag || (CG == 2 && *(volatile uint32_t *)&sy.peer_abort), 0)) {
            if (!SPLIT) {
                settle();
                // no result of this CTA can be told from a right one: NaN (asks
                // for its place again: the usual way keeps no registers for this)
                const int step = CG == 2 ? (int)cluster_count() : (int)gridDim.x;
                for (int t = CG == 2 ? (int)cluster_id() : (int)blockIdx.x; t < p.n_tiles; t += step) {
                    int tm, tn;
                    tile_at(p, t, tm, tn);
                    const int64_t row0 = ((int64_t)tm * CG + (CG == 2 ? cluster_rank() : 0)) * GM;
                    for (int i = threadIdx.x; i < GM * p.bn; i += GEMM_THREADS) {
                        const int64_t row = row0 + i / p.bn;
                        const int col = tn * p.bn + i % p.bn;
                        if (row >= p.M || col >= p.N) continue;
                        if (p.pre) store_any(p.pre, p.pre_type, row * p.ld_pre + col, NAN);
                        store_any(p.out, p.out_type, row * p.ld_out + col, NAN);
                    }
                }
            }
            if (threadIdx.x == 0 && p.dev_status) atomicOr(p.dev_status, SC_DEV_WAIT_LIMIT);
            __syncwarp();
            if (CG == 2) cluster_sync();
        }
        if (warp == 2) tmem_free<CG>(tmem);
        // what follows on the stream must find the other product done too
        if (p.beside) asm volatile("griddepcontrol.wait;" ::: "memory");
    };
    // 128 sums per epilogue thread: those warps take registers over from the
    // other four (launched with KEEP_REGS each, which the host checks: 56 + 2 x
    // 224 = 3 x 168).  The two sides share no code after this.
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
        // This warp and the next walk their loops as a whole, with one elected
        // lane issuing: descriptors, addresses and coordinates then live in
        // uniform registers, which the issued instructions take (a lone thread
        // moves them there for every instruction: 380 cycles a stage).
        Ring r = {0, 0};
        uint32_t issued = 0;
        bool ok = true;
        const uint32_t full0 = CG == 2 ? cluster_addr(smem_addr(&sy.full[0]), 0) : smem_addr(&sy.full[0]);
        for (int t = first_tile; t < p.n_tiles && ok; t += tile_step) {
            int tm, tn;
            tile_at(p, t, tm, tn);
            const int m0 = tm * (CG * GM) + (CG == 2 ? rank * GM : 0);
            const int n0 = tn * p.bn + (CG == 2 ? rank * (p.bn / 2) : 0);
            int k = it0, part = 0;
            for (int i = it0 * p.planes; i < it1 * p.planes; ++i, ++issued) {
                if (!wait(&sy.empty[r.slot], r.phase ^ 1)) {
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    const uint32_t sa = base + r.slot * stage_bytes, bar = full0 + r.slot * 8;
                    if (rank == 0 || CG == 1) mbar_expect_tx(&sy.full[r.slot], p.stage_tx);
                    load_tile<CG>(sa, &p.ma, bar, p.a_mn, GM, m0, k * GK, part);
                    load_tile<CG>(sa + A_STAGE, &p.mb, bar, p.b_mn, p.bn / CG, n0, k * GK, part);
                }
                if (++part == p.planes) {
                    part = 0;
                    ++k;
                }
                r.next(p.stages);
            }
        }
        if (lane == 0) sy.issued = issued;
        if (ok) {
            // the ring's last stages consumed, oldest first: no copy and no
            // arrival is in flight
            const uint32_t last = issued < (uint32_t)p.stages ? issued : p.stages;
            r.back(last, p.stages);
            for (uint32_t j = 0; j < last; ++j, r.next(p.stages)) wait(&sy.empty[r.slot], r.phase);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ================= MMA issuer =================
        if (CG == 1 || rank == 0) {
            const uint64_t da = swizzled_desc(0, p.a_mn), db = swizzled_desc(0, p.b_mn);
            const uint32_t ka = (p.a_mn ? 2048u : 32u) >> 4, kb = (p.b_mn ? 2048u : 32u) >> 4;
            Ring r = {0, 0};
            uint32_t n = 0;
            bool ok = true;
            for (int t = first_tile; t < p.n_tiles && ok; t += tile_step) {
                for (int i = it0; i < it1 && ok; ++n) {
                    const int buf = n & p.acc_two;
                    if (!wait(&sy.acc_empty[buf], ((n >> p.acc_two) & 1) ^ 1)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t acc = tmem + buf * ACC_COLS;
                    const int end = chunk_end(i);
                    // the slot of the next stage, once it is there
                    auto arrived = [&](int &slot) {
                        if (!wait(&sy.full[r.slot], r.phase)) return ok = false;
                        tc_fence_after();
                        slot = r.slot;
                        r.next(p.stages);
                        return true;
                    };
                    auto product = [&](int a, int b, bool first, int d = 0) {
                        stage_mmas<CG>(acc + d, da, db, ka, kb, p.idesc, base + a * stage_bytes, base + b * stage_bytes, first);
                    };
                    for (bool first = true; i < end; ++i, first = false) {
                        int s0 = 0, s1 = 0, s2 = 0;
                        if (!arrived(s0)) break;
                        if (p.planes == 1) {
                            if (elect_one()) {
                                product(s0, s0, first);
                                mma_commit<CG>(&sy.empty[s0]);
                                if (i + 1 == end) mma_commit<CG>(&sy.acc_full[buf]);
                            }
                            continue;
                        }
                        if (elect_one()) product(s0, s0, first);
                        if (!arrived(s1)) break;
                        if (elect_one()) {
                            product(s1, s0, first, p.rest);
                            product(s0, s1, false, p.rest);
                            product(s1, s1, false, p.rest);
                            mma_commit<CG>(&sy.empty[s1]);
                        }
                        if (!arrived(s2)) break;
                        if (elect_one()) {
                            product(s2, s0, false, p.rest);
                            product(s0, s2, false, p.rest);
                            mma_commit<CG>(&sy.empty[s0]);
                            mma_commit<CG>(&sy.empty[s2]);
                            if (i + 1 == end) mma_commit<CG>(&sy.acc_full[buf]);
                        }
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp == 3) {
        // ================= column sums =================
        if (p.sums.part) {
            // 8 columns at a time, a quarter of the partial rows per lane
            for (int64_t c0 = (int64_t)blockIdx.x * 8; c0 < p.sums.cols; c0 += (int64_t)gridDim.x * 8) {
                const int64_t c = c0 + (lane & 7);
                float v = 0.f;
                for (int i0 = lane >> 3; i0 < p.sums.n; i0 += 32) {
                    float t[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int i = i0 + 4 * k;
                        t[k] = i < p.sums.n && c < p.sums.cols ? p.sums.part[i * p.sums.cols + c] : 0.f;
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k) v += t[k];
                }
                v += __shfl_xor_sync(0xffffffffu, v, 8);
                v += __shfl_xor_sync(0xffffffffu, v, 16);
                if (lane < 8 && c < p.sums.cols) store_any(p.sums.out, p.sums.type, c, v);
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
        if (__builtin_expect(*abort_flag, 0)) {  // NaN in this part makes the sums NaN
            settle();
            for (int i = threadIdx.x; i < GM * SPLIT_LD; i += GEMM_THREADS) reinterpret_cast<float *>(ring)[i] = NAN;
            __syncthreads();
        }
        cluster_sync();
        const int parts = (int)gridDim.x / p.n_tiles;
        int tm, tn;
        tile_at(p, first_tile, tm, tn);
        const int m0 = tm * GM, n0 = tn * p.bn;
        const int groups = p.bn / 8;
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
            if (p.vec) {
                float b[8] = {};
                if (p.bias) load_any<8>(p.bias, p.bias_type, n0 + c, b);
                float o[1][8];
#pragma unroll
                for (int j = 0; j < 8; ++j) o[0][j] = v[j];
                const bool in[1] = {true};
                const RowPtrs q = row_ptrs(p, m0 + r, n0 + c);
                Residual<1, OUT_ANY> a;
                if (p.res) a.load(p, q.res, 0, in);
                epilogue_rows<ACT, OUT_ANY, 1>(p, o, b, a, q, 0, in);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (n0 + c + j >= p.N) break;
                    float b[1] = {0.f};
                    if (p.bias) load_any<1>(p.bias, p.bias_type, n0 + c + j, b);
                    epilogue1<ACT>(p, v[j], b[0], m0 + r, n0 + c + j);
                }
            }
        }
        __syncwarp();
    }
    finish();
}

using GemmFn = void (*)(GemmArgs);

// The kernels of one activation (sc_gemm_k_*.cu).
enum { SUM_16, SUM_16_LONG, SUM_F32 };  // result type, and whether its sums are kept in registers
struct GemmKernels {
    GemmFn pair[3], single[3];  // [SUM_*]
    GemmFn split;
};
template <int ACT>
GemmKernels gemm_kernels() {
    return {{gemm_kernel<2, false, false, OUT_16, ACT>, gemm_kernel<2, false, true, OUT_16, ACT>,
             gemm_kernel<2, false, true, OUT_F32, ACT>},
            {gemm_kernel<1, false, false, OUT_16, ACT>, gemm_kernel<1, false, true, OUT_16, ACT>,
             gemm_kernel<1, false, true, OUT_F32, ACT>},
            gemm_kernel<1, true, true, OUT_ANY, ACT>};
}
GemmKernels gemm_kernels_none();
GemmKernels gemm_kernels_relu();
GemmKernels gemm_kernels_gelu();
GemmKernels gemm_kernels_gelu_tanh();
GemmKernels gemm_kernels_silu();

}  // namespace gemm
}  // namespace scb
