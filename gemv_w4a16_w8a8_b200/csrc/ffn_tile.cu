// Large-tile tensor-core kernel of the scaled W8A8 matmul and of the gated feed-forward block's
// forward and backward products.
//
// One CTA pair (cta_group::2) owns a tile of 256 rows x BN columns of the result: tokens (or, for
// the weights' gradients, weight rows) are the MMA's M side, 128 to each CTA, so that a TMEM lane
// holds one row of the result and its columns are contiguous in memory; each CTA loads half of
// the BN rows of the other operand. Operands arrive by TMA in slabs of 128 bytes of the reduction
// under SWIZZLE_128B:
//   - K-major (the reduction contiguous in memory): activations and weights of the forward
//     products, dG / dU in dX;
//   - MN-major (the reduction along rows): Wg / Wu in dX, dG / dU and X in the weights'
//     gradients. A slab is then 64 rows, copied as chunks of 64 values, and the MMA reads it
//     transposed: no transposed copy of any tensor is made.
// Forms:
//   kScaled  C = sa sw (A W^T) + bias
//   kGated   the pair's first CTA loads BN / 2 rows of Wg, its second the same rows of Wu: one MMA
//            makes gate and up of the same columns in one accumulator, and the epilogue of each
//            token forms act(gate) * up
//   kDx      dG Wg + dU Wu as one reduction over 2 F: the slabs of dG Wg, then those of dU Wu
//   kDw      dG^T X and dU^T X: two results in one launch
// Few tiles and a long reduction (kDx, kDw): the reduction is cut into parts that store fp32 partial
// sums, added in order by a second kernel (no atomics: the same bits every run).
//
// Warps: 0-3 epilogue, 4 TMA producer, 5 MMA issue (the pair's first CTA issues for both) and
// TMEM. Accumulators are double buffered, so the epilogue of a tile runs under the next tile's
// MMAs. Every wait is bounded as in the other tensor-core kernels.
#include <algorithm>
#include <mutex>

#include "ffn.cuh"
#include "sm100.cuh"

namespace qg {
namespace {

enum Form { kScaled, kGated, kDx, kDw };

constexpr int kThreads = 192;
constexpr int kTileM = 256, kRows = 128;       // rows of the result: of a pair, of a CTA
constexpr int kSlab = 128;                     // bytes of the reduction per stage (K-major)
constexpr int kRasterM = 8;                    // row tiles per raster group

// Partial tiles: a CTA's 128 rows x 128 B, and BN / 2 rows x 128 B of the other operand
template <int BN> struct Ring {
    static constexpr int a_bytes = kRows * kSlab;
    static constexpr int b_bytes = BN / 2 * kSlab;
    static constexpr int stage = a_bytes + b_bytes;
    static constexpr int stages = BN == 256 ? 6 : 8;
    static constexpr int out_off = stages * stage;            // 4 warps x 32 rows x 128 B
    static constexpr int col_off = out_off + 4 * 32 * 128;    // 4 warps x (BN scales, BN biases)
    static constexpr int bar_off = col_off + 4 * 2 * BN * 4;
    static constexpr int nbars = 2 * stages + 5;
    static constexpr int total = 1024 + bar_off + nbars * 8 + 16;
};
static_assert(Ring<256>::total <= 227 * 1024 && Ring<128>::total <= 227 * 1024, "shared memory");

struct Shape {
    int M, N;               // the result's rows and columns (N: columns of H for kGated)
    int tiles_m, tiles_n;
    int seg_slabs;          // slabs of the reduction (of one of the two products for kDx)
    int slabs;              // slabs in all: 2 seg_slabs for kDx
    int parts, part_slabs;  // parts of the reduction and slabs of each (the last may have fewer)
    int units;              // results x tiles x parts
    int act;
};

struct Out {
    void *c0, *c1, *c2;                 // C / H, G, U / dX / dWg, dWu
    float *part;                        // fp32 partial sums [result][part][M][N]
    const float *sa, *sw, *sw1;
    const void *bias;
};

struct Unit {
    int which, m0, n0, part, s0, ns;    // result, origin of the tile, part, first slab, slabs
};

// Tiles in groups of kRasterM row tiles, rows fastest: the pairs at work at one time share a block
// of about kRasterM x 9 tiles whose operands stay in L2.
template <int NCOL>
__device__ __forceinline__ Unit unit_of(int u, const Shape &s)
{
    Unit w;
    w.part = u % s.parts;
    int t = u / s.parts;
    const int per = s.tiles_m * s.tiles_n;
    w.which = t / per;
    t -= w.which * per;
    const int group = t / (kRasterM * s.tiles_n);
    const int first = group * kRasterM;
    const int gm = min(kRasterM, s.tiles_m - first);
    t -= group * kRasterM * s.tiles_n;
    w.m0 = (first + t % gm) * kTileM;
    w.n0 = (t / gm) * NCOL;
    w.s0 = w.part * s.part_slabs;
    w.ns = min(s.part_slabs, s.slabs - w.s0);
    return w;
}

template <bool I8>
__device__ __forceinline__ void mma_pair(uint32_t dtm, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate)
{
    if constexpr (I8)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(dtm),
                     "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(dtm),
                     "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
                     : "memory");
}

// int8: s32 accumulator (2), signed operands (1). 16-bit: fp32 accumulator (1), fp16 (0) or bf16
// (1) operands; bits 15 and 16: MN-major A and B.
template <bool I8, typename T, int BN, bool AMN, bool BMN> constexpr uint32_t instr_desc()
{
    const uint32_t in = I8 ? 1u : (sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value ? 1u : 0u);
    return (I8 ? 2u : 1u) << 4 | in << 7 | in << 10 | (AMN ? 1u : 0u) << 15 | (BMN ? 1u : 0u) << 16 |
           (uint32_t)(BN >> 3) << 17 | (uint32_t)(kTileM >> 4) << 24;
}

// A warp's 32 rows x 128 bytes of results, staged in shared memory (16-byte piece j of row r at
// j ^ (r & 7): neither side has bank conflicts) and written as whole rows: 16 bytes a lane where
// rows of the result are 16-byte aligned, else a row at a time, an element a lane.
__device__ __forceinline__ void stage_put(uint8_t *stage, int lane, int j, const uint4 &v)
{
    *reinterpret_cast<uint4 *>(stage + lane * 128 + ((j ^ (lane & 7)) << 4)) = v;
}

template <typename E>
__device__ __forceinline__ void stage_flush(const uint8_t *stage, E *c, size_t ld, int rows, int cols,
                                            int lane, bool vec)
{
    constexpr int kPer = 16 / sizeof(E), kCols = 128 / sizeof(E);
    __syncwarp();
    if (vec) {
        const int j = lane & 7;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = i * 4 + (lane >> 3);
            const uint4 v = *reinterpret_cast<const uint4 *>(stage + r * 128 + ((j ^ (r & 7)) << 4));
            if (r < rows && j * kPer < cols)
                *reinterpret_cast<uint4 *>(c + (size_t)r * ld + j * kPer) = v;
        }
    } else {
#pragma unroll 8
        for (int r = 0; r < 32; ++r)
#pragma unroll
            for (int q = lane; q < kCols; q += 32)
                if (r < rows && q < cols)
                    c[(size_t)r * ld + q] = *reinterpret_cast<const E *>(
                        stage + r * 128 + (((q / kPer) ^ (r & 7)) << 4) + (q % kPer) * sizeof(E));
    }
    __syncwarp();
}

template <int FORM, bool I8, typename T, int BN>
__global__ void __launch_bounds__(kThreads, 1)
tile_kernel(const __grid_constant__ CUtensorMap tm_a0, const __grid_constant__ CUtensorMap tm_a1,
            const __grid_constant__ CUtensorMap tm_b0, const __grid_constant__ CUtensorMap tm_b1,
            const Shape shape, const Out out, unsigned int *err)
{
    using L = Ring<BN>;
    constexpr bool AMN = FORM == kDw, BMN = FORM == kDx || FORM == kDw;
    constexpr int NCOL = FORM == kGated ? BN / 2 : BN;         // result columns of a tile
    constexpr int kElems = I8 ? 128 : 64;                      // reduction values per slab
    constexpr uint32_t kIdesc = instr_desc<I8, T, BN, AMN, BMN>();
    constexpr uint32_t kCols = 2 * BN;
    constexpr int ST = L::stages;

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(base + L::bar_off);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + L::nbars);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    auto full_bar = [&](int s) { return smem_u32(bars + s); };
    auto empty_bar = [&](int s) { return smem_u32(bars + ST + s); };
    auto accf_bar = [&](int b) { return smem_u32(bars + 2 * ST + b); };
    auto acce_bar = [&](int b) { return smem_u32(bars + 2 * ST + 2 + b); };
    const uint32_t final_bar = smem_u32(bars + 2 * ST + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int ustart = blockIdx.x >> 1, ustep = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(accf_bar(b), 1);
            mbar_init(acce_bar(b), 8);       // the epilogue warps of both CTAs
        }
        mbar_init(final_bar, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async_smem();
    }
    if (warp == 5) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(tmem_holder)),
                     "r"(kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    grid_wait();

    // The producer and MMA warps run with all lanes and issue from lane 0, so that addresses and
    // coordinates stay warp-uniform.
    if (warp == 4) {
        // ---------------- TMA producer: this CTA's halves of both operands ----------------
        int it = 0;
        bool stop = false;
        for (int u = ustart; u < shape.units && !stop; u += ustep) {
            const Unit w = unit_of<NCOL>(u, shape);
            for (int i = 0; i < w.ns; ++i, ++it) {
                const int s = it % ST;
                if (!warp_wait(empty_bar(s), ((it / ST) & 1) ^ 1, abort_flag, err)) {
                    stop = true;
                    break;
                }
                if (lane == 0) {
                    const int slab = w.s0 + i;
                    const bool second = FORM == kDx && slab >= shape.seg_slabs;
                    const int k = (second ? slab - shape.seg_slabs : slab) * kElems;
                    const uint32_t fb = map_to_rank(full_bar(s), 0);
                    const uint32_t sa = smem_u32(base + s * L::stage), sb = sa + L::a_bytes;
                    const CUtensorMap *ma = (FORM == kDw ? w.which : (int)second) ? &tm_a1 : &tm_a0;
                    const CUtensorMap *mb = (FORM == kGated ? rank != 0 : second) ? &tm_b1 : &tm_b0;
                    // both CTAs' copies complete on the first CTA's barrier, which expects both
                    if (rank == 0) mbar_expect_tx(full_bar(s), 2 * L::stage);
                    const int am = w.m0 + (int)rank * kRows;
                    const int bn = FORM == kGated ? w.n0 : w.n0 + (int)rank * (BN / 2);
                    if constexpr (AMN) {
                        tma_load_2d_pair(sa, ma, fb, am, k);
                        tma_load_2d_pair(sa + 8192, ma, fb, am + 64, k);
                    } else {
                        tma_load_2d_pair(sa, ma, fb, k, am);
                    }
                    if constexpr (BMN) {
#pragma unroll
                        for (int c = 0; c < BN / 2; c += 64)
                            tma_load_2d_pair(sb + c * kSlab, mb, fb, bn + c, k);
                    } else {
                        tma_load_2d_pair(sb, mb, fb, k, bn);
                    }
                }
                __syncwarp();
            }
        }
        grid_release();        // every load is on its way: the next kernel may start
        // every copy this warp started must land before the CTA can exit
        if (rank == 0) {
            for (int i = max(0, it - ST); i < it; ++i) {
                int dummy_abort = 0;
                mbar_wait(full_bar(i % ST), (i / ST) & 1, &dummy_abort, nullptr);
            }
        } else if (*abort_flag) {
            // the second CTA's copies complete on the first's barrier: after a give-up (the only
            // way it can stop early) it waits far beyond the latency of a copy
            const uint64_t t0 = global_ns();
            while (global_ns() - t0 < 100000ull) __nanosleep(1000);
        }
    } else if (warp == 5 && rank == 0) {
        // ---------------- MMA issue for both CTAs ----------------
        int it = 0, j = 0;
        bool stop = false;
        for (int u = ustart; u < shape.units && !stop; u += ustep, ++j) {
            const Unit w = unit_of<NCOL>(u, shape);
            const int b = j & 1;
            if (!warp_wait(acce_bar(b), ((j >> 1) & 1) ^ 1, abort_flag, err)) break;
            tc_fence_after();
            const uint32_t dtm = tmem_base + (uint32_t)(b * BN);
            for (int i = 0; i < w.ns; ++i, ++it) {
                const int s = it % ST;
                if (!warp_wait(full_bar(s), (it / ST) & 1, abort_flag, err)) {
                    stop = true;
                    break;
                }
                tc_fence_after();
                const uint32_t sa = smem_u32(base + s * L::stage), sb = sa + L::a_bytes;
                const uint64_t da = AMN ? sw128_desc_mn(sa, 8192) : sw128_desc(sa);
                const uint64_t db = BMN ? sw128_desc_mn(sb, 8192) : sw128_desc(sb);
                // 32 bytes of a K-major slab, or 16 rows (2048 B) of an MN-major one, per MMA
                constexpr int ka = AMN ? 128 : 2, kb = BMN ? 128 : 2;
                if (lane == 0) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_pair<I8>(dtm, da + ka * k, db + kb * k, kIdesc, (i | k) != 0 ? 1u : 0u);
                    mma_commit_pair_both(empty_bar(s));
                }
                __syncwarp();
            }
            if (stop) break;
            if (lane == 0) mma_commit_pair_both(accf_bar(b));
            __syncwarp();
        }
        // nothing may still run on the tensor cores when TMEM is released
        if (lane == 0) mma_commit_pair_local(final_bar);
        __syncwarp();
        int dummy_abort = 0;
        mbar_wait(final_bar, 0, &dummy_abort, nullptr);
    } else if (warp < 4) {
        // ---------------- epilogue: lane = row of the result ----------------
        uint8_t *stage = base + L::out_off + warp * 32 * 128;
        float *col = reinterpret_cast<float *>(base + L::col_off) + warp * 2 * BN;
        const int N = shape.N;
        const bool vec = (N & 7) == 0;
        int j = 0;
        for (int u = ustart; u < shape.units; u += ustep, ++j) {
            const Unit w = unit_of<NCOL>(u, shape);
            const int b = j & 1;
            const int m = w.m0 + (int)rank * kRows + warp * 32;       // the warp's first row
            const int rows = min(32, shape.M - m);
            float sa = 0.f;
            if constexpr (I8) {
                // this tile's column scales (and biases), a copy for each warp
                sa = lane < rows ? out.sa[m + lane] : 0.f;
                for (int c = lane; c < BN; c += 32) {
                    if constexpr (FORM == kGated) {
                        const int n = w.n0 + (c % NCOL);
                        col[c] = n < N ? (c < NCOL ? out.sw : out.sw1)[n] : 0.f;
                    } else {
                        const int n = w.n0 + c;
                        col[c] = n < N ? out.sw[n] : 0.f;
                        col[BN + c] = out.bias && n < N ? to_f32(static_cast<const T *>(out.bias)[n]) : 0.f;
                    }
                }
                __syncwarp();
            }
            bool ok = mbar_wait(accf_bar(b), (j >> 1) & 1, abort_flag, err);
            tc_fence_after();
            ok = __all_sync(0xffffffffu, ok && !*abort_flag);
            if (!ok) break;
            const uint32_t tm = tmem_base + ((uint32_t)(warp * 32) << 16) + (uint32_t)(b * BN);
            if (rows > 0) {
                if constexpr (FORM == kDx || FORM == kDw) {
                    if (shape.parts > 1) {
                        float *dst = out.part + ((size_t)(w.which * shape.parts + w.part) * shape.M + m) * N;
#pragma unroll 1
                        for (int c = 0; c < NCOL && w.n0 + c < N; c += 32) {
                            uint32_t v[32];
                            tmem_ld32(tm + c, v);
                            tmem_wait_ld();
#pragma unroll
                            for (int q = 0; q < 8; ++q)
                                stage_put(stage, lane, q, make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]));
                            stage_flush(stage, dst + w.n0 + c, N, rows, N - w.n0 - c, lane, true);
                        }
                    }
                }
                if ((FORM != kDx && FORM != kDw) || shape.parts == 1) {
                    T *c0 = static_cast<T *>(FORM == kDw && w.which ? out.c1 : out.c0) + (size_t)m * N;
#pragma unroll 1
                    for (int c = 0; c < NCOL && w.n0 + c < N; c += 64) {
                        const int cols = N - w.n0 - c;
                        uint32_t hw[32], gw[32], uw[32];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t v[32];
                            tmem_ld32(tm + c + 32 * h, v);
                            if constexpr (FORM == kGated) {
                                uint32_t z[32];
                                tmem_ld32(tm + NCOL + c + 32 * h, z);
                                tmem_wait_ld();
                                auto pre = [&](uint32_t x, int at) {
                                    if constexpr (I8)
                                        return __fmul_rn(__fmul_rn(__int2float_rn((int)x), sa), col[at]);
                                    else
                                        return __uint_as_float(x);
                                };
                                auto gate = [&](auto act) {
                                    constexpr int ACT = decltype(act)::value;
#pragma unroll
                                    for (int q = 0; q < 16; ++q) {
                                        const int at = c + 32 * h + 2 * q;
                                        const float g0 = pre(v[2 * q], at), g1 = pre(v[2 * q + 1], at + 1);
                                        const float u0 = pre(z[2 * q], NCOL + at), u1 = pre(z[2 * q + 1], NCOL + at + 1);
                                        hw[16 * h + q] = pack2<T>(act_value<ACT>(g0) * u0, act_value<ACT>(g1) * u1);
                                        gw[16 * h + q] = pack2<T>(g0, g1);
                                        uw[16 * h + q] = pack2<T>(u0, u1);
                                    }
                                };
                                if (shape.act == QG_ACT_SILU) gate(Const<QG_ACT_SILU>{});
                                else if (shape.act == QG_ACT_GELU) gate(Const<QG_ACT_GELU>{});
                                else gate(Const<QG_ACT_GELU_TANH>{});
                            } else {
                                tmem_wait_ld();
#pragma unroll
                                for (int q = 0; q < 16; ++q) {
                                    float r[2];
#pragma unroll
                                    for (int e = 0; e < 2; ++e) {
                                        if constexpr (I8) {
                                            const int at = c + 32 * h + 2 * q + e;
                                            r[e] = __fmul_rn(__fmul_rn(__int2float_rn((int)v[2 * q + e]), sa), col[at]);
                                            if (out.bias) r[e] = __fadd_rn(r[e], col[BN + at]);
                                        } else {
                                            r[e] = __uint_as_float(v[2 * q + e]);
                                        }
                                    }
                                    hw[16 * h + q] = pack2<T>(r[0], r[1]);
                                }
                            }
                        }
                        auto write = [&](const uint32_t (&x)[32], T *dst) {
#pragma unroll
                            for (int q = 0; q < 8; ++q)
                                stage_put(stage, lane, q, make_uint4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]));
                            if (vec || (N & 1))
                                stage_flush(stage, dst + w.n0 + c, N, rows, cols, lane, vec);
                            else     // pairs of elements
                                stage_flush(stage, reinterpret_cast<uint32_t *>(dst + w.n0 + c), N / 2, rows,
                                            cols / 2, lane, false);
                        };
                        write(hw, c0);
                        if constexpr (FORM == kGated && !I8) {
                            if (out.c1) {
                                write(gw, static_cast<T *>(out.c1) + (size_t)m * N);
                                write(uw, static_cast<T *>(out.c2) + (size_t)m * N);
                            }
                        }
                    }
                }
            }
            // the accumulator goes back to the MMA warp (of the pair's first CTA)
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(map_to_rank(acce_bar(b), 0));
        }
    }

    tc_fence_before();
    __syncwarp();
    cluster_sync();
    if (warp == 5) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(kCols)
                     : "memory");
    }
}

// ---- host side -------------------------------------------------------------------------------------

struct Matrix {          // a 16-bit or int8 matrix [rows, cols] with `pitch` bytes a row
    const void *p;
    uint64_t rows, cols, pitch;
};

template <bool I8, typename T> bool map_of(CUtensorMap *m, const Matrix &x, bool mn, int box_rows)
{
    const CUtensorMapDataType dt = I8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                      : (std::is_same<T, __nv_bfloat16>::value ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                                     : CU_TENSOR_MAP_DATA_TYPE_FLOAT16);
    return make_map(m, dt, x.p, x.cols, x.rows, x.pitch, I8 ? 128 : 64, mn ? 64 : box_rows,
                    CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int FORM, bool I8, typename T, int BN>
cudaError_t launch_tile(const Matrix &a0, const Matrix &a1, const Matrix &b0, const Matrix &b1,
                        const Shape &shape, const Out &out, unsigned int *err, cudaStream_t stream)
{
    using L = Ring<BN>;
    constexpr bool AMN = FORM == kDw, BMN = FORM == kDx || FORM == kDw;
    auto kern = tile_kernel<FORM, I8, T, BN>;
    // per device: the shared-memory opt-in and the number of pairs that fit at once
    static std::mutex mu;
    static int pairs_of[64] = {};
    int dev = 0, pairs = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (!pairs_of[dev]) {
            cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::total);
            if (e != cudaSuccess) return e;
            cudaLaunchConfig_t cfg = {};
            cudaLaunchAttribute attr[1];
            cfg.gridDim = dim3(2);
            cfg.blockDim = dim3(kThreads);
            cfg.dynamicSmemBytes = L::total;
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 2;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            int n = 0;
            e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
            if (e != cudaSuccess) return e;
            if (n <= 0) return cudaErrorInvalidConfiguration;
            pairs_of[dev] = n;
        }
        pairs = pairs_of[dev];
    }
    CUtensorMap ta0, ta1, tb0, tb1;
    if (!map_of<I8, T>(&ta0, a0, AMN, kRows) || !map_of<I8, T>(&tb0, b0, BMN, BN / 2)) return cudaErrorInvalidValue;
    ta1 = ta0;
    tb1 = tb0;
    if (a1.p != a0.p && !map_of<I8, T>(&ta1, a1, AMN, kRows)) return cudaErrorInvalidValue;
    if (b1.p != b0.p && !map_of<I8, T>(&tb1, b1, BMN, BN / 2)) return cudaErrorInvalidValue;
    return launch_dependent(kern, dim3(2 * std::min(shape.units, pairs)), dim3(kThreads), L::total, 2, stream,
                            ta0, ta1, tb0, tb1, shape, out, err);
}

int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Tile width: 256 columns run at the MMA's full rate; 128 columns take about 0.55 of its time
// and fill the last wave of pairs better. The shorter schedule wins.
bool narrow_tile(int M, int ncol256, int N, int results, int pairs)
{
    const long tm = ceil_div(M, kTileM);
    const long wide = (tm * ceil_div(N, ncol256) * results + pairs - 1) / pairs;
    const long narrow = (tm * ceil_div(N, ncol256 / 2) * results + pairs - 1) / pairs;
    return 0.55 * narrow < wide;
}

Shape shape_of(int M, int N, int ncol, int results, int seg_slabs, int segs, int parts, int act)
{
    Shape s;
    s.M = M;
    s.N = N;
    s.tiles_m = ceil_div(M, kTileM);
    s.tiles_n = ceil_div(N, ncol);
    s.seg_slabs = seg_slabs;
    s.slabs = segs * seg_slabs;
    s.part_slabs = ceil_div(s.slabs, parts);
    s.parts = ceil_div(s.slabs, s.part_slabs);      // no empty part
    s.units = results * s.tiles_m * s.tiles_n * s.parts;
    s.act = act;
    return s;
}

} // namespace

cudaError_t launch_tile_scaled(const ScaledProblem &p, int sms, unsigned int *err, cudaStream_t stream)
{
    const uint64_t K = p.K;
    const Matrix a{p.A, (uint64_t)p.M, K, K}, w{p.W, (uint64_t)p.N, K, K};
    const Matrix w1{p.W1 ? p.W1 : p.W, (uint64_t)p.N, K, K};
    const Out out{p.C, nullptr, nullptr, nullptr, p.sa, p.sw, p.sw1, p.bias};
    const bool narrow = narrow_tile(p.M, p.W1 ? 128 : 256, p.N, 1, sms / 2);
    const int slabs = ceil_div(p.K, 128);
    QG_DISPATCH_16(p.dtype, T, {
        if (p.W1) {
            if (narrow)
                return launch_tile<kGated, true, T, 128>(a, a, w, w1, shape_of(p.M, p.N, 64, 1, slabs, 1, 1, p.act), out, err, stream);
            return launch_tile<kGated, true, T, 256>(a, a, w, w1, shape_of(p.M, p.N, 128, 1, slabs, 1, 1, p.act), out, err, stream);
        }
        if (narrow)
            return launch_tile<kScaled, true, T, 128>(a, a, w, w1, shape_of(p.M, p.N, 128, 1, slabs, 1, 1, 0), out, err, stream);
        return launch_tile<kScaled, true, T, 256>(a, a, w, w1, shape_of(p.M, p.N, 256, 1, slabs, 1, 1, 0), out, err, stream);
    });
}

cudaError_t launch_tile_gated(const GatedProblem &p, int sms, unsigned int *err, cudaStream_t stream)
{
    const uint64_t K = p.K, pitch = K * 2;
    const Matrix x{p.X, (uint64_t)p.M, K, pitch}, g{p.Wg, (uint64_t)p.F, K, pitch}, u{p.Wu, (uint64_t)p.F, K, pitch};
    const Out out{p.H, p.G, p.U, nullptr, nullptr, nullptr, nullptr, nullptr};
    const int slabs = ceil_div(p.K, 64);
    const bool narrow = narrow_tile(p.M, 128, p.F, 1, sms / 2);
    QG_DISPATCH_16(p.dtype, T, {
        if (narrow)
            return launch_tile<kGated, false, T, 128>(x, x, g, u, shape_of(p.M, p.F, 64, 1, slabs, 1, 1, p.act), out, err, stream);
        return launch_tile<kGated, false, T, 256>(x, x, g, u, shape_of(p.M, p.F, 128, 1, slabs, 1, 1, p.act), out, err, stream);
    });
}

cudaError_t launch_tile_dx(const GatedGrad &p, int sms, unsigned int *err, cudaStream_t stream)
{
    const uint64_t M = p.M, F = p.F, K = p.K;
    const Matrix dg{p.dG, M, F, (uint64_t)p.Fp * 2}, du{p.dU, M, F, (uint64_t)p.Fp * 2};
    const Matrix wg{p.Wg, F, K, K * 2}, wu{p.Wu, F, K, K * 2};
    const Out out{p.dX, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr};
    const int slabs = ceil_div(p.F, 64);
    const bool narrow = narrow_tile(p.M, 256, p.K, 1, sms / 2);
    QG_DISPATCH_16(p.dtype, T, {
        if (narrow)
            return launch_tile<kDx, false, T, 128>(dg, du, wg, wu, shape_of(p.M, p.K, 128, 1, slabs, 2, 1, 0), out, err, stream);
        return launch_tile<kDx, false, T, 256>(dg, du, wg, wu, shape_of(p.M, p.K, 256, 1, slabs, 2, 1, 0), out, err, stream);
    });
}

cudaError_t launch_tile_dw(const GatedGrad &p, int sms, unsigned int *err, cudaStream_t stream)
{
    const uint64_t M = p.M, F = p.F, K = p.K;
    const Matrix dg{p.dG, M, F, (uint64_t)p.Fp * 2}, du{p.dU, M, F, (uint64_t)p.Fp * 2};
    const Matrix x{p.X, M, K, K * 2};
    const Out out{p.dWg, p.dWu, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr};
    const int slabs = ceil_div(p.M, 64);
    const bool narrow = narrow_tile(p.F, 256, p.K, 2, sms / 2);
    QG_DISPATCH_16(p.dtype, T, {
        if (narrow)
            return launch_tile<kDw, false, T, 128>(dg, du, x, x, shape_of(p.F, p.K, 128, 2, slabs, 1, 1, 0), out, err, stream);
        return launch_tile<kDw, false, T, 256>(dg, du, x, x, shape_of(p.F, p.K, 256, 2, slabs, 1, 1, 0), out, err, stream);
    });
}

} // namespace qg
