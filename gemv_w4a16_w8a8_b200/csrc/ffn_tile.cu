// Large-tile tensor-core kernel of the scaled W8A8 matmul and of the gated feed-forward block's
// forward and backward products.
//
// One CTA pair (cta_group::2) owns a tile of 256 rows x bn columns of the result: tokens (or, for
// the weights' gradients, weight rows) are the MMA's M side, 128 to each CTA, so that a TMEM lane
// holds one row of the result and its columns are contiguous in memory; each CTA loads half of
// the bn rows of the other operand. bn is chosen per call (plan_tiles). Operands arrive by TMA in
// slabs of 128 bytes of the reduction under SWIZZLE_128B:
//   - K-major (the reduction contiguous in memory): activations and weights of the forward
//     products, dG / dU in dX;
//   - MN-major (the reduction along rows): Wg / Wu in dX, dG / dU and X in the weights'
//     gradients. A slab is then 64 rows, copied as chunks of 64 values, and the MMA reads it
//     transposed: no transposed copy of any tensor is made.
// Forms:
//   kScaled  C = sa sw (A W^T) + bias
//   kGated   the pair's first CTA loads bn / 2 rows of Wg, its second the same rows of Wu: one MMA
//            makes gate and up of the same columns in one accumulator, and the epilogue of each
//            token forms act(gate) * up
//   kDx      dG Wg + dU Wu as one reduction over 2 F: the slabs of dG Wg, then those of dU Wu
//   kDw      dG^T X and dU^T X: two results in one launch
//   kBoth    kDx and kDw in one launch. dX's tiles are few and long, the weights' many and short: the
//            pairs that get one tile of dX less than others take as many whole rounds of the weights'
//            tiles for it as fit, then all share the rest, instead of a partial wave of each product
//            (M x F x K = 3000 x 1500 x 696: 48.8 -> 33.1 us; 1741 x 580 x 2688: 37.8 -> 29.4). Its
//            slabs are 3 to 8 % slower (operand layouts are chosen unit by unit), so whole waves stay
//            with two launches
// Few tiles and a long reduction (gradients): the reduction is cut into parts that store fp32 partial
// sums, added in order by a second kernel (no atomics: the same bits every run).
//
// Warps: 0-7 epilogue (two for each quarter of the TMEM lanes, every other 32 columns each), 8 TMA
// producer, 9 MMA issue (the pair's first CTA issues for both) and TMEM. Accumulators are double
// buffered, so the epilogue of a tile runs under the next tile's MMAs. Every wait is bounded as in
// the other tensor-core kernels.
//
// Bound: the tensor pipe. A tile of 256 columns asks an SM for 32 KB of operands per slab of 512
// MMA cycles, about what L2 delivers to one (90 GB/s), so it reaches 75 to 80 % of the MMA's rate
// with int8 and 80 to 92 % with 16 bits inside a wave. Times on a cool GPU, and of calls that follow
// one another until its power cap holds the clock: 8192 x 11008 x 4096 bf16, G and U saved, 0.98 ms
// (1.5 PFLOP/s, 92 % of the burst matmul rate) and 1.16 ms (92 % of the sustained rate); its
// backward pass 2.0 and 2.4 ms; int8 16384^3 2.7 ms (3.2 POP/s) and 3.2 ms; int8 gated 11008 x 4096,
// 512 tokens 41 and 47 us, 8192 tokens 0.48 and 0.56 ms.
// Weights fetched into L2 one ring ahead: 1 to 20 % slower. A tile's epilogue takes about 2.5 us
// and bounds reductions shorter than 8 slabs (16384 x 4096 x 256 int8: 47 us, 3.0 TB/s).
#include <algorithm>
#include <mutex>

#include "ffn_mma.cuh"

namespace qg {
namespace {

using namespace tile;

constexpr bool is_grad(int form) { return form >= kDx; }

constexpr int kEpiWarps = 8, kTmaWarp = 8, kMmaWarp = 9;
constexpr int kThreads = 32 * (kEpiWarps + 2);
constexpr int kRows = kTileM / 2;              // rows of the result of a CTA
constexpr int kSlab = 128;                     // bytes of the reduction per stage (K-major)

// Shared memory: stages of a CTA's 128 rows x 128 B and up to 128 rows x 128 B of the other
// operand, then for each epilogue warp 32 rows x 64 B of results and 64 column factors.
namespace ring {
constexpr int a_bytes = kRows * kSlab;
constexpr int stage = a_bytes + kMaxBn / 2 * kSlab;
constexpr int stages = 6;
constexpr int out_off = stages * stage;
constexpr int col_off = out_off + kEpiWarps * 32 * 64;
constexpr int bar_off = col_off + kEpiWarps * 64 * 4;
constexpr int nbars = 2 * stages + 5;
constexpr int total = 1024 + bar_off + nbars * 8 + 16;
static_assert(total <= 227 * 1024, "shared memory");
} // namespace ring

struct Out {
    void *c0, *c1, *c2;                 // C / H, G, U / dX, dWg, dWu
    float *part_x, *part_w;             // fp32 partial sums [result][part][M][N]
    const float *sa, *sw, *sw1;
    const void *bias;
    const float *scale;                 // of fp16 gradients: of what dG and dU were multiplied by
};

// A warp's 32 rows x 64 bytes of results, staged in shared memory (16-byte piece j of row r at j ^
// (r / 2 & 3): neither side has bank conflicts) and written as whole rows: 16 bytes a lane where
// rows of the result are 16-byte aligned, else a row at a time, an element a lane.
__device__ __forceinline__ void stage_put(uint8_t *stage, int lane, const uint32_t (&x)[16])
{
#pragma unroll
    for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint4 *>(stage + lane * 64 + ((j ^ (lane >> 1 & 3)) << 4)) =
            make_uint4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
}

template <typename E>
__device__ __forceinline__ void stage_flush(const uint8_t *stage, E *c, size_t ld, int rows, int cols,
                                            int lane, bool vec)
{
    constexpr int kPer = 16 / sizeof(E), kCols = 64 / sizeof(E);
    __syncwarp();
    if (vec) {
        const int j = lane & 3;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = i * 8 + (lane >> 2);
            const uint4 v =
                *reinterpret_cast<const uint4 *>(stage + r * 64 + ((j ^ (r >> 1 & 3)) << 4));
            if (r < rows && j * kPer < cols)
                *reinterpret_cast<uint4 *>(c + (size_t)r * ld + j * kPer) = v;
        }
    } else {
        // 4-byte elements fill half a warp's lanes: two rows an instruction. Eight loads, then
        // their stores, from a pointer that moves down the rows.
        constexpr int kAt = 32 / kCols, kBatch = 8;
        const int q = lane % kCols, r0 = lane / kCols;
        const uint8_t *from = stage + r0 * 64 + (q % kPer) * sizeof(E);
        E *to = c + (size_t)r0 * ld + q;
        const size_t down = (size_t)kAt * ld;
        const int full = q < cols ? rows : 0;
#pragma unroll 1
        for (int r = r0; r < 32; r += kAt * kBatch) {
            E v[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int at = r + i * kAt;
                v[i] = *reinterpret_cast<const E *>(from + (at - r0) * 64 +
                                                    (((q / kPer) ^ (at >> 1 & 3)) << 4));
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (r + i * kAt < full) *to = v[i];
                to += down;
            }
        }
    }
    __syncwarp();
}

template <int FORM, bool I8, typename T>
__global__ void __launch_bounds__(kThreads, 1)
tile_kernel(const __grid_constant__ CUtensorMap tm_a0, const __grid_constant__ CUtensorMap tm_a1,
            const __grid_constant__ CUtensorMap tm_b0, const __grid_constant__ CUtensorMap tm_b1,
            const __grid_constant__ CUtensorMap tm_a2, const __grid_constant__ CUtensorMap tm_a3,
            const __grid_constant__ CUtensorMap tm_b2, const Shape shape, const Out out,
            unsigned int *err)
{
    // MN-major operands: B of every gradient, A of the weights' (kBoth: unit by unit, from the unit's
    // place alone, so that the compiler sees one value for the warp: what depends on it goes into
    // descriptors)
    constexpr bool BMN = is_grad(FORM);
    auto a_mn = [&](int j) {
        if constexpr (FORM == kBoth)
            return j * (int)(gridDim.x >> 1) + (int)(blockIdx.x >> 1) >= shape.x.units;
        else return FORM == kDw;
    };
    constexpr int kElems = I8 ? 128 : 64;                      // reduction values per slab
    constexpr uint32_t kCols = 2 * kMaxBn;
    constexpr int ST = ring::stages;
    const int bn = shape.bn, half = bn / 2;
    const int ncol = FORM == kGated ? half : bn;               // result columns of a tile

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(base + ring::bar_off);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + ring::nbars);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    auto full_bar = [&](int s) { return smem_u32(bars + s); };
    auto empty_bar = [&](int s) { return smem_u32(bars + ST + s); };
    auto accf_bar = [&](int b) { return smem_u32(bars + 2 * ST + b); };
    auto acce_bar = [&](int b) { return smem_u32(bars + 2 * ST + 2 + b); };
    const uint32_t final_bar = smem_u32(bars + 2 * ST + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = blockIdx.x & 1;          // in the pair (known to be the same for the CTA)

    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(accf_bar(b), 1);
            mbar_init(acce_bar(b), 2 * kEpiWarps);       // the epilogue warps of both CTAs
        }
        mbar_init(final_bar, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async_smem();
    }
    if (warp == kMmaWarp) {
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
    const uint32_t tx = ring::a_bytes + (BMN ? (half + 63) / 64 * 64 : half) * kSlab;
    // maps, first row of each operand, and place in the reduction of slab i of a unit
    auto second = [&](const Unit &w, int i) {
        return (FORM == kDx || (FORM == kBoth && w.which == 0)) && w.s0 + i >= shape.seg_slabs;
    };
    auto map_a = [&](const Unit &w, int i) {
        if (FORM == kDw || (FORM == kBoth && w.which)) return w.which == 2 ? &tm_a3 : &tm_a2;
        return second(w, i) ? &tm_a1 : &tm_a0;
    };
    auto map_b = [&](const Unit &w, int i) {
        if (FORM == kDw || (FORM == kBoth && w.which)) return &tm_b2;
        return (FORM == kGated ? rank != 0 : second(w, i)) ? &tm_b1 : &tm_b0;
    };
    auto row_a = [&](const Unit &w) { return w.m0 + (int)rank * kRows; };
    auto row_b = [&](const Unit &w) { return FORM == kGated ? w.n0 : w.n0 + (int)rank * half; };
    auto place = [&](const Unit &w, int i) {
        return (w.s0 + i - (second(w, i) ? shape.seg_slabs : 0)) * kElems;
    };
    auto unit_at = [&](int j, Unit *u) {
        return tile::unit_at<FORM>(j, (int)(gridDim.x >> 1), (int)(blockIdx.x >> 1), shape, ncol, u);
    };
    // The first slabs of the operand that is not a token's (weights, or X in the weights'
    // gradients) go to L2 before the kernels ahead on the stream have finished: what one of them
    // still writes is written in L2, so what is read behind grid_wait() is right either way.
    Unit w, w0;
    if (warp == kTmaWarp && unit_at(0, &w0) && lane == 0) {
        for (int i = 0; i < min(w0.ns, ST); ++i) {
            const int r = row_b(w0), k = place(w0, i);
            tma_prefetch_2d(map_b(w0, i), BMN ? r : k, BMN ? k : r);
            if (BMN && half > 64) tma_prefetch_2d(map_b(w0, i), r + 64, k);
        }
    }
    __syncwarp();
    grid_wait();

    // The producer and MMA warps run with all lanes and issue from lane 0, so that addresses and
    // coordinates stay warp-uniform.
    if (warp == kTmaWarp) {
        // ---------------- TMA producer: this CTA's halves of both operands ----------------
        const uint32_t lead = map_to_rank(full_bar(0), 0);     // the first CTA's barriers
        int it = 0, s = 0;
        uint32_t phase = 1;
        bool stop = false;
        for (int j = 0; !stop && unit_at(j, &w); ++j) {
            const int ra = row_a(w), rb = row_b(w);
            const bool amn = a_mn(j);
            // dX: the slabs of its first product, then those of the second
            constexpr bool two = FORM == kDx || FORM == kBoth;
            const int cut = two && !amn ? max(0, min(w.ns, shape.seg_slabs - w.s0)) : w.ns;
            for (int seg = 0; seg < (two ? 2 : 1) && !stop; ++seg) {
                const int i0 = seg ? cut : 0, i1 = seg ? w.ns : cut;
                const CUtensorMap *ma = map_a(w, i0), *mb = map_b(w, i0);
                int k = place(w, i0);
                for (int i = i0; i < i1; ++i, ++it, k += kElems) {
                    const uint32_t sa = smem_u32(base) + s * ring::stage, sb = sa + ring::a_bytes;
                    const uint32_t fb = lead + 8 * s;
                    if (!warp_wait(empty_bar(s), phase, abort_flag, err)) {
                        stop = true;
                        break;
                    }
                    if (lane == 0) {
                        // both CTAs' copies complete on the first CTA's barrier, which expects both
                        if (rank == 0) mbar_expect_tx(full_bar(s), 2 * tx);
                        if (amn) {
                            tma_load_2d_pair(sa, ma, fb, ra, k);
                            tma_load_2d_pair(sa + 8192, ma, fb, ra + 64, k);
                        } else {
                            tma_load_2d_pair(sa, ma, fb, k, ra);
                        }
                        tma_load_2d_pair(sb, mb, fb, BMN ? rb : k, BMN ? k : rb);
                        if (BMN && half > 64) tma_load_2d_pair(sb + 8192, mb, fb, rb + 64, k);
                    }
                    __syncwarp();
                    if (++s == ST) {
                        s = 0;
                        phase ^= 1;
                    }
                }
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
    } else if (warp == kMmaWarp && rank == 0) {
        // ---------------- MMA issue for both CTAs ----------------
        int s = 0;
        uint32_t phase = 0;
        bool stop = false;
        for (int j = 0; !stop && unit_at(j, &w); ++j) {
            const int b = j & 1;
            if (!warp_wait(acce_bar(b), ((j >> 1) & 1) ^ 1, abort_flag, err)) break;
            tc_fence_after();
            const uint32_t dtm = tmem_base + (uint32_t)(b * kMaxBn);
            const bool amn = a_mn(j);
            const uint32_t idesc = amn ? ffn_instr_desc<I8, T, true, BMN>(kTileM, bn)
                                       : ffn_instr_desc<I8, T, false, BMN>(kTileM, bn);
            // 32 bytes of a K-major slab, or 16 rows (2048 B) of an MN-major one, per MMA
            const uint32_t ka = amn ? 128 : 2;
            constexpr uint32_t kb = BMN ? 128 : 2;
            for (int i = 0; i < w.ns; ++i) {
                const uint32_t sa = smem_u32(base) + s * ring::stage, sb = sa + ring::a_bytes;
                const uint64_t da = amn ? sw128_desc_mn(sa, 8192) : sw128_desc(sa);
                const uint64_t db = BMN ? sw128_desc_mn(sb, 8192) : sw128_desc(sb);
                const uint64_t da1 = da + ka, da2 = da1 + ka, da3 = da2 + ka;
                if (!warp_wait(full_bar(s), phase, abort_flag, err)) {
                    stop = true;
                    break;
                }
                tc_fence_after();
                if (lane == 0) {
                    ffn_mma_pair<I8>(dtm, da, db, idesc, i != 0 ? 1u : 0u);
                    ffn_mma_pair<I8>(dtm, da1, db + kb, idesc, 1u);
                    ffn_mma_pair<I8>(dtm, da2, db + 2 * kb, idesc, 1u);
                    ffn_mma_pair<I8>(dtm, da3, db + 3 * kb, idesc, 1u);
                    mma_commit_pair_both(empty_bar(s));
                }
                __syncwarp();
                if (++s == ST) {
                    s = 0;
                    phase ^= 1;
                }
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
    } else if (warp < kEpiWarps) {
        // ---------------- epilogue: lane = row of the result ----------------
        uint8_t *stage = base + ring::out_off + warp * 32 * 64;
        float *col = reinterpret_cast<float *>(base + ring::col_off) + warp * 64;
        const int quarter = warp & 3, first = 32 * (warp >> 2);
        const int N = shape.N;
        const bool vec = (N & 7) == 0;
        // A lane's row scale, and the factors of column c + lane of a tile: the two scales of
        // kGated, or scale and bias. A tile's first ones are loaded while the tile before it is
        // written.
        float sa = 0.f, f0 = 0.f, f1 = 0.f;
        auto factors = [&](const Unit &w, int c) {
            const int n = min(w.n0 + min(c + lane, ncol - 1), N - 1);
            f0 = ld_behind_f32(out.sw + n);
            if constexpr (FORM == kGated) f1 = ld_behind_f32(out.sw1 + n);
            else f1 = out.bias ? ld_behind_16<T>(static_cast<const T *>(out.bias) + n) : 0.f;
        };
        auto first_row = [&](const Unit &w) { return w.m0 + (int)rank * kRows + quarter * 32; };
        auto row_scale = [&](const Unit &w) {
            const int m = first_row(w) + lane;
            return m < shape.x.M ? ld_behind_f32(out.sa + m) : 0.f;
        };
        Unit next;
        bool more = unit_at(0, &next);
        float sa_next = 0.f, back = 1.f;
        if constexpr (is_grad(FORM) && std::is_same<T, __half>::value) back = ld_behind_f32(out.scale);
        if constexpr (I8) {
            sa_next = row_scale(next);
            factors(next, first);
        }
        for (int j = 0; more; ++j) {
            w = next;
            const bool weights = a_mn(j);
            const int M = weights ? shape.w.M : shape.x.M;
            const int parts = weights ? shape.w.parts : shape.x.parts;
            const int b = j & 1;
            const int m = first_row(w);                               // the warp's first row
            const int rows = min(32, M - m);
            const int nc = min(ncol, N - w.n0);
            sa = sa_next;
            more = unit_at(j + 1, &next);
            if constexpr (I8) sa_next = row_scale(next);
            bool ok = mbar_wait(accf_bar(b), (j >> 1) & 1, abort_flag, err);
            tc_fence_after();
            ok = __all_sync(0xffffffffu, ok && !*abort_flag);
            if (!ok) break;
            const uint32_t tm = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(b * kMaxBn);
            if (rows > 0 && first < nc) {
#pragma unroll 1
                for (int c = first; c < nc; c += 64) {
                    uint32_t v[32], z[32];
                    tmem_ld32(tm + c, v);
                    if constexpr (FORM == kGated) tmem_ld32(tm + ncol + c, z);
                    if constexpr (I8) {
                        col[lane] = f0;
                        col[32 + lane] = f1;
                        __syncwarp();
                        if (c + 64 < nc) factors(w, c + 64);
                        else factors(next, first);
                    }
                    tmem_wait_ld();
                    const int cols = nc - c;
                    auto write = [&](const uint32_t (&x)[16], void *to) {
                        T *dst = static_cast<T *>(to) + (size_t)m * N + w.n0 + c;
                        stage_put(stage, lane, x);
                        if (vec || (N & 1)) stage_flush(stage, dst, N, rows, cols, lane, vec);
                        else     // pairs of elements
                            stage_flush(stage, reinterpret_cast<uint32_t *>(dst), N / 2, rows,
                                        cols / 2, lane, false);
                    };
                    // int32 sums to fp32, scaled by their row and then their column, as the
                    // definition has it; then the bias
                    if constexpr (I8) {
                        auto scale = [&](uint32_t (&x)[32], int at) {
#pragma unroll
                            for (int q = 0; q < 8; ++q) {
                                const float4 f = reinterpret_cast<const float4 *>(col)[at / 4 + q];
                                const float fs[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    x[4 * q + e] = __float_as_uint(__fmul_rn(
                                        __fmul_rn(__int2float_rn((int)x[4 * q + e]), sa), fs[e]));
                            }
                        };
                        scale(v, 0);
                        if constexpr (FORM == kGated) {
                            scale(z, 32);
                        } else if (out.bias) {
#pragma unroll
                            for (int q = 0; q < 8; ++q) {
                                const float4 f = reinterpret_cast<const float4 *>(col)[8 + q];
                                const float fs[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    v[4 * q + e] = __float_as_uint(
                                        __fadd_rn(__uint_as_float(v[4 * q + e]), fs[e]));
                            }
                        }
                    }
                    if constexpr (is_grad(FORM) && std::is_same<T, __half>::value) {
#pragma unroll
                        for (int q = 0; q < 32; ++q)
                            v[q] = __float_as_uint(__uint_as_float(v[q]) * back);
                    }
                    uint32_t hw[16];
                    if constexpr (FORM == kGated) {
                        uint32_t gw[16], uw[16];
                        auto gate = [&](auto act) {
                            constexpr int ACT = decltype(act)::value;
#pragma unroll
                            for (int q = 0; q < 16; ++q) {
                                const float g0 = __uint_as_float(v[2 * q]);
                                const float g1 = __uint_as_float(v[2 * q + 1]);
                                const float u0 = __uint_as_float(z[2 * q]);
                                const float u1 = __uint_as_float(z[2 * q + 1]);
                                hw[q] = pack2<T>(act_value<ACT>(g0) * u0, act_value<ACT>(g1) * u1);
                                gw[q] = pack2<T>(g0, g1);
                                uw[q] = pack2<T>(u0, u1);
                            }
                        };
                        if (shape.act == QG_ACT_SILU) gate(Const<QG_ACT_SILU>{});
                        else if (shape.act == QG_ACT_GELU) gate(Const<QG_ACT_GELU>{});
                        else gate(Const<QG_ACT_GELU_TANH>{});
                        write(hw, out.c0);
                        if constexpr (!I8) {
                            if (out.c1) {
                                write(gw, out.c1);
                                write(uw, out.c2);
                            }
                        }
                    } else if (is_grad(FORM) && parts > 1) {
                        const int part = w.which == 2 ? parts + w.part : w.part;
                        float *dst = (weights ? out.part_w : out.part_x) +
                                     ((size_t)part * M + m) * N + w.n0 + c;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
#pragma unroll
                            for (int q = 0; q < 16; ++q) hw[q] = v[16 * h + q];
                            stage_put(stage, lane, hw);
                            stage_flush(stage, dst + 16 * h, N, rows, cols - 16 * h, lane, true);
                        }
                    } else {
#pragma unroll
                        for (int q = 0; q < 16; ++q)
                            hw[q] = pack2<T>(__uint_as_float(v[2 * q]), __uint_as_float(v[2 * q + 1]));
                        write(hw, is_grad(FORM) && w.which
                                      ? (w.which == 1 ? out.c1 : out.c2)
                                      : out.c0);
                    }
                    if constexpr (I8) __syncwarp();       // the column factors are read
                }
            }
            else if constexpr (I8) factors(next, first);
            // The accumulator goes back to the MMA warp (of the pair's first CTA). The order that this
            // needs is of tcgen05 operations alone: the reads of TMEM are complete behind their
            // wait::ld, fence::before_thread_sync orders them before the arrival, and the MMA warp's
            // fence::after_thread_sync its MMAs behind the barrier. That is PTX's rule for tcgen05
            // across threads, and it asks for no release, which would wait for the results' stores too.
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(map_to_rank(acce_bar(b), 0));
        }
    }

    tc_fence_before();
    __syncwarp();
    cluster_sync();
    if (warp == kMmaWarp) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                     "r"(kCols)
                     : "memory");
    }
}

// ---- host side -------------------------------------------------------------------------------------

template <int FORM, bool I8, typename T>
cudaError_t launch_tile(const Matrix &a0, const Matrix &a1, const Matrix &b0, const Matrix &b1,
                        const Matrix &b2, Shape shape, const Out &out, unsigned int *err,
                        cudaStream_t stream)
{
    auto kern = tile_kernel<FORM, I8, T>;
    // per device: the shared-memory opt-in and the number of pairs that fit at once
    static std::mutex mu;
    static int pairs_of[64] = {};
    int dev = 0, pairs = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (!pairs_of[dev]) {
            cudaError_t e = cudaFuncSetAttribute(
                kern, cudaFuncAttributeMaxDynamicSharedMemorySize, ring::total);
            if (e != cudaSuccess) return e;
            cudaLaunchConfig_t cfg = {};
            cudaLaunchAttribute attr[1];
            cfg.gridDim = dim3(2);
            cfg.blockDim = dim3(kThreads);
            cfg.dynamicSmemBytes = ring::total;
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
    if (shape.x.units < 0 || shape.w.units < 0) return cudaErrorInvalidValue;    // beyond an int
    const long long units = (long long)shape.x.units + shape.w.units;
    pairs = (int)std::min<long long>(units, pairs);
    share_units(&shape, pairs);
    CUtensorMap ta0, ta1, ta2, ta3, tb0, tb1, tb2;
    // MN-major operands arrive in boxes of 64 rows
    const int b_rows = is_grad(FORM) ? 64 : shape.bn / 2;
    if (!map_of<I8, T>(&ta0, a0, kRows) || !map_of<I8, T>(&tb0, b0, b_rows))
        return cudaErrorInvalidValue;
    ta1 = ta2 = ta3 = ta0;
    tb1 = tb2 = tb0;
    if (a1.p != a0.p && !map_of<I8, T>(&ta1, a1, kRows)) return cudaErrorInvalidValue;
    if (b1.p != b0.p && !map_of<I8, T>(&tb1, b1, b_rows)) return cudaErrorInvalidValue;
    if (is_grad(FORM) && (!map_of<I8, T>(&ta2, a0, 64) || !map_of<I8, T>(&ta3, a1, 64) ||
                          !map_of<I8, T>(&tb2, b2, b_rows)))
        return cudaErrorInvalidValue;
    return launch_dependent(kern, dim3(2 * pairs), dim3(kThreads), ring::total, 2, stream, ta0, ta1,
                            tb0, tb1, ta2, ta3, tb2, shape, out, err);
}

// Sum of the parts in order, rounded to 16 bits: [which][part][n] -> c0, c1 [n], n a multiple of 8
template <typename T>
__global__ void __launch_bounds__(256)
join_kernel(const float *part, T *c0, T *c1, int parts, long long n)
{
    grid_release();
    grid_wait();
    const long long at = ((long long)blockIdx.x * 256 + threadIdx.x) * 8;
    if (at >= n) return;
    const float *src = part + (size_t)blockIdx.y * parts * n + at;
    float r[8] = {};
    // two parts' loads in flight (with four, at 80 registers, the CTAs do not fit beside those of the
    // kernel ahead); the sum in the parts' order
    for (int p = 0; p < parts; p += 2, src += 2 * n) {
        uint4 v[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (p + i < parts) {
                v[i][0] = ld_behind_v4(src + i * n);
                v[i][1] = ld_behind_v4(src + i * n + 4);
            }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (p + i < parts) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    r[4 * h] += __uint_as_float(v[i][h].x);
                    r[4 * h + 1] += __uint_as_float(v[i][h].y);
                    r[4 * h + 2] += __uint_as_float(v[i][h].z);
                    r[4 * h + 3] += __uint_as_float(v[i][h].w);
                }
            }
    }
    *reinterpret_cast<uint4 *>((blockIdx.y ? c1 : c0) + at) =
        make_uint4(pack2<T>(r[0], r[1]), pack2<T>(r[2], r[3]), pack2<T>(r[4], r[5]),
                   pack2<T>(r[6], r[7]));
}

template <typename T>
cudaError_t join_parts(const float *part, void *c0, void *c1, const Work &k, int N,
                       cudaStream_t stream)
{
    const long long n = (long long)k.M * N;
    const dim3 grid((unsigned)((n / 8 + 255) / 256), c1 ? 2 : 1);
    return launch_dependent(join_kernel<T>, grid, dim3(256), 0, 1, stream, part,
                            static_cast<T *>(c0), static_cast<T *>(c1), k.parts, n);
}

} // namespace

cudaError_t launch_tile_scaled(const ScaledProblem &p, unsigned int *err, cudaStream_t stream)
{
    const uint64_t K = p.K;
    const bool gated = p.W1 != nullptr;
    const Matrix a{p.A, (uint64_t)p.M, K, K}, w{p.W, (uint64_t)p.N, K, K};
    const Matrix w1{gated ? p.W1 : p.W, (uint64_t)p.N, K, K};
    const Out out{p.C, nullptr, nullptr, nullptr, nullptr, p.sa, p.sw, p.sw1, p.bias, nullptr};
    const int slabs = ceil_div(p.K, 128);
    const int bn = plan_tiles(p.M, p.N, gated, kStepI8, slabs).bn;
    const Shape shape = shape_of(p.M, p.N, bn, gated ? bn / 2 : bn, slabs, p.act);
    QG_DISPATCH_16(p.dtype, T, {
        if (gated) return launch_tile<kGated, true, T>(a, a, w, w1, w, shape, out, err, stream);
        return launch_tile<kScaled, true, T>(a, a, w, w1, w, shape, out, err, stream);
    });
}

cudaError_t launch_tile_gated(const GatedProblem &p, unsigned int *err, cudaStream_t stream)
{
    const uint64_t K = p.K, pitch = K * 2;
    const Matrix x{p.X, (uint64_t)p.M, K, pitch};
    const Matrix g{p.Wg, (uint64_t)p.F, K, pitch}, u{p.Wu, (uint64_t)p.F, K, pitch};
    Out out = {};
    out.c0 = p.H;
    out.c1 = p.G;
    out.c2 = p.U;
    const int slabs = ceil_div(p.K, 64);
    const int bn = plan_tiles(p.M, p.F, true, kStep16, slabs).bn;
    const Shape shape = shape_of(p.M, p.F, bn, bn / 2, slabs, p.act);
    QG_DISPATCH_16(p.dtype, T, {
        return launch_tile<kGated, false, T>(x, x, g, u, g, shape, out, err, stream);
    });
}

cudaError_t launch_tile_grad(const GatedGrad &p, unsigned int *err, cudaStream_t stream)
{
    const GradPlan &plan = p.plan;
    const bool dx = !plan.few && p.dX, dw = p.dWg != nullptr;
    if (!dx && !dw) return cudaSuccess;
    const uint64_t M = p.M, F = p.F, K = p.K;
    const Matrix dg{p.dG, M, F, (uint64_t)p.Fp * 2}, du{p.dU, M, F, (uint64_t)p.Fp * 2};
    const Matrix wg{p.Wg, F, K, K * 2}, wu{p.Wu, F, K, K * 2}, x{p.X, M, K, K * 2};
    const bool both = plan.together && dx && dw;
    const Shape sx = dx ? grad_shape(plan.x, p.M, p.F, p.K, true, both) : Shape{};
    const Shape sw = grad_shape(plan.w, p.M, p.F, p.K, false, dw);
    Out out = {};
    out.c0 = p.dX;
    out.c1 = p.dWg;
    out.c2 = p.dWu;
    out.part_x = p.part;
    out.part_w = p.part;
    out.scale = p.scale;
    if (!plan.few && plan.x.parts_x > 1) out.part_w += (size_t)plan.x.parts_x * p.M * p.K;
    QG_DISPATCH_16(p.dtype, T, {
        cudaError_t e = cudaSuccess;
        if (both) {
            e = launch_tile<kBoth, false, T>(dg, du, wg, wu, x, sx, out, err, stream);
        } else {
            if (dx) e = launch_tile<kDx, false, T>(dg, du, wg, wu, x, sx, out, err, stream);
            if (e == cudaSuccess && dw)
                e = launch_tile<kDw, false, T>(dg, du, wg, wu, x, sw, out, err, stream);
        }
        if (e == cudaSuccess && dx && sx.x.parts > 1)
            e = join_parts<T>(out.part_x, p.dX, nullptr, sx.x, p.K, stream);
        if (e == cudaSuccess && dw && sw.w.parts > 1)
            e = join_parts<T>(out.part_w, p.dWg, p.dWu, sw.w, p.K, stream);
        return e;
    });
}

} // namespace qg
