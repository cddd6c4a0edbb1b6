// Few tokens: tensor-core kernel of the scaled W8A8 matmul, the gated forward products and dX.
//
// Bound: HBM (every weight is read once, 2 M operations a byte). A CTA owns 128 weight rows (the
// MMA's M side; 64 of the gate and the same 64 of up for kGated) and BN = 16 .. 128 tokens (its N
// side): with few tokens an MMA costs the same for any N up to 128, so the weights go where a
// whole 16 KB slab is consumed by four MMAs (about 40 B a clock, twice what HBM delivers to an
// SM). Two CTAs share an SM, 100 KB of TMA ring each, which hides one CTA's start and end behind
// the other's stream.
//
// Split reduction: the CTAs of a cluster (1, 2, 4 or 8) take consecutive parts of the reduction of
// one tile, so that a small weight matrix still occupies every SM. Each leaves its partial tile
// in its own shared memory as [token][weight row]; after a cluster barrier every CTA adds its share of
// the tile over the cluster (distributed shared memory, parts in order: the same bits every run),
// applies scales, bias or activation and writes runs of weight rows of one token. No workspace, no
// atomics, one launch.
#include <algorithm>
#include <mutex>

#include "ffn.cuh"
#include "sm100.cuh"

namespace qg {
namespace {

enum Form { kScaled, kGated, kDx };

constexpr int kThreads = 192;          // warps 0-3 accumulator and output, 4 TMA, 5 MMA
constexpr int kRows = 128, kSlab = 128;

template <int BN> struct Ring {
    static constexpr int w_bytes = kRows * kSlab;
    static constexpr int stage = w_bytes + BN * kSlab;
    static constexpr int stages = BN == 16 ? 6 : (BN == 32 ? 5 : (BN == 64 ? 4 : 3));
    static constexpr int bar_off = stages * stage;
    static constexpr int nbars = 2 * stages + 1;
    static constexpr int total = 1024 + bar_off + nbars * 8 + 16;
    static_assert(BN * kRows * 4 <= bar_off, "the partial tile reuses the ring");
    static_assert(2 * (total + 1024) <= 228 * 1024, "two CTAs an SM");
};

struct Shape {
    int M, N;               // tokens; columns of the result
    int seg_slabs, slabs;   // slabs of the reduction: of one product, of all
    int act;
};

struct Out {
    void *c0, *c1, *c2;
    const float *sa, *sw, *sw1;
    const void *bias;
};

template <bool I8>
__device__ __forceinline__ void mma_one(uint32_t dtm, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t accumulate)
{
    if constexpr (I8)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(dtm),
                     "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(dtm),
                     "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
                     : "memory");
}

template <bool I8, typename T, int BN, bool AMN> constexpr uint32_t instr_desc()
{
    const uint32_t in = I8 ? 1u : (std::is_same<T, __nv_bfloat16>::value ? 1u : 0u);
    return (I8 ? 2u : 1u) << 4 | in << 7 | in << 10 | (AMN ? 1u : 0u) << 15 | (uint32_t)(BN >> 3) << 17 |
           (uint32_t)(kRows >> 4) << 24;
}

__device__ __forceinline__ uint4 ld_cluster_v4(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared::cluster.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// four results of one token, columns n .. n + 3
template <typename T>
__device__ __forceinline__ void store4(T *row, int n, int N, const float (&r)[4])
{
    if ((N & 3) == 0) {
        if (n < N)
            *reinterpret_cast<uint2 *>(row + n) = make_uint2(pack2<T>(r[0], r[1]), pack2<T>(r[2], r[3]));
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (n + e < N) row[n + e] = from_f32<T>(r[e]);
    }
}

template <int FORM, bool I8, typename T, int BN>
__global__ void __launch_bounds__(kThreads, 2)
small_kernel(const __grid_constant__ CUtensorMap tm_w0, const __grid_constant__ CUtensorMap tm_w1,
             const __grid_constant__ CUtensorMap tm_x0, const __grid_constant__ CUtensorMap tm_x1,
             const Shape shape, const Out out, unsigned int *err)
{
    using L = Ring<BN>;
    using Acc = typename std::conditional<I8, int, float>::type;
    constexpr bool AMN = FORM == kDx;
    constexpr int NROW = FORM == kGated ? kRows / 2 : kRows;      // result columns of a tile
    constexpr int kElems = I8 ? 128 : 64;
    constexpr uint32_t kIdesc = instr_desc<I8, T, BN, AMN>();
    constexpr uint32_t kCols = BN < 32 ? 32u : (uint32_t)BN;
    constexpr int ST = L::stages;

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(base + L::bar_off);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + L::nbars);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    auto full_bar = [&](int s) { return smem_u32(bars + s); };
    auto empty_bar = [&](int s) { return smem_u32(bars + ST + s); };
    const uint32_t done_bar = smem_u32(bars + 2 * ST);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cl = (int)cluster_size(), rank = (int)cluster_rank();
    // tiles of the same weight rows are neighbours: those rows come from memory once
    const int tile = (int)(blockIdx.x / cl), tiles_t = (shape.M + BN - 1) / BN;
    const int n0 = tile / tiles_t * NROW;
    const int t0 = tile % tiles_t * BN;
    // this CTA's part of the reduction
    const int s0 = (int)((long long)shape.slabs * rank / cl);
    const int ns = (int)((long long)shape.slabs * (rank + 1) / cl) - s0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        mbar_init(done_bar, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async_smem();
    }
    if (threadIdx.x == 32) {
        prefetch_map(&tm_w0);
        prefetch_map(&tm_x0);
        if (FORM != kScaled) prefetch_map(&tm_w1);
        if (FORM == kDx) prefetch_map(&tm_x1);
    }
    if (warp == 5) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(tmem_holder)),
                     "r"(kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    // The first slabs of weights go to L2 before the kernels ahead on the stream have finished: a
    // weight that one of them still writes is written in L2, so what is read behind grid_wait() is
    // right either way.
    auto load_w = [&](int it, auto &&copy) {
        const int slab = s0 + it;
        const bool second = FORM == kDx && slab >= shape.seg_slabs;
        const int k = (second ? slab - shape.seg_slabs : slab) * kElems;
        if constexpr (FORM == kDx) {
            copy(0, second ? &tm_w1 : &tm_w0, n0, k);
            copy(8192, second ? &tm_w1 : &tm_w0, n0 + 64, k);
        } else if constexpr (FORM == kGated) {
            copy(0, &tm_w0, k, n0);
            copy(8192, &tm_w1, k, n0);
        } else {
            copy(0, &tm_w0, k, n0);
        }
    };
    if (warp == 4 && lane == 0)
        for (int it = 0; it < min(ns, ST); ++it)
            load_w(it, [](int, const CUtensorMap *map, int x, int y) { tma_prefetch_2d(map, x, y); });
    __syncwarp();
    grid_wait();

    if (warp == 4) {
        // ---------------- TMA producer ----------------
        int it = 0;
        for (; it < ns; ++it) {
            const int s = it % ST;
            if (!warp_wait(empty_bar(s), ((it / ST) & 1) ^ 1, abort_flag, err)) break;
            if (lane == 0) {
                const int slab = s0 + it;
                const bool second = FORM == kDx && slab >= shape.seg_slabs;
                const int k = (second ? slab - shape.seg_slabs : slab) * kElems;
                const uint32_t sw = smem_u32(base + s * L::stage), sx = sw + L::w_bytes;
                mbar_expect_tx(full_bar(s), L::stage);
                load_w(it, [&](int at, const CUtensorMap *map, int x, int y) {
                    tma_load_2d(sw + at, map, full_bar(s), x, y);
                });
                tma_load_2d(sx, second ? &tm_x1 : &tm_x0, full_bar(s), k, t0);
            }
            __syncwarp();
        }
        // every load is on its way: the next kernel may start (and fetch its weights into L2; any
        // earlier, what it fetches is evicted again by what this kernel still streams)
        grid_release();
        // every copy this warp started must land before the ring is reused or the CTA exits
        for (int i = max(0, it - ST); i < it; ++i) {
            int dummy_abort = 0;
            mbar_wait(full_bar(i % ST), (i / ST) & 1, &dummy_abort, nullptr);
        }
    } else if (warp == 5) {
        // ---------------- MMA issue ----------------
        for (int it = 0; it < ns; ++it) {
            const int s = it % ST;
            if (!warp_wait(full_bar(s), (it / ST) & 1, abort_flag, err)) break;
            tc_fence_after();
            const uint32_t sw = smem_u32(base + s * L::stage);
            const uint64_t dw = AMN ? sw128_desc_mn(sw, 8192) : sw128_desc(sw);
            const uint64_t dx = sw128_desc(sw + L::w_bytes);
            constexpr int kw = AMN ? 128 : 2;
            if (lane == 0) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_one<I8>(tmem_base, dw + kw * k, dx + 2 * k, kIdesc, (it | k) != 0 ? 1u : 0u);
                mma_commit(empty_bar(s));
            }
            __syncwarp();
        }
        if (lane == 0) mma_commit(done_bar);
        __syncwarp();
        int dummy_abort = 0;
        mbar_wait(done_bar, 0, &dummy_abort, nullptr);
    }
    // The accumulator to shared memory as [token][weight row]: lane = weight row. A CTA whose waits
    // gave up has raised the error word; it goes through the same steps so that nobody hangs.
    Acc *part = reinterpret_cast<Acc *>(base);
    const int tokens = min(BN, shape.M - t0);
    if (warp < 4) mbar_wait(done_bar, 0, abort_flag, err);
    __syncthreads();               // the copies have landed and the MMAs have read them
    if (warp < 4) {
        tc_fence_after();
        const uint32_t tm = tmem_base + ((uint32_t)(warp * 32) << 16);
#pragma unroll 1
        for (int c = 0; c < tokens; c += 16) {
            uint32_t v[16];
            tmem_ld16(tm + c, v);
#pragma unroll
            for (int q = 0; q < 16; ++q)
                reinterpret_cast<uint32_t *>(part)[(c + q) * kRows + threadIdx.x] = v[q];
        }
        tc_fence_before();
    }
    __syncwarp();
    if (cl > 1) cluster_sync();
    else __syncthreads();

    // This CTA's share of the tile: (token, 4 columns) items, tokens outermost
    {
        constexpr int kPer = NROW / 4;
        const int items = tokens * kPer;
        const int i0 = items * rank / cl, i1 = items * (rank + 1) / cl;
        const uint32_t mine = smem_u32(part);
        const int N = shape.N;
        auto total = [&](int token, int row, Acc (&r)[4]) {
            const uint32_t at = mine + (uint32_t)(token * kRows + row) * 4;
            uint4 v[8];
#pragma unroll
            for (int p = 0; p < 8; ++p)          // all in flight before the first is added
                v[p] = p < cl ? ld_cluster_v4(map_to_rank(at, p)) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int e = 0; e < 4; ++e) r[e] = 0;
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                const uint32_t x[4] = {v[p].x, v[p].y, v[p].z, v[p].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (I8) r[e] += (int)x[e];
                    else r[e] += __uint_as_float(x[e]);
                }
            }
        };
        for (int i = i0 + threadIdx.x; i < i1; i += kThreads) {
            const int t = i / kPer, row = (i % kPer) * 4;
            const int m = t0 + t, n = n0 + row;
            if (n >= N) continue;
            const size_t at = (size_t)m * N;
            Acc a[4];
            total(t, row, a);
            float r[4];
            const float sa = I8 ? out.sa[m] : 0.f;
            if constexpr (FORM == kGated) {
                Acc b[4];
                total(t, NROW + row, b);
                float g[4], u[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (I8) {
                        const int c = min(n + e, N - 1);
                        g[e] = __fmul_rn(__fmul_rn(__int2float_rn(a[e]), sa), out.sw[c]);
                        u[e] = __fmul_rn(__fmul_rn(__int2float_rn(b[e]), sa), out.sw1[c]);
                    } else {
                        g[e] = a[e];
                        u[e] = b[e];
                    }
                }
                QG_DISPATCH_ACT(shape.act, ACT, {
#pragma unroll
                    for (int e = 0; e < 4; ++e) r[e] = act_value<ACT>(g[e]) * u[e];
                });
                store4(static_cast<T *>(out.c0) + at, n, N, r);
                if constexpr (!I8) {
                    if (out.c1) {
                        store4(static_cast<T *>(out.c1) + at, n, N, g);
                        store4(static_cast<T *>(out.c2) + at, n, N, u);
                    }
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (I8) {
                        const int c = min(n + e, N - 1);
                        r[e] = __fmul_rn(__fmul_rn(__int2float_rn(a[e]), sa), out.sw[c]);
                        if (out.bias) r[e] = __fadd_rn(r[e], to_f32(static_cast<const T *>(out.bias)[c]));
                    } else {
                        r[e] = a[e];
                    }
                }
                store4(static_cast<T *>(out.c0) + at, n, N, r);
            }
        }
    }
    __syncwarp();
    // no CTA may leave while another reads its shared memory
    if (cl > 1) cluster_sync();
    else __syncthreads();
    if (warp == 5) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(kCols)
                     : "memory");
    }
}

// ---- host side -------------------------------------------------------------------------------------

struct Matrix {
    const void *p;
    uint64_t rows, cols, pitch;
};

template <bool I8, typename T> bool map_of(CUtensorMap *m, const Matrix &x, int box_rows)
{
    const CUtensorMapDataType dt = I8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                      : (std::is_same<T, __nv_bfloat16>::value ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                                     : CU_TENSOR_MAP_DATA_TYPE_FLOAT16);
    return make_map(m, dt, x.p, x.cols, x.rows, x.pitch, I8 ? 128 : 64, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Clusters of 1, 2, 4 and 8 CTAs that run at once on the device (two CTAs an SM; larger clusters
// leave SMs of a partly filled processing cluster idle: 296, 148, 71 and 33 on a B200).
struct Slots {
    int clusters[4];
};

// Parts of the reduction: the most, up to 8, with which every tile's cluster still runs at once and a
// part keeps four slabs (a shorter stream does not pay for the barrier that joins the parts).
int parts_of(long long tiles, int slabs, const Slots &slots)
{
    int parts = 1;
    for (int i = 1; i < 4; ++i)
        if (tiles <= slots.clusters[i] && slabs >= 4 << i) parts = 1 << i;
    return parts;
}

template <typename Kern> cudaError_t slots_of(Kern kern, int smem, Slots *slots)
{
    for (int i = 0; i < 4; ++i) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        cfg.gridDim = dim3(1 << i);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = smem;
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 1 << i;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        const cudaError_t e = cudaOccupancyMaxActiveClusters(&slots->clusters[i], kern, &cfg);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <int FORM, bool I8, typename T, int BN>
cudaError_t launch_bn(const Matrix &w0, const Matrix &w1, const Matrix &x0, const Matrix &x1,
                      const Shape &shape, const Out &out, unsigned int *err, cudaStream_t stream)
{
    using L = Ring<BN>;
    auto kern = small_kernel<FORM, I8, T, BN>;
    static std::mutex mu;
    static Slots slots_dev[64] = {};
    Slots slots;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (!slots_dev[dev].clusters[0]) {
            cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::total);
            if (e == cudaSuccess) e = slots_of(kern, L::total, &slots);
            if (e != cudaSuccess) return e;
            slots_dev[dev] = slots;
        }
        slots = slots_dev[dev];
    }
    const int tiles_n = ceil_div(shape.N, FORM == kGated ? 64 : 128), tiles_t = ceil_div(shape.M, BN);
    const long long tiles = (long long)tiles_n * tiles_t;
    const int parts = parts_of(tiles, shape.slabs, slots);
    if (tiles * parts > 0x7fffffffLL) return cudaErrorInvalidValue;
    // weights: 128 rows, 64 of each for kGated, 64 rows of the reduction for kDx
    CUtensorMap tw0, tw1, tx0, tx1;
    const int wbox = FORM == kScaled ? 128 : 64;
    if (!map_of<I8, T>(&tw0, w0, wbox) || !map_of<I8, T>(&tx0, x0, BN)) return cudaErrorInvalidValue;
    tw1 = tw0;
    tx1 = tx0;
    if (w1.p != w0.p && !map_of<I8, T>(&tw1, w1, wbox)) return cudaErrorInvalidValue;
    if (x1.p != x0.p && !map_of<I8, T>(&tx1, x1, BN)) return cudaErrorInvalidValue;
    return launch_dependent(kern, dim3((unsigned)(tiles * parts)), dim3(kThreads), L::total, parts, stream,
                            tw0, tw1, tx0, tx1, shape, out, err);
}

template <int FORM, bool I8, typename T>
cudaError_t launch_small(const Matrix &w0, const Matrix &w1, const Matrix &x0, const Matrix &x1,
                         const Shape &shape, const Out &out, unsigned int *err, cudaStream_t stream)
{
    if (shape.M <= 16) return launch_bn<FORM, I8, T, 16>(w0, w1, x0, x1, shape, out, err, stream);
    if (shape.M <= 32) return launch_bn<FORM, I8, T, 32>(w0, w1, x0, x1, shape, out, err, stream);
    if (shape.M <= 64) return launch_bn<FORM, I8, T, 64>(w0, w1, x0, x1, shape, out, err, stream);
    return launch_bn<FORM, I8, T, 128>(w0, w1, x0, x1, shape, out, err, stream);
}

} // namespace

// Estimate for a B200, from the device times of 100 to 1024 tokens at 512 to 11008 columns and 2048 to
// 11008 values of reduction: with 128 tokens a tile an SM takes a slab in 0.5 us alone and two
// in 0.75 us (32 KB each, at what L2 delivers to an SM).
double small_us(int M, int N, bool gated, int slabs)
{
    const Slots b200 = {{296, 148, 71, 33}};
    const long long tiles = (long long)ceil_div(N, gated ? 64 : 128) * ceil_div(M, 128);
    const int parts = parts_of(tiles, slabs, b200);
    const long long ctas = tiles * parts;
    const double waves = ctas <= 296 ? 1.0 : ctas / 296.0;
    return 5.5 + waves * ceil_div(slabs, parts) * (ctas <= 148 ? 0.5 : 0.75);
}

cudaError_t launch_small_scaled(const ScaledProblem &p, unsigned int *err, cudaStream_t stream)
{
    const uint64_t K = p.K;
    const Matrix a{p.A, (uint64_t)p.M, K, K}, w{p.W, (uint64_t)p.N, K, K};
    const Matrix w1{p.W1 ? p.W1 : p.W, (uint64_t)p.N, K, K};
    const Out out{p.C, nullptr, nullptr, p.sa, p.sw, p.sw1, p.bias};
    const int slabs = ceil_div(p.K, 128);
    const Shape shape{p.M, p.N, slabs, slabs, p.act};
    QG_DISPATCH_16(p.dtype, T, {
        if (p.W1) return launch_small<kGated, true, T>(w, w1, a, a, shape, out, err, stream);
        return launch_small<kScaled, true, T>(w, w, a, a, shape, out, err, stream);
    });
}

cudaError_t launch_small_gated(const GatedProblem &p, unsigned int *err, cudaStream_t stream)
{
    const uint64_t K = p.K, pitch = K * 2;
    const Matrix x{p.X, (uint64_t)p.M, K, pitch}, g{p.Wg, (uint64_t)p.F, K, pitch}, u{p.Wu, (uint64_t)p.F, K, pitch};
    const Out out{p.H, p.G, p.U, nullptr, nullptr, nullptr, nullptr};
    const int slabs = ceil_div(p.K, 64);
    const Shape shape{p.M, p.F, slabs, slabs, p.act};
    QG_DISPATCH_16(p.dtype, T, {
        return launch_small<kGated, false, T>(g, u, x, x, shape, out, err, stream);
    });
}

cudaError_t launch_small_dx(const GatedGrad &p, unsigned int *err, cudaStream_t stream)
{
    const uint64_t M = p.M, F = p.F, K = p.K;
    const Matrix dg{p.dG, M, F, (uint64_t)p.Fp * 2}, du{p.dU, M, F, (uint64_t)p.Fp * 2};
    const Matrix wg{p.Wg, F, K, K * 2}, wu{p.Wu, F, K, K * 2};
    const Out out{p.dX, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr};
    const int slabs = ceil_div(p.F, 64);
    const Shape shape{p.M, p.K, slabs, 2 * slabs, 0};
    QG_DISPATCH_16(p.dtype, T, {
        return launch_small<kDx, false, T>(wg, wu, dg, du, shape, out, err, stream);
    });
}

} // namespace qg
