// Few tokens: tensor-core kernel of the scaled W8A8 matmul, the gated forward products and dX.
//
// Bound: HBM (every weight is read once, 2 M operations a byte). A CTA owns up to 128 tokens and R
// rows of the weights (for kGated R / 2 of the gate and the same of up). R is any multiple of four,
// so that the weights divide evenly over the SMs: tiles of 64 gate and up rows left 24 of 148 SMs
// with twice the others' work at 11008 columns. The ring of 108 KB covers the memory's latency (44
// GB/s x 2 us) and leaves room for a second CTA: of this kernel, or of the next on the stream,
// which sets itself up while this one ends.
//
// Orientation (WM): up to 64 tokens the weights are the MMA's M side, in one or two blocks of 128,
// and the tokens its N side; above, the tokens are the M side and the weights the N side. Unused
// rows of the M side hold whatever follows in shared memory and reach no result, but the tensor
// core multiplies them: with 16 tokens in an M of 128 the SMs drew enough power to fall from 1.8 to
// 1.45 GHz within a tenth of a second, and the stream of weights slowed from 32.4 to 36 us with
// them. An MMA takes about 100 cycles for up to 128 rows of 32 bytes by up to 128, 128 cycles by
// 256: 40 to 64 B of weights a clock, against the 24 B that HBM delivers to an SM.
//
// Split reduction: the CTAs of a cluster (1, 2, 4 or 8) take consecutive parts of the reduction of
// one tile, so that a small weight matrix still occupies the device. Each leaves its partial tile
// in its own shared memory as [token][weight row]; after a cluster barrier every CTA adds its share
// of the columns over the cluster (distributed shared memory, parts in order: the same bits every
// run), applies scales, bias or activation and writes runs of columns of one token. No workspace,
// no atomics, one launch.
//
// Device time of calls that follow one another, weights not in L2: one token, 4096 x 11008 int8,
// 11.0 us (45 MB, 4.1 TB/s); gate and up 11008 x 4096 int8, 17.1 us (90 MB, 5.3 TB/s); 16 tokens in
// 16 bits, 30.6 us (181 MB, 5.9 TB/s); 32 tokens, 32000 x 4096, 24.7 us (133 MB, 5.4 TB/s); 16384 x
// 16384, 41.8 us (268 MB, 6.4 TB/s). Of each about 3.5 us pass before the first slab arrives and
// after the last.
#include <algorithm>
#include <cmath>
#include <mutex>

#include "ffn_mma.cuh"

namespace qg {
namespace {

using namespace few;

constexpr int kThreads = 192;          // warps 0-3 accumulator and output, 4 TMA, 5 MMA
constexpr int kOutThreads = 128;

// after the ring: 8 rows that no copy fills, token scales, barriers, TMEM address and abort flag
constexpr int kScaleOff = kRingBytes + 8 * kSlab, kBarOff = kScaleOff + kTokens * 4;
constexpr int kBars = 2 * kMaxStages + 1;
constexpr int kSmem = 1024 + kBarOff + kBars * 8 + 16;
static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs an SM");

struct Out {
    void *c0, *c1, *c2;
    const float *sa, *sw, *sw1;
    const void *bias;
    const float *scale;     // of fp16 gradients: of what dG and dU were multiplied by
};

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
        *reinterpret_cast<uint2 *>(row + n) = make_uint2(pack2<T>(r[0], r[1]), pack2<T>(r[2], r[3]));
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (n + e < N) row[n + e] = from_f32<T>(r[e]);
    }
}

template <int FORM, bool I8, typename T, bool WM>
__global__ void __launch_bounds__(kThreads, 2)
small_kernel(const __grid_constant__ CUtensorMap tm_w0, const __grid_constant__ CUtensorMap tm_w1,
             const __grid_constant__ CUtensorMap tm_x0, const __grid_constant__ CUtensorMap tm_x1,
             const Shape shape, const Out out, unsigned int *err)
{
    using Acc = typename std::conditional<I8, int, float>::type;
    constexpr bool WMN = FORM == kDx;              // MN-major weights
    constexpr int kElems = I8 ? 128 : 64;
    const int ST = shape.stages, N = shape.N;
    const int x_bytes = shape.box_tokens * kSlab, w_bytes = shape.slab_rows * kSlab;
    // the MMA's N, and accumulator columns: of each block of 128 weight rows (WM), or of the
    // weights
    const int mma_n = ((WM ? shape.box_tokens : shape.used) + 15) / 16 * 16;
    const int blocks = WM ? (shape.used + kMmaM - 1) / kMmaM : 1;
    const int acc_cols = mma_n * blocks;
    uint32_t cols_alloc = 32;                      // a power of two
    while ((int)cols_alloc < acc_cols) cols_alloc *= 2;

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    // The slabs of the M side first: the MMA reads whole blocks of 128 rows from the start of one,
    // which reach into later slabs and into the N side's; the N side's last slab, 8 rows at most,
    // into the rows behind the ring.
    const uint32_t ring_m = smem_u32(base), ring_n = ring_m + ST * (WM ? w_bytes : x_bytes);
    const uint32_t ring_w = WM ? ring_m : ring_n, ring_x = WM ? ring_n : ring_m;
    float *scale_s = reinterpret_cast<float *>(base + kScaleOff);
    uint64_t *bars = reinterpret_cast<uint64_t *>(base + kBarOff);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + kBars);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    auto full_bar = [&](int s) { return smem_u32(bars + s); };
    auto empty_bar = [&](int s) { return smem_u32(bars + kMaxStages + s); };
    const uint32_t done_bar = smem_u32(bars + 2 * kMaxStages);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cl = (int)cluster_size(), rank = (int)blockIdx.x % cl;
    // tiles of the same weight rows are neighbours: those rows come from memory once
    const int tile = (int)blockIdx.x / cl, tiles_t = (shape.M + kTokens - 1) / kTokens;
    const int n0 = tile / tiles_t * shape.cols;
    const int t0 = tile % tiles_t * kTokens;
    const int tokens = min(kTokens, shape.M - t0);
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
    if (warp == 5) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(tmem_holder)),
                     "r"(cols_alloc)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // The weights of slab i of this part: copy(offset in the slab, map, x, y)
    auto weights = [&](int i, auto &&copy) {
        const bool second = FORM == kDx && s0 + i >= shape.seg_slabs;
        const int k = (s0 + i - (second ? shape.seg_slabs : 0)) * kElems;
        if constexpr (FORM == kDx) {
            for (int c = 0; c < shape.used; c += 64)
                copy(c * kSlab, second ? &tm_w1 : &tm_w0, n0 + c, k);
        } else {
            copy(0, &tm_w0, k, n0);
            if constexpr (FORM == kGated) copy(shape.second * kSlab, &tm_w1, k, n0);
        }
    };
    // The first slabs of weights go to L2 before the kernels ahead on the stream have finished: a
    // weight that one of them still writes is written in L2, so what is read behind grid_wait() is
    // right either way.
    if (warp == 4 && lane == 0) {
        prefetch_map(&tm_x0);
        if (FORM == kDx) prefetch_map(&tm_x1);
        for (int i = 0; i < min(ns, ST); ++i)
            weights(i, [](int, const CUtensorMap *map, int x, int y) { tma_prefetch_2d(map, x, y); });
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    grid_wait();

    // This CTA's share of the tile, in groups of four columns: some of the tokens where there are
    // enough of them (whole rows, the longest runs), else some of the groups. A thread keeps one
    // group, whose factors it loads now, under the weights' stream, and takes every `step`-th
    // token.
    const int groups = shape.cols / 4;
    const bool by_token = tokens >= 2 * cl;
    const int g0 = by_token ? 0 : groups * rank / cl;
    const int ng = by_token ? groups : groups * (rank + 1) / cl - g0;
    const int token0 = by_token ? tokens * rank / cl : 0;
    const int token1 = by_token ? tokens * (rank + 1) / cl : tokens;
    const int step = ng > 0 ? kOutThreads / ng : 1;
    const int n = n0 + 4 * (g0 + (ng > 0 ? (int)threadIdx.x % ng : 0));
    const int first = token0 + (ng > 0 ? (int)threadIdx.x / ng : 0);
    const bool mine = (int)threadIdx.x < ng * step && n < N;
    float f0[4] = {}, f1[4] = {}, back = 1.f;
    if constexpr (FORM == kDx && std::is_same<T, __half>::value)
        if (warp < 4) back = ld_behind_f32(out.scale);
    if (I8 && warp < 4) {
        scale_s[threadIdx.x] = (int)threadIdx.x < tokens ? ld_behind_f32(out.sa + t0 + threadIdx.x) : 0.f;
        if (mine) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int c = min(n + e, N - 1);
                f0[e] = ld_behind_f32(out.sw + c);
                if constexpr (FORM == kGated) f1[e] = ld_behind_f32(out.sw1 + c);
                else if (out.bias) f1[e] = ld_behind_16<T>(static_cast<const T *>(out.bias) + c);
            }
        }
    }

    if (warp == 4) {
        // ---------------- TMA producer ----------------
        const uint32_t tx = (uint32_t)x_bytes + (FORM == kGated ? 2 : 1) * shape.cols * kSlab;
        int it = 0, s = 0;
        uint32_t phase = 1;
        for (; it < ns; ++it) {
            const bool second = FORM == kDx && s0 + it >= shape.seg_slabs;
            const int k = (s0 + it - (second ? shape.seg_slabs : 0)) * kElems;
            const uint32_t xa = ring_x + s * x_bytes, wa = ring_w + s * w_bytes;
            if (!warp_wait(empty_bar(s), phase, abort_flag, err)) break;
            if (lane == 0) {
                mbar_expect_tx(full_bar(s), tx);
                weights(it, [&](int at, const CUtensorMap *map, int x, int y) {
                    tma_load_2d(wa + at, map, full_bar(s), x, y);
                });
                tma_load_2d(xa, second ? &tm_x1 : &tm_x0, full_bar(s), k, t0);
            }
            __syncwarp();
            if (++s == ST) {
                s = 0;
                phase ^= 1;
            }
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
        const uint32_t idesc = ffn_instr_desc<I8, T, WM && WMN, !WM && WMN>(kMmaM, mma_n);
        constexpr int kw = WMN ? 128 : 2;      // 16 rows of an MN-major slab, 32 bytes of the other
        int s = 0;
        uint32_t phase = 0;
        for (int it = 0; it < ns; ++it) {
            const uint64_t dx = sw128_desc(ring_x + s * x_bytes);
            const uint32_t wa = ring_w + s * w_bytes;
            const uint64_t dw = WMN ? sw128_desc_mn(wa, 8192) : sw128_desc(wa);
            if (!warp_wait(full_bar(s), phase, abort_flag, err)) break;
            tc_fence_after();
            if (lane == 0) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t accumulate = (it | k) != 0 ? 1u : 0u;
                    if constexpr (WM) {
                        ffn_mma<I8>(tmem_base, dw + kw * k, dx + 2 * k, idesc, accumulate);
                        // the next 128 rows: 16 KB on, in either layout
                        if (blocks > 1)
                            ffn_mma<I8>(tmem_base + mma_n, dw + kw * k + 1024, dx + 2 * k, idesc,
                                        accumulate);
                    } else {
                        ffn_mma<I8>(tmem_base, dx + 2 * k, dw + kw * k, idesc, accumulate);
                    }
                }
                mma_commit(empty_bar(s));
            }
            __syncwarp();
            if (++s == ST) {
                s = 0;
                phase ^= 1;
            }
        }
        if (lane == 0) mma_commit(done_bar);
        __syncwarp();
        int dummy_abort = 0;
        mbar_wait(done_bar, 0, &dummy_abort, nullptr);
    }
    // The accumulator to shared memory as [token][weight row]: lane = weight row (WM) or token. A
    // CTA whose waits gave up has raised the error word; it goes through the same steps so that
    // nobody hangs.
    if (warp < 4) mbar_wait(done_bar, 0, abort_flag, err);
    __syncthreads();               // the copies have landed and the MMAs have read them
    uint32_t *part = reinterpret_cast<uint32_t *>(base);
    if (warp < 4) {
        tc_fence_after();
        const uint32_t tm = tmem_base + ((uint32_t)(warp * 32) << 16);
        if constexpr (WM) {
            for (int b = 0; b < blocks; ++b) {
                const int row = b * kMmaM + (int)threadIdx.x;
#pragma unroll 1
                for (int c = 0; c < tokens; c += 16) {
                    uint32_t v[16];
                    tmem_ld16(tm + b * mma_n + c, v);
                    if (row < shape.used)
#pragma unroll
                        for (int q = 0; q < 16; ++q)
                            if (c + q < tokens) part[(c + q) * shape.pitch + row] = v[q];
                }
            }
        } else if (warp * 32 < tokens) {
            uint32_t *to = part + threadIdx.x * shape.pitch;
#pragma unroll 1
            for (int c = 0; c < shape.used; c += 16) {
                uint32_t v[16];
                tmem_ld16(tm + c, v);
                if ((int)threadIdx.x < tokens)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (c + 4 * q < shape.used)
                            *reinterpret_cast<uint4 *>(to + c + 4 * q) =
                                make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    // TMEM goes back before this CTA waits for others of its cluster: a kernel of another stream
    // whose CTAs wait for it on one SM while theirs keep a CTA of this cluster waiting on another
    // would otherwise never see it freed.
    if (warp == 5) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                     "r"(cols_alloc)
                     : "memory");
    }
    if (cl > 1) cluster_sync();

    if (warp < 4 && mine) {
        const uint32_t group = smem_u32(part) + (uint32_t)(n - n0) * 4;
        auto total = [&](int token, int shift, Acc (&r)[4]) {
            const uint32_t at = group + (uint32_t)(token * shape.pitch + shift) * 4;
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
        // an int32 sum scaled by its token and then its column, as the definition has it
        auto scaled = [&](Acc x, float sa, float f) {
            if constexpr (I8) return __fmul_rn(__fmul_rn(__int2float_rn(x), sa), f);
            else return x;
        };
        for (int t = first; t < token1; t += step) {
            const size_t at = (size_t)(t0 + t) * N;
            Acc a[4];
            total(t, 0, a);
            float r[4];
            const float sa = I8 ? scale_s[t] : 0.f;
            if constexpr (FORM == kGated) {
                Acc b[4];
                total(t, shape.second, b);
                float g[4], u[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    g[e] = scaled(a[e], sa, f0[e]);
                    u[e] = scaled(b[e], sa, f1[e]);
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
                    r[e] = scaled(a[e], sa, f0[e]);
                    if constexpr (FORM == kDx) r[e] *= back;
                    if constexpr (I8) {
                        if (out.bias) r[e] = __fadd_rn(r[e], f1[e]);
                    }
                }
                store4(static_cast<T *>(out.c0) + at, n, N, r);
            }
        }
    }
    __syncwarp();
    // no CTA may leave while another reads its shared memory
    if (cl > 1) cluster_sync();
}

// ---- host side -------------------------------------------------------------------------------------

template <int FORM, bool I8, typename T, bool WM>
cudaError_t launch_plan(const Matrix &w0, const Matrix &w1, const Matrix &x0, const Matrix &x1,
                        Shape shape, const Out &out, unsigned int *err, cudaStream_t stream)
{
    auto kern = small_kernel<FORM, I8, T, WM>;
    static std::mutex mu;
    static bool opted_in[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (!opted_in[dev]) {
            const cudaError_t e =
                cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
            if (e != cudaSuccess) return e;
            opted_in[dev] = true;
        }
    }
    const Plan plan = plan_small(FORM, shape.M, shape.N, shape.slabs);
    if (!lay_out(&shape, plan.cols, FORM)) return cudaErrorInvalidConfiguration;
    const long long tiles = (long long)ceil_div(shape.N, plan.cols) * ceil_div(shape.M, kTokens);
    if (tiles * plan.parts > 0x7fffffffLL) return cudaErrorInvalidValue;
    // a slab's box: the tile's columns of a weight matrix, or 64 rows of the reduction for kDx
    CUtensorMap tw0, tw1, tx0, tx1;
    const int wbox = FORM == kDx ? 64 : plan.cols;
    if (!map_of<I8, T>(&tw0, w0, wbox) || !map_of<I8, T>(&tx0, x0, shape.box_tokens))
        return cudaErrorInvalidValue;
    tw1 = tw0;
    tx1 = tx0;
    if (w1.p != w0.p && !map_of<I8, T>(&tw1, w1, wbox)) return cudaErrorInvalidValue;
    if (x1.p != x0.p && !map_of<I8, T>(&tx1, x1, shape.box_tokens)) return cudaErrorInvalidValue;
    return launch_dependent(kern, dim3((unsigned)(tiles * plan.parts)), dim3(kThreads), kSmem,
                            plan.parts, stream, tw0, tw1, tx0, tx1, shape, out, err);
}

template <int FORM, bool I8, typename T>
cudaError_t launch_small(const Matrix &w0, const Matrix &w1, const Matrix &x0, const Matrix &x1,
                         const Shape &shape, const Out &out, unsigned int *err, cudaStream_t stream)
{
    if (shape.M <= kWeightMajor)
        return launch_plan<FORM, I8, T, true>(w0, w1, x0, x1, shape, out, err, stream);
    return launch_plan<FORM, I8, T, false>(w0, w1, x0, x1, shape, out, err, stream);
}

} // namespace

cudaError_t launch_small_scaled(const ScaledProblem &p, unsigned int *err, cudaStream_t stream)
{
    const uint64_t K = p.K;
    const Matrix a{p.A, (uint64_t)p.M, K, K}, w{p.W, (uint64_t)p.N, K, K};
    const Matrix w1{p.W1 ? p.W1 : p.W, (uint64_t)p.N, K, K};
    const Out out{p.C, nullptr, nullptr, p.sa, p.sw, p.sw1, p.bias, nullptr};
    const Shape shape = shape_of(p.M, p.N, ceil_div(p.K, 128), 1, p.act);
    QG_DISPATCH_16(p.dtype, T, {
        if (p.W1) return launch_small<kGated, true, T>(w, w1, a, a, shape, out, err, stream);
        return launch_small<kScaled, true, T>(w, w, a, a, shape, out, err, stream);
    });
}

cudaError_t launch_small_gated(const GatedProblem &p, unsigned int *err, cudaStream_t stream)
{
    const uint64_t K = p.K, pitch = K * 2;
    const Matrix x{p.X, (uint64_t)p.M, K, pitch};
    const Matrix g{p.Wg, (uint64_t)p.F, K, pitch}, u{p.Wu, (uint64_t)p.F, K, pitch};
    const Out out{p.H, p.G, p.U, nullptr, nullptr, nullptr, nullptr, nullptr};
    const Shape shape = shape_of(p.M, p.F, ceil_div(p.K, 64), 1, p.act);
    QG_DISPATCH_16(p.dtype, T, {
        return launch_small<kGated, false, T>(g, u, x, x, shape, out, err, stream);
    });
}

cudaError_t launch_small_dx(const GatedGrad &p, unsigned int *err, cudaStream_t stream)
{
    const uint64_t M = p.M, F = p.F, K = p.K;
    const Matrix dg{p.dG, M, F, (uint64_t)p.Fp * 2}, du{p.dU, M, F, (uint64_t)p.Fp * 2};
    const Matrix wg{p.Wg, F, K, K * 2}, wu{p.Wu, F, K, K * 2};
    const Out out{p.dX, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, p.scale};
    const Shape shape = shape_of(p.M, p.K, ceil_div(p.F, 64), 2, 0);
    QG_DISPATCH_16(p.dtype, T, {
        return launch_small<kDx, false, T>(wg, wu, dg, du, shape, out, err, stream);
    });
}

} // namespace qg
