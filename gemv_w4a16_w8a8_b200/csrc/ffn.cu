// Choice of kernel for the scaled W8A8 matmul and the gated feed-forward block, and the
// elementwise half of its backward pass.
#include <algorithm>

#include "ffn.cuh"

namespace qg {
namespace {

constexpr int kThreads = 256;

// dG = dH U act'(G), dU = dH act(G), rounded to 16 bits for the tensor cores (the products that
// read them sum in fp32; the rounding is as large as that of the gradients themselves). Rows of Fp
// elements, a multiple of eight, which TMA asks for. Bound: HBM, 10 bytes an element. F % 8 == 0:
// the matrices are one run of eight elements a thread by 16-byte loads and stores. Otherwise rows
// start anywhere: a CTA takes kSpan elements of a row, by pairs where F is even, else one by one.
//
// Range: bf16 has that of fp32. In fp16 dG would overflow from dH U = 65504 on and lose bits below
// 2^-14, where the gradients, sums of it times weights or activations, may be ordinary fp16 numbers.
// So a first pass takes the largest finite |dG| or |dU| (6 bytes an element; gelu: a bound of it), dG
// and dU are multiplied by the power of two that brings it to 2^14 .. 2^15, and the products by its
// inverse in fp32, before they are rounded: exact but for values below 2^-28 of the largest, which
// become subnormal (an error of at most 2^-39 of the largest). One power for both, since dX adds
// them up.
constexpr int kSpan = 2048;

template <typename T> constexpr bool kScaledRange = std::is_same<T, __half>::value;

template <typename T, int ACT>
__device__ __forceinline__ void grad_f32(uint32_t dh, uint32_t g, uint32_t u, float2 &dg, float2 &du)
{
    const float2 h2 = unpack2<T>(dh), g2 = unpack2<T>(g), u2 = unpack2<T>(u);
    float v0, d0, v1, d1;
    act_both<ACT>(g2.x, v0, d0);
    act_both<ACT>(g2.y, v1, d1);
    dg = make_float2(h2.x * u2.x * d0, h2.y * u2.y * d1);
    du = make_float2(h2.x * v0, h2.y * v1);
}

template <typename T, int ACT>
__device__ __forceinline__ void grad_pair(uint32_t dh, uint32_t g, uint32_t u, float scale, uint32_t &dg,
                                          uint32_t &du)
{
    float2 a, b;
    grad_f32<T, ACT>(dh, g, u, a, b);
    if constexpr (kScaledRange<T>) a.x *= scale, a.y *= scale, b.x *= scale, b.y *= scale;
    dg = pack2<T>(a.x, a.y);
    du = pack2<T>(b.x, b.y);
}

// The larger of `top` and a finite |x|
__device__ __forceinline__ float finite_max(float top, float x)
{
    x = fabsf(x);
    return x < __int_as_float(0x7f800000) ? fmaxf(top, x) : top;
}

// The largest of a CTA, in every thread (non-negative floats are ordered like their bits)
template <int WARPS> __device__ __forceinline__ float cta_max(float top)
{
    __shared__ uint32_t part[WARPS];
    const int t = threadIdx.x;
    const uint32_t w = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
    if ((t & 31) == 0) part[t >> 5] = w;
    __syncthreads();
    return __uint_as_float(__reduce_max_sync(0xffffffffu, part[t & 31 & (WARPS - 1)]));
}

// |act| and |act'|, or for gelu bounds of them that take one exponential instead of the normal
// distribution's hundred instructions: the logistic function of 1.702 g is Phi(g) within 4 % or above it,
// so 17/16 of it is an upper bound, 1 + |g| times that one of the derivative, and 1.13 another (at
// most 1.3 times too large for positive g, and never below the value). With Phi itself this pass took
// 340 us of 8192 x 11007 values, with the bounds 140.
template <int ACT> __device__ __forceinline__ void act_bounds(float g, float &value, float &slope)
{
    if constexpr (ACT == QG_ACT_GELU) {
        const float s = 1.0625f * logistic(1.702f * g);
        value = g * s;
        slope = fminf(1.13f, (1.0f + fabsf(g)) * s);
    } else {
        act_both<ACT>(g, value, slope);
    }
}

// The largest finite |dG| or |dU| (gelu: bound of it) that each CTA sees. Eight values a load, two loads of each matrix in
// flight, up to four CTAs an SM: enough for HBM, and few enough registers to start beside the CTAs
// of a tile kernel ahead on the stream. It costs 1 us of a short batch (77 x 1371 x 520: 13.8 -> 14.8
// us) and its reading of a long one (8192 x 11008 x 4096: 2.55 -> 2.68 ms). Releasing as it starts, as
// its successor does, let the weights' stream behind both begin under the tiles ahead and slowed those
// (16 x 11008 x 4096: 106 us against 92).
template <int ACT>
__global__ void __launch_bounds__(kThreads, 5)
grad_top_kernel(const __half *dH, const __half *G, const __half *U, float *scale, size_t n)
{
    grid_wait();
    constexpr int kBatch = 2;
    const size_t vecs = n / 8, step = (size_t)gridDim.x * kThreads;
    float top = 0.f;
    auto see1 = [&](float dh, float g, float u) {
        float v, d;
        act_bounds<ACT>(g, v, d);
        top = finite_max(finite_max(top, dh * u * d), dh * v);
    };
    auto see = [&](uint32_t dh, uint32_t g, uint32_t u) {
        const float2 h2 = unpack2<__half>(dh), g2 = unpack2<__half>(g), u2 = unpack2<__half>(u);
        see1(h2.x, g2.x, u2.x);
        see1(h2.y, g2.y, u2.y);
    };
#pragma unroll 1
    for (size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x; i < vecs; i += kBatch * step) {
        uint4 h[kBatch], g[kBatch], u[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (i + k * step < vecs) {
                const size_t at = (i + k * step) * 8;
                h[k] = ld_behind_v4(dH + at);
                g[k] = ld_behind_v4(G + at);
                u[k] = ld_behind_v4(U + at);
            }
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (i + k * step < vecs) {
                see(h[k].x, g[k].x, u[k].x);
                see(h[k].y, g[k].y, u[k].y);
                see(h[k].z, g[k].z, u[k].z);
                see(h[k].w, g[k].w, u[k].w);
            }
    }
    grid_release();
    const size_t at = vecs * 8 + threadIdx.x;              // up to seven values at the end
    if (blockIdx.x == 0 && at < n)
        see1(ld_behind_16<__half>(dH + at), ld_behind_16<__half>(G + at), ld_behind_16<__half>(U + at));
    top = cta_max<kThreads / 32>(top);
    if (threadIdx.x == 0) scale[4 + blockIdx.x] = top;
}

// The power of two for dG and dU from the CTAs' largest values; its inverse to scale[0]
__device__ __forceinline__ float grad_scale(float *scale, int tops)
{
    const int t = threadIdx.x;
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < (kGradTops + kThreads - 1) / kThreads; ++i)
        if (t + i * kThreads < tops) top = fmaxf(top, ld_behind_f32(scale + 4 + t + i * kThreads));
    top = cta_max<kThreads / 32>(top);
    const int e = (int)(__float_as_uint(top) >> 23) - 127;         // floor of the logarithm
    const int k = top > 0.f ? min(14 - e, 100) : 0;
    if (blockIdx.x == 0 && t == 0) scale[0] = __uint_as_float((uint32_t)(127 - k) << 23);
    return __uint_as_float((uint32_t)(127 + k) << 23);
}

template <typename T, int ACT>
__global__ void __launch_bounds__(kThreads)
grad_act_kernel(const T *dH, const T *G, const T *U, T *dG, T *dU, size_t n, float *scale, int tops)
{
    grid_release();
    grid_wait();
    const size_t at = ((size_t)blockIdx.x * kThreads + threadIdx.x) * 8;
    const bool live = at < n;
    uint4 h = {}, g = {}, u = {};
    if (live) {
        h = ld_behind_v4(dH + at);
        g = ld_behind_v4(G + at);
        u = ld_behind_v4(U + at);
    }
    float s = 1.f;
    if constexpr (kScaledRange<T>) s = grad_scale(scale, tops);
    if (!live) return;
    uint4 dg, du;
    grad_pair<T, ACT>(h.x, g.x, u.x, s, dg.x, du.x);
    grad_pair<T, ACT>(h.y, g.y, u.y, s, dg.y, du.y);
    grad_pair<T, ACT>(h.z, g.z, u.z, s, dg.z, du.z);
    grad_pair<T, ACT>(h.w, g.w, u.w, s, dg.w, du.w);
    *reinterpret_cast<uint4 *>(dG + at) = dg;
    *reinterpret_cast<uint4 *>(dU + at) = du;
}

template <typename T, int ACT, bool PAIRS>
__global__ void __launch_bounds__(kThreads)
grad_act_rows_kernel(const T *dH, const T *G, const T *U, T *dG, T *dU, int F, int Fp, float *scale,
                     int tops)
{
    grid_release();
    grid_wait();
    float s = 1.f;
    if constexpr (kScaledRange<T>) s = grad_scale(scale, tops);
    const unsigned spans = (unsigned)(F + kSpan - 1) / kSpan;
    const size_t m = blockIdx.x / spans;
    const int f0 = (int)(blockIdx.x % spans) * kSpan, f1 = min(f0 + kSpan, F);
    const size_t in = m * F, to = m * Fp;
    // kBatch loads of each matrix in flight, then what is made of them: the loads keep their order
    constexpr int kBatch = PAIRS ? 4 : 8, kStep = (PAIRS ? 2 : 1) * kThreads;
#pragma unroll 1
    for (int f = f0 + (PAIRS ? 2 : 1) * (int)threadIdx.x; f < f1; f += kBatch * kStep) {
        if constexpr (PAIRS) {
            uint32_t h[kBatch] = {}, g[kBatch] = {}, u[kBatch] = {};
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int at = f + i * kStep;
                if (at < f1) {
                    h[i] = ld_behind_u32(dH + in + at);
                    g[i] = ld_behind_u32(G + in + at);
                    u[i] = ld_behind_u32(U + in + at);
                }
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int at = f + i * kStep;
                uint32_t dg, du;
                grad_pair<T, ACT>(h[i], g[i], u[i], s, dg, du);
                if (at < f1) {
                    *reinterpret_cast<uint32_t *>(dG + to + at) = dg;
                    *reinterpret_cast<uint32_t *>(dU + to + at) = du;
                }
            }
        } else {
            float h[kBatch] = {}, g[kBatch] = {}, u[kBatch] = {};
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int at = f + i * kStep;
                if (at < f1) {
                    h[i] = ld_behind_16<T>(dH + in + at);
                    g[i] = ld_behind_16<T>(G + in + at);
                    u[i] = ld_behind_16<T>(U + in + at);
                }
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int at = f + i * kStep;
                float v, d;
                act_both<ACT>(g[i], v, d);
                if (at < f1) {
                    dG[to + at] = from_f32<T>(h[i] * u[i] * d * s);
                    dU[to + at] = from_f32<T>(h[i] * v * s);
                }
            }
        }
    }
}

template <typename T, int ACT> cudaError_t run_grad_act(const GatedGrad &p, cudaStream_t stream)
{
    const T *dH = static_cast<const T *>(p.dH), *G = static_cast<const T *>(p.G);
    const T *U = static_cast<const T *>(p.U);
    T *dG = static_cast<T *>(p.dG), *dU = static_cast<T *>(p.dU);
    const size_t n = (size_t)p.M * p.F, rows = (size_t)p.M * ((p.F + kSpan - 1) / kSpan);
    const size_t ctas = p.F % 8 ? rows : (n / 8 + kThreads - 1) / kThreads;
    if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)ctas), block(kThreads);
    int tops = 0;
    if constexpr (kScaledRange<T>) {
        const size_t most = std::max<size_t>(1, (n / 8 + kThreads - 1) / kThreads);
        tops = (int)std::min<size_t>(kGradTops, most);
        const cudaError_t e = launch_dependent(grad_top_kernel<ACT>, dim3(tops), dim3(kThreads), 0, 1,
                                               stream, dH, G, U, p.scale, n);
        if (e != cudaSuccess) return e;
    }
    if (p.F % 8 == 0)
        return launch_dependent(grad_act_kernel<T, ACT>, grid, block, 0, 1, stream, dH, G, U, dG,
                                dU, n, p.scale, tops);
    if (p.F % 2 == 0)
        return launch_dependent(grad_act_rows_kernel<T, ACT, true>, grid, block, 0, 1, stream, dH, G,
                                U, dG, dU, p.F, p.Fp, p.scale, tops);
    return launch_dependent(grad_act_rows_kernel<T, ACT, false>, grid, block, 0, 1, stream, dH, G, U,
                            dG, dU, p.F, p.Fp, p.scale, tops);
}

} // namespace

cudaError_t launch_w8a8_scaled(const ScaledProblem &p, unsigned int *err, cudaStream_t stream)
{
    const int slabs = (p.K + 127) / 128;
    const bool gated = p.W1 != nullptr;
    if (few_tokens(p.M, p.N, gated, true, slabs))
        return launch_small_scaled(p, err, stream);
    return launch_tile_scaled(p, err, stream);
}

cudaError_t launch_dense_gated(const GatedProblem &p, unsigned int *err, cudaStream_t stream)
{
    const int slabs = (p.K + 63) / 64;
    if (few_tokens(p.M, p.F, true, false, slabs))
        return launch_small_gated(p, err, stream);
    return launch_tile_gated(p, err, stream);
}

cudaError_t launch_gated_backward(const GatedGrad &p, unsigned int *err, cudaStream_t stream)
{
    cudaError_t e = cudaSuccess;
    QG_DISPATCH_16(p.dtype, T, {
        QG_DISPATCH_ACT(p.act, ACT, {
            e = run_grad_act<T, ACT>(p, stream);
        });
    });
    if (e == cudaSuccess && p.plan.few && p.dX) e = launch_small_dx(p, err, stream);
    if (e == cudaSuccess) e = launch_tile_grad(p, err, stream);
    return e;
}

} // namespace qg
