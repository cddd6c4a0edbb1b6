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
constexpr int kSpan = 2048;

template <typename T, int ACT>
__device__ __forceinline__ void grad_pair(uint32_t dh, uint32_t g, uint32_t u, uint32_t &dg,
                                          uint32_t &du)
{
    const float2 h2 = unpack2<T>(dh), g2 = unpack2<T>(g), u2 = unpack2<T>(u);
    float v0, d0, v1, d1;
    act_both<ACT>(g2.x, v0, d0);
    act_both<ACT>(g2.y, v1, d1);
    dg = pack2<T>(h2.x * u2.x * d0, h2.y * u2.y * d1);
    du = pack2<T>(h2.x * v0, h2.y * v1);
}

template <typename T, int ACT>
__global__ void __launch_bounds__(kThreads)
grad_act_kernel(const T *dH, const T *G, const T *U, T *dG, T *dU, size_t n)
{
    grid_release();
    grid_wait();
    const size_t at = ((size_t)blockIdx.x * kThreads + threadIdx.x) * 8;
    if (at >= n) return;
    const uint4 h = ld_behind_v4(dH + at), g = ld_behind_v4(G + at), u = ld_behind_v4(U + at);
    uint4 dg, du;
    grad_pair<T, ACT>(h.x, g.x, u.x, dg.x, du.x);
    grad_pair<T, ACT>(h.y, g.y, u.y, dg.y, du.y);
    grad_pair<T, ACT>(h.z, g.z, u.z, dg.z, du.z);
    grad_pair<T, ACT>(h.w, g.w, u.w, dg.w, du.w);
    *reinterpret_cast<uint4 *>(dG + at) = dg;
    *reinterpret_cast<uint4 *>(dU + at) = du;
}

template <typename T, int ACT, bool PAIRS>
__global__ void __launch_bounds__(kThreads)
grad_act_rows_kernel(const T *dH, const T *G, const T *U, T *dG, T *dU, int F, int Fp)
{
    grid_release();
    grid_wait();
    const unsigned spans = (unsigned)(F + kSpan - 1) / kSpan;
    const size_t m = blockIdx.x / spans;
    const int f0 = (int)(blockIdx.x % spans) * kSpan, f1 = min(f0 + kSpan, F);
    const size_t in = m * F, to = m * Fp;
    // kBatch loads of each matrix in flight, then what is made of them: the loads keep their order
    constexpr int kBatch = 4, kStep = (PAIRS ? 2 : 1) * kThreads;
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
                grad_pair<T, ACT>(h[i], g[i], u[i], dg, du);
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
                    dG[to + at] = from_f32<T>(h[i] * u[i] * d);
                    dU[to + at] = from_f32<T>(h[i] * v);
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
    if (p.F % 8 == 0)
        return launch_dependent(grad_act_kernel<T, ACT>, grid, block, 0, 1, stream, dH, G, U, dG,
                                dU, n);
    if (p.F % 2 == 0)
        return launch_dependent(grad_act_rows_kernel<T, ACT, true>, grid, block, 0, 1, stream, dH, G,
                                U, dG, dU, p.F, p.Fp);
    return launch_dependent(grad_act_rows_kernel<T, ACT, false>, grid, block, 0, 1, stream, dH, G, U,
                            dG, dU, p.F, p.Fp);
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
