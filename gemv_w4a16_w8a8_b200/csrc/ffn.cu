// Choice of kernel for the scaled W8A8 matmul and the gated feed-forward block, and the
// elementwise half of its backward pass.
#include <algorithm>

#include "ffn.cuh"

namespace qg {
namespace {

constexpr int kThreads = 256;
constexpr int kFewTokens = 128;        // up to here the weights' stream is the bound

// dG = dH U act'(G), dU = dH act(G), rounded to 16 bits for the tensor cores (the products that
// read them sum in fp32); rows of Fp elements. Bound: HBM, 10 bytes an element.
template <typename T, int ACT>
__global__ void __launch_bounds__(kThreads)
grad_act_kernel(const T *__restrict__ dH, const T *__restrict__ G, const T *__restrict__ U,
                T *__restrict__ dG, T *__restrict__ dU, int F, int Fp)
{
    const size_t in = (size_t)blockIdx.x * F, out = (size_t)blockIdx.x * Fp;
    for (int f = threadIdx.x; f < F; f += kThreads) {
        float v, d;
        act_both<ACT>(to_f32(G[in + f]), v, d);
        const float dh = to_f32(dH[in + f]);
        dG[out + f] = from_f32<T>(dh * to_f32(U[in + f]) * d);
        dU[out + f] = from_f32<T>(dh * v);
    }
}

} // namespace

cudaError_t launch_w8a8_scaled(const ScaledProblem &p, int sms, unsigned int *err, cudaStream_t stream)
{
    if (p.M <= kFewTokens) return launch_small_scaled(p, sms, err, stream);
    return launch_tile_scaled(p, sms, err, stream);
}

cudaError_t launch_dense_gated(const GatedProblem &p, int sms, unsigned int *err, cudaStream_t stream)
{
    if (p.M <= kFewTokens) return launch_small_gated(p, sms, err, stream);
    return launch_tile_gated(p, sms, err, stream);
}

cudaError_t launch_gated_backward(const GatedGrad &p, int sms, unsigned int *err, cudaStream_t stream)
{
    QG_DISPATCH_16(p.dtype, T, {
        QG_DISPATCH_ACT(p.act, ACT, {
            grad_act_kernel<T, ACT><<<p.M, kThreads, 0, stream>>>(
                static_cast<const T *>(p.dH), static_cast<const T *>(p.G), static_cast<const T *>(p.U),
                static_cast<T *>(p.dG), static_cast<T *>(p.dU), p.F, p.Fp);
        });
    });
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && p.dX)
        e = p.M <= kFewTokens ? launch_small_dx(p, sms, err, stream) : launch_tile_dx(p, sms, err, stream);
    if (e == cudaSuccess && p.dWg) e = launch_tile_dw(p, sms, err, stream);
    return e;
}

} // namespace qg
