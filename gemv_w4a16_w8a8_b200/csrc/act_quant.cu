// int8 quantisation of 16-bit activations, one scale a token (quant_int8_tokens).
//
//   amax = max_k |x|,  s = amax / 127,  q = rint(x * (127 / amax))
//
// One CTA a token: it keeps its part of the row in registers between the maximum and the
// rounding, so that a row is read once. Bound: HBM (2 K bytes in, K out a token).
#include "ffn.cuh"

namespace qg {
namespace {

constexpr int kThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kThreads) quant_tokens_kernel(const T *__restrict__ X,
                                                                int8_t *__restrict__ Q,
                                                                float *__restrict__ scales, int K)
{
    const size_t row = blockIdx.x;
    const T *x = X + row * K;
    __shared__ float part[kThreads / 32];
    float amax = 0.0f;
    bool odd = false;                       // an infinity or a NaN
    for (int k = threadIdx.x; k < K; k += kThreads) {
        const float v = fabsf(to_f32(x[k]));
        odd |= !(v <= 3.4028234e38f);
        amax = fmaxf(amax, v);
    }
    if (odd) amax = __int_as_float(0x7f800000);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
    __syncthreads();
    amax = part[0];
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) amax = fmaxf(amax, part[w]);
    const bool bad = amax > 3.4028234e38f;
    const float up = amax < 8.6736174e-19f ? 1.8446744e19f : 1.0f;      // 2^-60, 2^64
    const float inv = (amax == 0.0f || bad) ? 0.0f : __fdiv_rn(127.0f, amax * up);
    if (threadIdx.x == 0)
        scales[row] = bad ? __int_as_float(0x7fffffff) : (amax == 0.0f ? 1.0f : __fdiv_rn(amax, 127.0f));
    for (int k = threadIdx.x; k < K; k += kThreads)
        Q[row * K + k] = bad ? (int8_t)0 : (int8_t)__float2int_rn(__fmul_rn(to_f32(x[k]) * up, inv));
}

} // namespace

cudaError_t launch_quant_int8_tokens(const void *X, int8_t *Q, float *scales, int M, int K,
                                     int dtype, cudaStream_t stream)
{
    QG_DISPATCH_16(dtype, T, {
        quant_tokens_kernel<T><<<M, kThreads, 0, stream>>>(static_cast<const T *>(X), Q, scales, K);
    });
    return cudaGetLastError();
}

} // namespace qg
