// Internal interface and device arithmetic of the 8-bit scaled matmul and the gated feed-forward
// block (token quantisation, scaled W8A8, gated forward in 8 and 16 bits, gated backward).
#pragma once

#include <cuda_bf16.h>

#include <type_traits>

#include "common.cuh"
#include "ffn_plan.cuh"

namespace qg {

// ------------------------------------------------------------------------------------------
// 16-bit types
// ------------------------------------------------------------------------------------------
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v)
{
    return __float2bfloat16_rn(v);
}

// two values rounded to nearest even, the first in the low half of the word
template <typename T> __device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <> __device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi)
{
    return pack_half2_rn(lo, hi);
}
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi)
{
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&v);
}

// the two values of a word
template <typename T> __device__ __forceinline__ float2 unpack2(uint32_t w);
template <> __device__ __forceinline__ float2 unpack2<__half>(uint32_t w)
{
    return __half22float2(*reinterpret_cast<__half2 *>(&w));
}
template <> __device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// ------------------------------------------------------------------------------------------
// Activations, in fp32. The logistic function takes the fast exponential and division (relative
// error a few 2^-23 at the arguments that matter): every result is rounded to 16 bits, whose half
// step is 2^-11 or 2^-8. Arguments of the tanh form are held to +-100, where its logistic
// function is 0 or 1 in fp32, so that g^2 and g^3 cannot overflow; comparisons let NaN through.
// ------------------------------------------------------------------------------------------
__device__ __forceinline__ float logistic(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }

__device__ __forceinline__ float hold100(float g)
{
    return g > 100.0f ? 100.0f : (g < -100.0f ? -100.0f : g);
}

constexpr float kGeluRoot = 0.7978845608028654f;     // sqrt(2 / pi)
constexpr float kGeluCube = 0.044715f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

template <int ACT> __device__ __forceinline__ float act_value(float g)
{
    if constexpr (ACT == QG_ACT_SILU) {
        return g * logistic(g);
    } else if constexpr (ACT == QG_ACT_GELU) {
        return g * normcdff(g);
    } else {
        // 0.5 (1 + tanh w) = logistic(2 w): no cancellation for negative g
        const float h = hold100(g);
        return g * logistic(2.0f * kGeluRoot * h * (1.0f + kGeluCube * h * h));
    }
}

// value and derivative
template <int ACT> __device__ __forceinline__ void act_both(float g, float &value, float &slope)
{
    if constexpr (ACT == QG_ACT_SILU) {
        const float s = logistic(g);
        value = g * s;
        slope = s * (1.0f + g * (1.0f - s));
    } else if constexpr (ACT == QG_ACT_GELU) {
        const float p = normcdff(g);
        value = g * p;
        slope = p + g * (kInvSqrt2Pi * __expf(-0.5f * g * g));
    } else {
        const float h = hold100(g);
        const float s = logistic(2.0f * kGeluRoot * h * (1.0f + kGeluCube * h * h));
        value = g * s;
        slope = s + h * (s * (1.0f - s)) * (2.0f * kGeluRoot * (1.0f + 3.0f * kGeluCube * h * h));
    }
}

// Run f with the activation and 16-bit type as template arguments.
template <int V> struct Const {
    static constexpr int value = V;
};
#define QG_DISPATCH_16(dtype, T, ...)                                                              \
    do {                                                                                           \
        if ((dtype) == QG_BF16) { using T = __nv_bfloat16; __VA_ARGS__; }                          \
        else { using T = __half; __VA_ARGS__; }                                                    \
    } while (0)
#define QG_DISPATCH_ACT(act, ACT, ...)                                                             \
    do {                                                                                           \
        if ((act) == QG_ACT_SILU) { constexpr int ACT = QG_ACT_SILU; __VA_ARGS__; }                \
        else if ((act) == QG_ACT_GELU) { constexpr int ACT = QG_ACT_GELU; __VA_ARGS__; }           \
        else { constexpr int ACT = QG_ACT_GELU_TANH; __VA_ARGS__; }                                \
    } while (0)

// ------------------------------------------------------------------------------------------
// Programmatic dependent launch. grid_wait() returns when the kernels before this one on the stream
// have finished and their writes are visible; grid_release() lets the next kernel's CTAs start once
// every CTA of this one has called it. Quantisation, the elementwise half of the gradients and the
// joining of parts release as soon as they start, the tensor-core kernels and the first pass of
// fp16 gradients when the last of their loads is on its way. Results are written, and operands read, only behind
// grid_wait(); before it the tensor-core kernels do no more than ask for their first weights to be
// brought into L2, where a predecessor's writes to them land too. So a kernel's launch, barrier and
// tensor-memory set-up run under the end of its predecessor, and stream order is kept: 1 to 3 us
// less a call, measured on calls of 2 to 60 us that follow one another.
//
// Such a kernel runs while what it will read is still being written. Its loads are therefore the
// ld_behind_* below: volatile with a memory clobber, so that the compiler leaves them behind
// grid_wait(), and not .nc, which asks for data that does not change during the kernel's life.
// ------------------------------------------------------------------------------------------
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_release()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// 16 bytes that are read once
__device__ __forceinline__ uint4 ld_behind_v4(const void *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// 16 bytes that are read again
__device__ __forceinline__ uint4 ld_behind_cached_v4(const void *p)
{
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

__device__ __forceinline__ uint32_t ld_behind_u32(const void *p)
{
    uint32_t v;
    asm volatile("ld.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ float ld_behind_f32(const float *p)
{
    return __uint_as_float(ld_behind_u32(p));
}

template <typename T> __device__ __forceinline__ float ld_behind_16(const void *p)
{
    uint16_t v;
    asm volatile("ld.global.u16 %0, [%1];" : "=h"(v) : "l"(p) : "memory");
    return unpack2<T>(v).x;
}

// Launch with `cluster` CTAs a cluster (along x) and programmatic dependent launch.
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, int cluster,
                             cudaStream_t stream, A &&...args)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// ------------------------------------------------------------------------------------------
// Launchers: queue on `stream`, return cudaGetLastError().
// ------------------------------------------------------------------------------------------
struct ScaledProblem {      // int8 operands: scaled matmul (W1 null) or gated (W1 = Wu)
    const int8_t *A, *W, *W1;
    const float *sa, *sw, *sw1;
    const void *bias;
    void *C;
    int M, N, K, act, dtype;
};
struct GatedProblem {       // 16-bit operands, forward
    const void *X, *Wg, *Wu;
    void *H, *G, *U;
    int M, F, K, act, dtype;
};
// fp16: the factor, and behind it the largest value that each CTA of a first pass has seen
constexpr int kGradTops = 4 * 148, kGradScale = 4 + kGradTops;
struct GatedGrad {          // backward; dG, dU and part live in the caller's workspace
    const void *dH, *X, *Wg, *Wu, *G, *U;
    void *dX, *dWg, *dWu, *dG, *dU;
    int M, F, K, act, dtype;
    int Fp;                 // row pitch of dG and dU in elements (a multiple of 8)
    float *part;            // partial sums, grad_part_bytes() bytes
    float *scale;           // fp16: what the products of dG and dU are multiplied by; kGradScale floats
    GradPlan plan;
};

cudaError_t launch_quant_int8_tokens(const void *X, int8_t *Q, float *scales, int M, int K,
                                     int dtype, cudaStream_t stream);
cudaError_t launch_w8a8_scaled(const ScaledProblem &p, unsigned int *err, cudaStream_t stream);
cudaError_t launch_dense_gated(const GatedProblem &p, unsigned int *err, cudaStream_t stream);
cudaError_t launch_gated_backward(const GatedGrad &p, unsigned int *err, cudaStream_t stream);

// Large tiles (ffn_tile.cu) and few tokens (ffn_small.cu): each takes any sizes, ffn_plan.cuh chooses.
cudaError_t launch_tile_scaled(const ScaledProblem &p, unsigned int *err, cudaStream_t stream);
cudaError_t launch_tile_gated(const GatedProblem &p, unsigned int *err, cudaStream_t stream);
cudaError_t launch_tile_grad(const GatedGrad &p, unsigned int *err, cudaStream_t stream);
cudaError_t launch_small_scaled(const ScaledProblem &p, unsigned int *err, cudaStream_t stream);
cudaError_t launch_small_gated(const GatedProblem &p, unsigned int *err, cudaStream_t stream);
cudaError_t launch_small_dx(const GatedGrad &p, unsigned int *err, cudaStream_t stream);

} // namespace qg
