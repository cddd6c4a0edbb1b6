// int8 quantisation of 16-bit activations, one scale a token (quant_int8_tokens).
//
//   amax = max_k |x|,  s = amax / 127,  q = rint(x * (127 / amax))
//
// Bound: HBM (2 K bytes in, K out a token). A row belongs to TPR threads (one warp for short rows,
// so that a CTA takes eight; a CTA of 128 or 512 for longer ones), which hold it in registers
// between the maximum and the rounding: it is read once up to 16384 values, and a second time,
// from L2, beyond.
//   - The maximum is taken on the bit patterns without their sign, two values a SIMD instruction:
//     as integers they are ordered like the magnitudes, infinities and NaNs above every number.
//   - Rounding adds 1.5 * 2^23 in fp32: the sum's unit is 1, so the addition rounds to the nearest
//     integer, ties to even, and its low byte is the code in two's complement. Conversion
//     instructions run at an eighth of this rate and would take half of the kernel's time.
#include "ffn.cuh"

namespace qg {
namespace {

constexpr int kVec = 4;                  // 16-byte loads a thread holds

template <typename T> constexpr uint32_t inf_bits()
{
    return std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
}

__device__ __forceinline__ uint32_t max_abs(uint32_t m, const uint4 &v)
{
    m = __vmaxu2(m, v.x & 0x7fff7fffu);
    m = __vmaxu2(m, v.y & 0x7fff7fffu);
    m = __vmaxu2(m, v.z & 0x7fff7fffu);
    return __vmaxu2(m, v.w & 0x7fff7fffu);
}

// the codes of four values, as bytes
template <typename T>
__device__ __forceinline__ uint32_t codes4(uint32_t lo, uint32_t hi, float up, float inv)
{
    const float2 a = unpack2<T>(lo), b = unpack2<T>(hi);
    auto code = [&](float x) {
        return __float_as_uint(__fadd_rn(__fmul_rn(x * up, inv), 12582912.0f));
    };
    return prmt(prmt(code(a.x), code(a.y), 0x0040), prmt(code(b.x), code(b.y), 0x0040), 0x5410);
}

template <typename T>
__device__ __forceinline__ uint2 codes8(const uint4 &v, float up, float inv)
{
    return make_uint2(codes4<T>(v.x, v.y, up, inv), codes4<T>(v.z, v.w, up, inv));
}

template <typename T, int TPR, bool LONG>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR)
quant_tokens_kernel(const T *X, int8_t *Q, float *scales, int M, int K)
{
    constexpr int kThreads = TPR < 256 ? 256 : TPR, kRows = kThreads / TPR, kWarps = TPR / 32;
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    const long long row = (long long)blockIdx.x * kRows + sub;
    const bool live = row < M;
    const uint4 *x = reinterpret_cast<const uint4 *>(X + (live ? row : 0) * K);
    uint2 *q = reinterpret_cast<uint2 *>(Q + (live ? row : 0) * K);
    const int n = live ? K / 8 : 0;
    grid_release();
    grid_wait();

    uint4 v[kVec];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        v[i] = make_uint4(0u, 0u, 0u, 0u);
        if (t + i * TPR < n)
            v[i] = LONG ? ld_behind_cached_v4(x + t + i * TPR) : ld_behind_v4(x + t + i * TPR);
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) top = max_abs(top, v[i]);
    if constexpr (LONG)
        for (int j = t + kVec * TPR; j < n; j += TPR) top = max_abs(top, ld_behind_cached_v4(x + j));
    top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
    if constexpr (kWarps > 1) {
        __shared__ uint32_t part[kRows][kWarps];
        if ((t & 31) == 0) part[sub][t >> 5] = top;
        __syncthreads();
        top = part[sub][t & 31 & (kWarps - 1)];
        top = __reduce_max_sync(0xffffffffu, top);
    }
    const bool bad = top >= inf_bits<T>();
    const float amax = unpack2<T>(top).x;
    const float up = amax < 8.6736174e-19f ? 1.8446744e19f : 1.0f;      // 2^-60, 2^64
    // codes 0 for rows of zeros and rows with an infinity or a NaN
    const float inv = (top == 0 || bad) ? 0.0f : __fdiv_rn(127.0f, amax * up);
    if (live && t == 0)
        scales[row] = bad ? __int_as_float(0x7fffffff) : (top == 0 ? 1.0f : __fdiv_rn(amax, 127.0f));
#pragma unroll
    for (int i = 0; i < kVec; ++i)
        if (t + i * TPR < n) q[t + i * TPR] = bad ? make_uint2(0u, 0u) : codes8<T>(v[i], up, inv);
    if constexpr (LONG)
        for (int j = t + kVec * TPR; j < n; j += TPR)
            q[j] = bad ? make_uint2(0u, 0u) : codes8<T>(ld_behind_cached_v4(x + j), up, inv);
}

template <typename T, int TPR, bool LONG>
cudaError_t run(const void *X, int8_t *Q, float *scales, int M, int K, cudaStream_t stream)
{
    constexpr int kThreads = TPR < 256 ? 256 : TPR, kRows = kThreads / TPR;
    const dim3 grid((unsigned)((M + (long long)kRows - 1) / kRows));
    return launch_dependent(quant_tokens_kernel<T, TPR, LONG>, grid, dim3(kThreads), 0, 1, stream,
                            static_cast<const T *>(X), Q, scales, M, K);
}

} // namespace

cudaError_t launch_quant_int8_tokens(const void *X, int8_t *Q, float *scales, int M, int K,
                                     int dtype, cudaStream_t stream)
{
    // the fewest threads whose registers hold the row: 32 values a thread
    QG_DISPATCH_16(dtype, T, {
        if (K <= 32 * 32) return run<T, 32, false>(X, Q, scales, M, K, stream);
        if (K <= 128 * 32) return run<T, 128, false>(X, Q, scales, M, K, stream);
        if (K <= 512 * 32) return run<T, 512, false>(X, Q, scales, M, K, stream);
        return run<T, 512, true>(X, Q, scales, M, K, stream);
    });
}

} // namespace qg
