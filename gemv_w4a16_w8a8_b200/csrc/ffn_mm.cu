// Matmuls of the scaled W8A8 product and of the gated feed-forward block's forward and backward
// passes: a plain shared-memory tile on the CUDA cores, any strides, up to two weight matrices
// that share the activations (gate and up) or two products summed into one result (dX).
#include <algorithm>

#include "ffn.cuh"

namespace qg {
namespace {

constexpr int kTile = 64, kStep = 16;

template <typename T> struct AccOf { using type = float; };
template <> struct AccOf<int8_t> { using type = int; };

__device__ __forceinline__ int widen(int8_t v) { return v; }
__device__ __forceinline__ float widen(__half v) { return to_f32(v); }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return to_f32(v); }

// a matrix by strides: element (i, k) at p[i * si + k * sk]
template <typename T> struct View {
    const T *p;
    size_t si, sk;
};

// D_j[m, n] = sum_k A_s[m, k] B_{j,s}[n, k] over NB results j (A shared) and NS summed products s
template <typename T, int NB, int NS, typename Epi>
__global__ void __launch_bounds__(256) tile_kernel(View<T> a0, View<T> a1, View<T> b0, View<T> b1,
                                                   int M, int N, int K, int tiles_n, Epi epi)
{
    using Acc = typename AccOf<T>::type;
    __shared__ Acc sa[kStep][kTile + 1], sb[NB][kStep][kTile + 1];
    const int m0 = (blockIdx.x / tiles_n) * kTile, n0 = (blockIdx.x % tiles_n) * kTile;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    Acc acc[NB][4][4] = {};
    for (int s = 0; s < NS; ++s) {
        const View<T> a = s ? a1 : a0;
        for (int k0 = 0; k0 < K; k0 += kStep) {
            for (int e = threadIdx.x; e < kTile * kStep; e += 256) {
                const int i = e / kStep, k = e % kStep;
                const bool in = k0 + k < K;
                sa[k][i] = in && m0 + i < M ? widen(a.p[(m0 + i) * a.si + (k0 + k) * a.sk]) : Acc(0);
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                    const View<T> b = (j + s) ? b1 : b0;
                    sb[j][k][i] = in && n0 + i < N ? widen(b.p[(n0 + i) * b.si + (k0 + k) * b.sk]) : Acc(0);
                }
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kStep; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < NB; ++j)
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            acc[j][i][q] += sa[k][ty + 16 * i] * sb[j][k][tx + 16 * q];
            __syncthreads();
        }
    }
    for (int i = 0; i < 4; ++i)
        for (int q = 0; q < 4; ++q) {
            const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * q;
            if (m < M && n < N) epi(m, n, acc[0][i][q], acc[NB - 1][i][q]);
        }
}

template <typename T, int NB, int NS, typename Epi>
cudaError_t run_tiles(View<T> a0, View<T> a1, View<T> b0, View<T> b1, int M, int N, int K,
                      const Epi &epi, cudaStream_t stream)
{
    const int tm = (M + kTile - 1) / kTile, tn = (N + kTile - 1) / kTile;
    tile_kernel<T, NB, NS, Epi><<<(unsigned)tm * tn, 256, 0, stream>>>(a0, a1, b0, b1, M, N, K, tn, epi);
    return cudaGetLastError();
}

template <typename T> struct ScaledEpi {
    const float *sa, *sw;
    const T *bias;
    T *C;
    int N;
    __device__ void operator()(int m, int n, int v, int) const
    {
        float r = __fmul_rn(__fmul_rn(__int2float_rn(v), sa[m]), sw[n]);
        if (bias) r = __fadd_rn(r, to_f32(bias[n]));
        C[(size_t)m * N + n] = from_f32<T>(r);
    }
};
template <typename T, int ACT> struct Gated8Epi {
    const float *sa, *sg, *su;
    T *H;
    int N;
    __device__ void operator()(int m, int n, int g, int u) const
    {
        const float gf = __fmul_rn(__fmul_rn(__int2float_rn(g), sa[m]), sg[n]);
        const float uf = __fmul_rn(__fmul_rn(__int2float_rn(u), sa[m]), su[n]);
        H[(size_t)m * N + n] = from_f32<T>(act_value<ACT>(gf) * uf);
    }
};
template <typename T, int ACT> struct GatedEpi {
    T *H, *G, *U;
    int N;
    __device__ void operator()(int m, int n, float g, float u) const
    {
        const size_t at = (size_t)m * N + n;
        H[at] = from_f32<T>(act_value<ACT>(g) * u);
        if (G) {
            G[at] = from_f32<T>(g);
            U[at] = from_f32<T>(u);
        }
    }
};
template <typename T> struct StoreEpi {
    T *C;
    int N;
    __device__ void operator()(int m, int n, float v, float) const
    {
        C[(size_t)m * N + n] = from_f32<T>(v);
    }
};

// dG = dH U act'(G), dU = dH act(G), rows of Fp elements in the workspace
template <typename T, int ACT>
__global__ void grad_act_kernel(const T *dH, const T *G, const T *U, T *dG, T *dU, int F, int Fp)
{
    const size_t in = (size_t)blockIdx.x * F, out = (size_t)blockIdx.x * Fp;
    for (int f = threadIdx.x; f < F; f += blockDim.x) {
        float v, d;
        act_both<ACT>(to_f32(G[in + f]), v, d);
        const float dh = to_f32(dH[in + f]);
        dG[out + f] = from_f32<T>(dh * to_f32(U[in + f]) * d);
        dU[out + f] = from_f32<T>(dh * v);
    }
}

} // namespace

cudaError_t launch_w8a8_scaled(const ScaledProblem &p, int, unsigned int *, cudaStream_t stream)
{
    const size_t K = p.K;
    const View<int8_t> a{p.A, K, 1}, w{p.W, K, 1}, w1{p.W1, K, 1};
    QG_DISPATCH_16(p.dtype, T, {
        if (!p.W1)
            return run_tiles<int8_t, 1, 1>(a, a, w, w, p.M, p.N, p.K,
                                           ScaledEpi<T>{p.sa, p.sw, (const T *)p.bias, (T *)p.C, p.N},
                                           stream);
        QG_DISPATCH_ACT(p.act, ACT, {
            return run_tiles<int8_t, 2, 1>(a, a, w, w1, p.M, p.N, p.K,
                                           Gated8Epi<T, ACT>{p.sa, p.sw, p.sw1, (T *)p.C, p.N}, stream);
        });
    });
}

cudaError_t launch_dense_gated(const GatedProblem &p, int, unsigned int *, cudaStream_t stream)
{
    const size_t K = p.K;
    QG_DISPATCH_16(p.dtype, T, {
        const View<T> x{(const T *)p.X, K, 1}, g{(const T *)p.Wg, K, 1}, u{(const T *)p.Wu, K, 1};
        QG_DISPATCH_ACT(p.act, ACT, {
            return run_tiles<T, 2, 1>(x, x, g, u, p.M, p.F, p.K,
                                      GatedEpi<T, ACT>{(T *)p.H, (T *)p.G, (T *)p.U, p.F}, stream);
        });
    });
}

cudaError_t launch_gated_backward(const GatedGrad &p, int, unsigned int *, cudaStream_t stream)
{
    const size_t K = p.K, Fp = p.Fp;
    QG_DISPATCH_16(p.dtype, T, {
        QG_DISPATCH_ACT(p.act, ACT, {
            grad_act_kernel<T, ACT><<<p.M, 256, 0, stream>>>((const T *)p.dH, (const T *)p.G,
                                                             (const T *)p.U, (T *)p.dG, (T *)p.dU,
                                                             p.F, p.Fp);
        });
        cudaError_t e = cudaGetLastError();
        const View<T> dg{(const T *)p.dG, Fp, 1}, du{(const T *)p.dU, Fp, 1};
        const View<T> wg{(const T *)p.Wg, 1, K}, wu{(const T *)p.Wu, 1, K};
        if (e == cudaSuccess && p.dX)
            e = run_tiles<T, 1, 2>(dg, du, wg, wu, p.M, p.K, p.F, StoreEpi<T>{(T *)p.dX, p.K}, stream);
        const View<T> dgt{(const T *)p.dG, 1, Fp}, dut{(const T *)p.dU, 1, Fp}, x{(const T *)p.X, 1, K};
        if (e == cudaSuccess && p.dWg)
            e = run_tiles<T, 1, 1>(dgt, dgt, x, x, p.F, p.K, p.M, StoreEpi<T>{(T *)p.dWg, p.K}, stream);
        if (e == cudaSuccess && p.dWu)
            e = run_tiles<T, 1, 1>(dut, dut, x, x, p.F, p.K, p.M, StoreEpi<T>{(T *)p.dWu, p.K}, stream);
        return e;
    });
}

} // namespace qg
