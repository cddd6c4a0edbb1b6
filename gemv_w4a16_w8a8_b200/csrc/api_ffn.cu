// C-ABI entry points of token quantisation, the scaled W8A8 matmul and the gated feed-forward
// block: argument checks, then the launchers of ffn.cuh.
#include <initializer_list>

#include "ffn.cuh"

namespace qg {
namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool bad_dtype(int dtype) { return dtype != QG_F16 && dtype != QG_BF16; }
bool bad_act(int act) { return act != QG_ACT_SILU && act != QG_ACT_GELU && act != QG_ACT_GELU_TANH; }

qg_status launched(cudaError_t e)
{
    if (e == cudaSuccess) return QG_OK;
    cudaGetLastError();
    return QG_ERR_CUDA;
}

constexpr int kMaxInt8K = 131072;      // 128 * 128 * K < 2^31 below it
// Rows and columns of the products: their kernels and plans round sizes up to whole tiles, and step
// past the last one by less than 4096, in int arithmetic.
constexpr int kMaxSize = 0x7fffffff - 4095;

bool too_large(int M, int N, int K) { return M > kMaxSize || N > kMaxSize || K > kMaxSize; }

// A buffer of a call; null where the call has none
struct Buffer {
    const void *p;
    size_t bytes;
};

// Whether an output shares memory with an input or with another output
bool overlap(std::initializer_list<Buffer> outputs, std::initializer_list<Buffer> inputs)
{
    auto meet = [](const Buffer &a, const Buffer &b) {
        const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
        return a.p && b.p && (x < y ? y - x < a.bytes : x - y < b.bytes);
    };
    for (const Buffer *o = outputs.begin(); o != outputs.end(); ++o) {
        for (const Buffer &i : inputs)
            if (meet(*o, i)) return true;
        for (const Buffer *q = o + 1; q != outputs.end(); ++q)
            if (meet(*o, *q)) return true;
    }
    return false;
}

size_t round256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }

int padded_f(int F) { return (F + 7) & ~7; }

// bytes of dG (and of dU): M rows of padded_f(F) 16-bit values
size_t grad_bytes(int M, int F) { return round256((size_t)M * padded_f(F) * 2); }

constexpr size_t kScaleBytes = (kGradScale * 4 + 255) / 256 * 256;

size_t backward_bytes(const GradPlan &plan, int M, int F, int K)
{
    return 2 * grad_bytes(M, F) + kScaleBytes + round256(grad_part_bytes(plan, M, F, K));
}

} // namespace
} // namespace qg

using namespace qg;

extern "C" {

qg_status quant_int8_tokens(const void *X, int8_t *Q, float *scales, int M, int K, int dtype,
                            cudaStream_t stream)
{
    if (!X || !Q || !scales || M <= 0 || K <= 0 || bad_dtype(dtype)) return QG_ERR_INVALID_ARG;
    if (K % 8) return QG_ERR_UNSUPPORTED_SHAPE;
    if (!aligned(X, 16) || !aligned(Q, 16) || !aligned(scales, 4)) return QG_ERR_ALIGNMENT;
    const size_t mk = (size_t)M * K;
    if (overlap({{Q, mk}, {scales, (size_t)M * 4}}, {{X, mk * 2}})) return QG_ERR_INVALID_ARG;
    int sms = 0;
    unsigned int *err = nullptr;
    const qg_status s = current_device(&sms, &err);
    if (s != QG_OK) return s;
    return launched(launch_quant_int8_tokens(X, Q, scales, M, K, dtype, stream));
}

qg_status qgemm_w8a8_scaled(const int8_t *A, const int8_t *W, const float *a_scales,
                            const float *w_scales, const void *bias, void *C, int M, int N, int K,
                            int dtype, cudaStream_t stream)
{
    if (!A || !W || !a_scales || !w_scales || !C || M <= 0 || N <= 0 || K <= 0 || bad_dtype(dtype))
        return QG_ERR_INVALID_ARG;
    if (K % 16 || K >= kMaxInt8K || too_large(M, N, K)) return QG_ERR_UNSUPPORTED_SHAPE;
    if (!aligned(A, 16) || !aligned(W, 16) || !aligned(C, 16) || !aligned(a_scales, 4) ||
        !aligned(w_scales, 4) || !aligned(bias, 2))
        return QG_ERR_ALIGNMENT;
    if (overlap({{C, (size_t)M * N * 2}},
                {{A, (size_t)M * K}, {W, (size_t)N * K}, {a_scales, (size_t)M * 4},
                 {w_scales, (size_t)N * 4}, {bias, (size_t)N * 2}}))
        return QG_ERR_INVALID_ARG;
    int sms = 0;
    unsigned int *err = nullptr;
    const qg_status s = current_device(&sms, &err);
    if (s != QG_OK) return s;
    const ScaledProblem p{A, W, nullptr, a_scales, w_scales, nullptr, bias, C, M, N, K, 0, dtype};
    return launched(launch_w8a8_scaled(p, err, stream));
}

qg_status qgemm_w8a8_gated(const int8_t *A, const int8_t *Wg, const int8_t *Wu,
                           const float *a_scales, const float *g_scales, const float *u_scales,
                           void *H, int M, int F, int K, int act, int dtype, cudaStream_t stream)
{
    if (!A || !Wg || !Wu || !a_scales || !g_scales || !u_scales || !H || M <= 0 || F <= 0 ||
        K <= 0 || bad_dtype(dtype) || bad_act(act))
        return QG_ERR_INVALID_ARG;
    if (K % 16 || K >= kMaxInt8K || too_large(M, F, K)) return QG_ERR_UNSUPPORTED_SHAPE;
    if (!aligned(A, 16) || !aligned(Wg, 16) || !aligned(Wu, 16) || !aligned(H, 16) ||
        !aligned(a_scales, 4) || !aligned(g_scales, 4) || !aligned(u_scales, 4))
        return QG_ERR_ALIGNMENT;
    if (overlap({{H, (size_t)M * F * 2}},
                {{A, (size_t)M * K}, {Wg, (size_t)F * K}, {Wu, (size_t)F * K},
                 {a_scales, (size_t)M * 4}, {g_scales, (size_t)F * 4}, {u_scales, (size_t)F * 4}}))
        return QG_ERR_INVALID_ARG;
    int sms = 0;
    unsigned int *err = nullptr;
    const qg_status s = current_device(&sms, &err);
    if (s != QG_OK) return s;
    const ScaledProblem p{A, Wg, Wu, a_scales, g_scales, u_scales, nullptr, H, M, F, K, act, dtype};
    return launched(launch_w8a8_scaled(p, err, stream));
}

qg_status qgemm_dense_gated(const void *X, const void *Wg, const void *Wu, void *H, void *G,
                            void *U, int M, int F, int K, int act, int dtype,
                            cudaStream_t stream)
{
    if (!X || !Wg || !Wu || !H || !G != !U || M <= 0 || F <= 0 || K <= 0 || bad_dtype(dtype) ||
        bad_act(act))
        return QG_ERR_INVALID_ARG;
    if (K % 8 || too_large(M, F, K)) return QG_ERR_UNSUPPORTED_SHAPE;
    if (!aligned(X, 16) || !aligned(Wg, 16) || !aligned(Wu, 16) || !aligned(H, 16) ||
        !aligned(G, 16) || !aligned(U, 16))
        return QG_ERR_ALIGNMENT;
    const size_t mf = (size_t)M * F * 2, fk = (size_t)F * K * 2;
    if (overlap({{H, mf}, {G, mf}, {U, mf}}, {{X, (size_t)M * K * 2}, {Wg, fk}, {Wu, fk}}))
        return QG_ERR_INVALID_ARG;
    int sms = 0;
    unsigned int *err = nullptr;
    const qg_status s = current_device(&sms, &err);
    if (s != QG_OK) return s;
    const GatedProblem p{X, Wg, Wu, H, G, U, M, F, K, act, dtype};
    return launched(launch_dense_gated(p, err, stream));
}

size_t qgemm_dense_gated_backward_workspace_bytes(int M, int F, int K)
{
    if (M <= 0 || F <= 0 || K <= 0 || K % 8 || too_large(M, F, K)) return 0;
    return backward_bytes(plan_gated_backward(M, F, K), M, F, K);
}

qg_status qgemm_dense_gated_backward(const void *dH, const void *X, const void *Wg, const void *Wu,
                                     const void *G, const void *U, void *dX, void *dWg, void *dWu,
                                     int M, int F, int K, int act, int dtype, void *workspace,
                                     size_t workspace_bytes, cudaStream_t stream)
{
    if (!dH || !X || !Wg || !Wu || !G || !U || !dWg != !dWu || (!dX && !dWg) || M <= 0 || F <= 0 ||
        K <= 0 || bad_dtype(dtype) || bad_act(act) || !workspace)
        return QG_ERR_INVALID_ARG;
    if (K % 8 || too_large(M, F, K)) return QG_ERR_UNSUPPORTED_SHAPE;
    if (!aligned(dH, 16) || !aligned(X, 16) || !aligned(Wg, 16) || !aligned(Wu, 16) ||
        !aligned(G, 16) || !aligned(U, 16) || !aligned(dX, 16) || !aligned(dWg, 16) ||
        !aligned(dWu, 16) || !aligned(workspace, 256))
        return QG_ERR_ALIGNMENT;
    const GradPlan plan = plan_gated_backward(M, F, K);
    const size_t need = backward_bytes(plan, M, F, K);
    if (workspace_bytes < need) return QG_ERR_SCRATCH_TOO_SMALL;
    const size_t mf = (size_t)M * F * 2, mk = (size_t)M * K * 2, fk = (size_t)F * K * 2;
    if (overlap({{dX, mk}, {dWg, fk}, {dWu, fk}, {workspace, need}},
                {{dH, mf}, {X, mk}, {Wg, fk}, {Wu, fk}, {G, mf}, {U, mf}}))
        return QG_ERR_INVALID_ARG;
    int sms = 0;
    unsigned int *err = nullptr;
    const qg_status s = current_device(&sms, &err);
    if (s != QG_OK) return s;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    uint8_t *scale = ws + 2 * grad_bytes(M, F);
    const GatedGrad p{dH, X, Wg, Wu, G, U, dX, dWg, dWu, ws, ws + grad_bytes(M, F), M, F, K, act,
                      dtype, padded_f(F), reinterpret_cast<float *>(scale + kScaleBytes),
                      reinterpret_cast<float *>(scale), plan};
    return launched(launch_gated_backward(p, err, stream));
}

} // extern "C"
