"""Every way in which the gradients and the forward products are cut into tiles, parts, waves and
launches, on the GPU against plain 64-bit forms. test_ffn_plan.py holds the sizes to the plans that
they stand for."""
import pytest
import torch

import ffn_ref as R
import gemv_w4a16_w8a8_b200 as qg
from test_gpu_ffn import ACTS, DEV, TYPES, backward_case, codes, guarded, normal, rng, scaled_case

pytestmark = pytest.mark.gpu

# plan of the gradients: (M, F, K)
GRADIENTS = {
    "few-token dX above 64 tokens": (65, 640, 1312),
    "few-token dX, three waves of the weights' gradients": (77, 4114, 1096),
    "few-token dX, many token tiles, the weights' gradients in parts": (3643, 1199, 8),
    "two launches, dX in parts": (512, 11008, 512),
    "two launches, the weights' gradients in parts": (4108, 49, 1816),
    "two launches, both in parts": (4047, 1205, 8),
    "two launches, three waves of dX": (2561, 17, 3352),
    "two launches, three waves of each": (2843, 1357, 3888),
    "two launches, 128 columns, two waves": (2728, 682, 1568),
    "one launch, no round of its own for the weights": (265, 16, 8),
    "one launch, no round of its own, three waves": (5024, 16, 800),
    "one launch, two rounds of its own, dX in parts": (300, 4096, 512),
    "one launch, three rounds of its own, four waves": (66, 562, 3512),
    "one launch, six rounds of its own": (1024, 4096, 2048),
    "one launch, both in parts": (1536, 761, 8),
    "one launch, both in parts, two waves of dX": (5252, 1826, 8),
    "one launch, three waves of dX": (1935, 19, 3352),
}
# forward products by tiles, three waves or more of them: (M, N, K)
SCALED = [(2049, 4097, 272), (3001, 5003, 272), (1500, 8190, 144)]
GATED = [(2600, 2999, 264), (1700, 4098, 136), (2304, 4096, 200)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("plan", GRADIENTS)
def test_gradients(plan, dtype):
    M, F, K = GRADIENTS[plan]
    act = ACTS[(M + F) % 3]
    c = backward_case(M, F, K, dtype)
    outs = {"dX": guarded((M, K), dtype), "dWg": guarded((F, K), dtype), "dWu": guarded((F, K), dtype)}
    n = qg.qgemm_dense_gated_backward_workspace_bytes(M, F, K)
    ws = torch.full((n + 4096,), 0xFF, dtype=torch.uint8, device=DEV)       # NaN wherever it is read first
    qg.qgemm_dense_gated_backward(**c, act=act, workspace=ws[:n], **{k: v for k, (v, _) in outs.items()})
    qg.qgemm_sync_check()
    assert bool((ws[n:] == 0xFF).all()), "wrote past the workspace"
    ref = R.backward(**c, act=act)
    for k, (v, guard) in outs.items():
        guard()
        R.check(v, ref[k], k)
    # the same bits from a second call, and from calls that ask for one of the two alone
    dX, _, _ = qg.qgemm_dense_gated_backward(**c, act=act, need_dw=False, workspace=ws[:n])
    _, dWg, dWu = qg.qgemm_dense_gated_backward(**c, act=act, need_dx=False, workspace=ws[:n])
    for k, v in dict(dX=dX, dWg=dWg, dWu=dWu).items():
        assert torch.equal(v, outs[k][0]), k


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", SCALED)
def test_scaled(M, N, K, dtype):
    """Scales and bias of the next tile are loaded while one is written: all of the result."""
    A, W, sa, sw, b = scaled_case(M, N, K, dtype, True)
    C, guard = guarded((M, N), dtype)
    qg.qgemm_w8a8_scaled(A, W, sa, sw, bias=b, C=C)
    qg.qgemm_sync_check()
    guard()
    step = (A.double() @ W.double().T).to(torch.int32).float() * sa[:, None] * sw + b.float()
    assert torch.equal(C, step.to(dtype))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,F,K", GATED)
def test_gated(M, F, K, dtype):
    act = ACTS[(M + F) % 3]
    g = rng(M + F)
    X = normal((M, K), 1.0, dtype, g)
    Wg, Wu = (normal((F, K), 1.5 / K ** 0.5, dtype, g) for _ in range(2))
    outs = {n: guarded((M, F), dtype) for n in ("H", "G", "U")}
    qg.qgemm_dense_gated(X, Wg, Wu, act=act, **{n: v for n, (v, _) in outs.items()})
    qg.qgemm_sync_check()
    ref = R.gated(X, Wg, Wu, act)
    for n, (v, guard) in outs.items():
        guard()
        R.check(v, ref[n], n)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,F,K", [(2600, 2999, 272), (1700, 4098, 144), (2304, 4096, 208)])
def test_gated8(M, F, K, dtype):
    act = ACTS[(M + F) % 3]
    g = rng(M + F)
    A, Wg, Wu = codes(M, K, g), codes(F, K, g), codes(F, K, g)
    s = 1.5 / (74.0 * 74.0 * K ** 0.5)
    sa = torch.rand(M, generator=g, device=DEV) + 0.5
    sg, su = ((torch.rand(F, generator=g, device=DEV) + 0.5) * s for _ in range(2))
    H, guard = guarded((M, F), dtype)
    qg.qgemm_w8a8_gated(A, Wg, Wu, sa, sg, su, H=H, act=act)
    qg.qgemm_sync_check()
    guard()
    R.check(H, R.gated8(A, Wg, Wu, sa, sg, su, act, dtype))
