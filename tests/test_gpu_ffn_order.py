"""Calls that follow one another without a synchronisation, on data that changes with every one of
them and through buffers that are used again: each kernel starts before its predecessor has ended,
and has to read what that one wrote. The reference is the same calls with the device waited for in
between: the same bits."""
import pytest
import torch

import gemv_w4a16_w8a8_b200 as qg

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TURNS = 6


def rng(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(shape, spread, dtype, g):
    return (torch.randn(shape, generator=g, device=DEV) * spread).to(dtype)


def same(unsynchronised, synchronised):
    for turn, (a, b) in enumerate(zip(unsynchronised, synchronised)):
        for name in a:
            assert torch.equal(a[name], b[name]), (turn, name)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("M,F,K", [(1, 1376, 512), (48, 640, 1024), (300, 1376, 512), (3000, 1376, 512), (2500, 2752, 1024)])
def test_8bit_block_on_changing_data(M, F, K, dtype):
    """quantise -> gate and up -> quantise -> down, twice the scales' and codes' buffers a turn."""
    g = rng(M)
    xs = [normal((M, K), 0.5 + i, dtype, g) for i in range(TURNS)]
    weights = []
    for rows, cols in ((F, K), (F, K), (K, F)):
        weights += list(qg.quant_int8_tokens(normal((rows, cols), cols ** -0.5, dtype, g)))
    Wg, sg, Wu, su, Wd, sd = weights
    torch.cuda.synchronize()

    def turns(wait):
        q, s = torch.zeros(M, K, dtype=torch.int8, device=DEV), torch.zeros(M, device=DEV)
        q2, h = torch.zeros(M, F, dtype=torch.int8, device=DEV), torch.zeros(M, F, dtype=dtype, device=DEV)
        out = [dict(Y=torch.zeros(M, K, dtype=dtype, device=DEV)) for _ in xs]
        torch.cuda.synchronize()
        for x, o in zip(xs, out):
            for call in (lambda: qg.quant_int8_tokens(x, Q=q, scales=s),
                         lambda: qg.qgemm_w8a8_gated(q, Wg, Wu, s, sg, su, H=h),
                         lambda: qg.quant_int8_tokens(h, Q=q2, scales=s),
                         lambda: qg.qgemm_w8a8_scaled(q2, Wd, s, sd, C=o["Y"])):
                call()
                if wait:
                    torch.cuda.synchronize()
        qg.qgemm_sync_check()
        return out

    want = turns(True)
    for _ in range(3):
        same(turns(False), want)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("M,F,K", [(1, 1376, 512), (40, 1371, 520), (77, 1371, 520), (300, 1374, 512),
                                   (3000, 1376, 512), (3000, 1371, 512), (2500, 688, 1024)])
def test_training_steps_on_changing_data(M, F, K, dtype):
    """Forward with saved pre-activations, then its gradients: H, G, U and the workspace are used
    again by the next turn."""
    g = rng(M + F)
    xs = [normal((M, K), 0.5 + 0.1 * i, dtype, g) for i in range(TURNS)]
    Wg, Wu = (normal((F, K), K ** -0.5, dtype, g) for _ in range(2))
    ws = torch.empty(qg.qgemm_dense_gated_backward_workspace_bytes(M, F, K), dtype=torch.uint8, device=DEV)

    def turns(wait):
        H, G, U = (torch.zeros(M, F, dtype=dtype, device=DEV) for _ in range(3))
        out = [dict(dX=torch.zeros(M, K, dtype=dtype, device=DEV),
                    dWg=torch.zeros(F, K, dtype=dtype, device=DEV),
                    dWu=torch.zeros(F, K, dtype=dtype, device=DEV)) for _ in xs]
        torch.cuda.synchronize()
        for x, o in zip(xs, out):
            # H stands for the gradient that comes back from what follows
            for call in (lambda: qg.qgemm_dense_gated(x, Wg, Wu, H=H, G=G, U=U),
                         lambda: qg.qgemm_dense_gated_backward(H, x, Wg, Wu, G, U, workspace=ws, **o)):
                call()
                if wait:
                    torch.cuda.synchronize()
        qg.qgemm_sync_check()
        return out

    want = turns(True)
    assert all(bool(torch.isfinite(v).all()) for o in want for v in o.values())
    for _ in range(3):
        same(turns(False), want)
