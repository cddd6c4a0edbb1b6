"""More than 2^31 elements in an input or an output of each call: rows on both sides of that border
against plain 64-bit forms."""
import numpy as np
import pytest
import torch

import ffn_ref as R
import gemv_w4a16_w8a8_b200 as qg
from test_gpu_ffn import DEV, codes, normal, rng, scaled_case

pytestmark = pytest.mark.gpu
M, F = 140000, 16000                       # 2.24e9
ROWS = [0, 67107, 134217, 134218, 139999]  # element 2^31 is in row 134217


def check(got, ref_bound, what):
    """R.check where the gradients of 140000 tokens may leave the type: what is 65520 or more, half a step
    past fp16's largest, rounds to an infinity. So a value that is that large by its bound has to be
    one, one that may be is free, and the others are within their bounds."""
    ref, bound = ref_bound
    past = 65520.0 if got.dtype == torch.float16 else float("inf")
    sure, may = ref.abs() - bound >= past, ref.abs() + bound >= past
    assert torch.equal(got[sure].double(), torch.sign(ref[sure]) * float("inf")), what
    R.check(torch.where(may, torch.zeros_like(ref), got.double()),
            (torch.where(may, torch.zeros_like(ref), ref), bound), what)


@pytest.fixture(autouse=True)
def memory():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB of device memory")
    yield
    torch.cuda.empty_cache()


def test_quant():
    x = normal((300000, 8192), 1.0, torch.float16, rng(1))
    q, s = qg.quant_int8_tokens(x)
    for m in (0, 131071, 262143, 262144, 299999):
        rq, rs = R.quant(x[m:m + 1].float().cpu().numpy())
        assert np.array_equal(q[m:m + 1].cpu().numpy(), rq) and np.array_equal(s[m:m + 1].cpu().numpy(), rs), m


@pytest.mark.parametrize("tokens,N", [(3, 720_000_001), (64, 33_700_000)])
def test_scaled_few_tokens(tokens, N):
    A, W, sa, sw, b = scaled_case(tokens, N, 16, torch.bfloat16, True)
    C = qg.qgemm_w8a8_scaled(A, W, sa, sw, bias=b, out_dtype=torch.bfloat16)
    qg.qgemm_sync_check()
    for at in (0, N // 2, N - 1000):
        n = slice(at, at + 1000)
        R.check(C[:, n], R.scaled(A, W[n], sa, sw[n], b[n], torch.bfloat16), at)


def test_gated8():
    g = rng(2)
    A, Wg, Wu = codes(M, 16, g), codes(F, 16, g), codes(F, 16, g)
    sa = torch.rand(M, generator=g, device=DEV) + 0.5
    sg, su = ((torch.rand(F, generator=g, device=DEV) + 0.5) * 1.5 / (74.0 * 74.0 * 4) for _ in range(2))
    H = qg.qgemm_w8a8_gated(A, Wg, Wu, sa, sg, su)
    qg.qgemm_sync_check()
    R.check(H[ROWS], R.gated8(A[ROWS], Wg, Wu, sa[ROWS], sg, su, "silu", torch.float16))


@pytest.mark.parametrize("width", [F, F - 1])
def test_gated_and_its_gradients(width):
    """Rows of a multiple of eight values, and odd ones; fp16 with its first pass, then bf16."""
    K = 8
    for dtype in (torch.float16, torch.bfloat16):
        g = rng(width)
        X = normal((M, K), 1.0, dtype, g)
        Wg, Wu = (normal((width, K), 0.5, dtype, g) for _ in range(2))
        H, G, U = qg.qgemm_dense_gated(X, Wg, Wu, save_preact=True)
        qg.qgemm_sync_check()
        ref = R.gated(X[ROWS], Wg, Wu, "silu")
        for name, got in dict(H=H, G=G, U=U).items():
            R.check(got[ROWS], ref[name], name)
        # H stands for the gradient that comes back
        dX, dWg, dWu = qg.qgemm_dense_gated_backward(H, X, Wg, Wu, G, U)
        qg.qgemm_sync_check()
        want = R.backward(H[ROWS], X[ROWS], Wg, Wu, G[ROWS], U[ROWS], "silu")
        check(dX[ROWS], want["dX"], "dX")
        cols = [0, 1, 777, width - 1]
        h, gg, u = (t[:, cols].contiguous() for t in (H, G, U))
        want = R.backward(h, X, Wg[cols], Wu[cols], gg, u, "silu")
        check(dWg[cols], want["dWg"], "dWg")
        check(dWu[cols], want["dWu"], "dWu")
        del H, G, U, dX, h, gg, u
        torch.cuda.empty_cache()
