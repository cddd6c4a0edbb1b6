"""Operands that require gradients: the calls record no graph of their own, so a backward pass that
comes to one of their results has to say so instead of leaving what is upstream without gradients."""
import pytest
import torch

import gemv_w4a16_w8a8_b200 as qg

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
M, F, K = 5, 64, 32


def operands(dtype=torch.float16):
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    X, Wg, Wu = (torch.randn(n, K, generator=g, device=DEV).to(dtype) for n in (M, F, F))
    return X, Wg, Wu


@pytest.mark.parametrize("which", [0, 1, 2])
@pytest.mark.parametrize("kw", [{}, dict(save_preact=True), dict(stream=0), "buffer"])
def test_gated_says_so_at_the_backward_pass(which, kw):
    ops = list(operands())
    want = qg.qgemm_dense_gated(*ops, save_preact=True)
    ops[which].requires_grad_()
    if kw == "buffer":
        kw = dict(H=torch.empty(M, F, dtype=torch.float16, device=DEV))
    got = qg.qgemm_dense_gated(*ops, **kw)
    got = got if isinstance(got, tuple) else (got,)
    torch.cuda.synchronize()
    other = torch.ones(F, device=DEV, requires_grad=True)
    for h, w in zip(got, want):
        assert torch.equal(h.detach(), w)                      # the call itself is the same
        with pytest.raises(RuntimeError, match="qgemm_dense_gated_backward"):
            (h.float() * other).sum().backward()
    if "H" in kw:                                              # the caller's own buffer stays a buffer
        assert got[0].data_ptr() == kw["H"].data_ptr() and not kw["H"].requires_grad
        qg.qgemm_dense_gated(*ops, **kw)


def test_8bit_calls_say_so_too():
    X, Wg, Wu = operands(torch.bfloat16)
    (q, s), (qw, sw) = qg.quant_int8_tokens(X), qg.quant_int8_tokens(Wg)
    bias = torch.zeros(F, dtype=torch.bfloat16, device=DEV, requires_grad=True)
    leaf = sw.clone().requires_grad_()
    for out in (qg.qgemm_w8a8_scaled(q, qw, s, sw, bias=bias, out_dtype=torch.bfloat16),
                qg.qgemm_w8a8_scaled(q, qw, s, leaf), qg.qgemm_w8a8_gated(q, qw, qw, s, sw, leaf),
                qg.quant_int8_tokens(X.clone().requires_grad_())[1]):
        with pytest.raises(RuntimeError, match="no gradient"):
            out.float().sum().backward()


def test_nothing_is_recorded_where_nothing_asks():
    X, Wg, Wu = operands()
    assert not qg.qgemm_dense_gated(X, Wg, Wu).requires_grad
    X.requires_grad_()
    with torch.no_grad():
        H, G, U = qg.qgemm_dense_gated(X, Wg, Wu, save_preact=True)
        assert not (H.requires_grad or G.requires_grad or U.requires_grad)
    # gradients by hand, on parameters: plain tensors, outside of no_grad too
    H, G, U = qg.qgemm_dense_gated(X, Wg, Wu, save_preact=True)
    for t in qg.qgemm_dense_gated_backward(torch.ones_like(H).detach(), X, Wg, Wu, G, U):
        assert not t.requires_grad and bool(torch.isfinite(t).all())


def test_inside_an_autograd_function():
    """How a training program has them: forward and backward of a Function of its own."""
    class Gated(torch.autograd.Function):
        @staticmethod
        def forward(ctx, X, Wg, Wu):
            H, G, U = qg.qgemm_dense_gated(X, Wg, Wu, save_preact=True)
            ctx.save_for_backward(X, Wg, Wu, G, U)
            return H

        @staticmethod
        def backward(ctx, dH):
            return qg.qgemm_dense_gated_backward(dH.contiguous(), *ctx.saved_tensors)

    leaves = [t.requires_grad_() for t in operands()]
    dH = torch.randn(M, F, device=DEV).half()
    Gated.apply(*leaves).backward(dH)
    wide = [t.detach().double().requires_grad_() for t in leaves]
    (torch.nn.functional.silu(wide[0] @ wide[1].T) * (wide[0] @ wide[2].T)).backward(dH.double())
    for got, want in zip(leaves, wide):
        assert float((got.grad.double() - want.grad).norm() / want.grad.norm()) < 2e-3
