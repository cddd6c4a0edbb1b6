"""Token quantisation, the scaled W8A8 matmul and the gated feed-forward block without a GPU: every
refusal comes before a device is touched, from the C entry points and from the Python binding."""
import ctypes

import pytest
import torch

import gemv_w4a16_w8a8_b200 as qg

# fake, aligned device addresses: every call below must fail validation (or the device probe)
# before it could dereference them
P = [ctypes.c_void_p(0x10000 * i) for i in range(1, 11)]
ODD = ctypes.c_void_p(0x10008)
ODD4 = ctypes.c_void_p(0x10002)


def quant(M=4, K=64, dtype=0, x=P[0], q=P[1], s=P[2]):
    return qg.lib().quant_int8_tokens(x, q, s, M, K, dtype, None)


def scaled(M=4, N=64, K=64, dtype=0, a=P[0], w=P[1], sa=P[2], sw=P[3], b=None, c=P[5]):
    return qg.lib().qgemm_w8a8_scaled(a, w, sa, sw, b, c, M, N, K, dtype, None)


def gated8(M=4, F=64, K=64, act=0, dtype=0, a=P[0], g=P[1], u=P[2], sa=P[3], sg=P[4], su=P[5], h=P[6]):
    return qg.lib().qgemm_w8a8_gated(a, g, u, sa, sg, su, h, M, F, K, act, dtype, None)


def gated(M=4, F=64, K=64, act=0, dtype=0, x=P[0], wg=P[1], wu=P[2], h=P[3], g=None, u=None):
    return qg.lib().qgemm_dense_gated(x, wg, wu, h, g, u, M, F, K, act, dtype, None)


def backward(M=4, F=64, K=64, act=0, dtype=0, dh=P[0], x=P[1], wg=P[2], wu=P[3], g=P[4], u=P[5],
             dx=P[6], dwg=P[7], dwu=P[8], ws=P[9], nbytes=1 << 30):
    return qg.lib().qgemm_dense_gated_backward(dh, x, wg, wu, g, u, dx, dwg, dwu, M, F, K, act,
                                               dtype, ws, nbytes, None)


INVALID, ALIGN, SHAPE = qg.QG_ERR_INVALID_ARG, qg.QG_ERR_ALIGNMENT, qg.QG_ERR_UNSUPPORTED_SHAPE


@pytest.mark.parametrize("kw,status", [
    (dict(M=0), INVALID), (dict(K=0), INVALID), (dict(K=-8), INVALID), (dict(dtype=2), INVALID),
    (dict(x=None), INVALID), (dict(q=None), INVALID), (dict(s=None), INVALID),
    (dict(K=63), SHAPE), (dict(x=ODD), ALIGN), (dict(q=ODD), ALIGN), (dict(s=ODD4), ALIGN)])
def test_quant_refuses(kw, status):
    assert quant(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(M=0), INVALID), (dict(N=-1), INVALID), (dict(K=0), INVALID), (dict(dtype=-1), INVALID),
    (dict(a=None), INVALID), (dict(w=None), INVALID), (dict(sa=None), INVALID),
    (dict(sw=None), INVALID), (dict(c=None), INVALID),
    (dict(K=72), SHAPE), (dict(K=131072), SHAPE),
    (dict(a=ODD), ALIGN), (dict(w=ODD), ALIGN), (dict(c=ODD), ALIGN), (dict(sa=ODD4), ALIGN),
    (dict(sw=ODD4), ALIGN), (dict(b=ctypes.c_void_p(0x10001)), ALIGN)])
def test_scaled_refuses(kw, status):
    assert scaled(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), INVALID), (dict(F=0), INVALID), (dict(act=3), INVALID), (dict(dtype=5), INVALID),
    (dict(g=None), INVALID), (dict(u=None), INVALID), (dict(su=None), INVALID), (dict(h=None), INVALID),
    (dict(K=40), SHAPE), (dict(K=131072), SHAPE), (dict(u=ODD), ALIGN), (dict(h=ODD), ALIGN),
    (dict(su=ODD4), ALIGN)])
def test_gated8_refuses(kw, status):
    assert gated8(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(M=0), INVALID), (dict(F=0), INVALID), (dict(act=-1), INVALID), (dict(dtype=2), INVALID),
    (dict(x=None), INVALID), (dict(wu=None), INVALID), (dict(h=None), INVALID),
    (dict(g=P[4]), INVALID), (dict(u=P[4]), INVALID),                 # one of the two alone
    (dict(K=36), SHAPE), (dict(wg=ODD), ALIGN), (dict(g=P[4], u=ODD), ALIGN)])
def test_gated_refuses(kw, status):
    assert gated(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(M=0), INVALID), (dict(act=9), INVALID), (dict(dh=None), INVALID), (dict(g=None), INVALID),
    (dict(dwg=None), INVALID), (dict(dwu=None), INVALID), (dict(dx=None, dwg=None, dwu=None), INVALID),
    (dict(ws=None), INVALID), (dict(K=12), SHAPE), (dict(dx=ODD), ALIGN),
    (dict(ws=ctypes.c_void_p(0x10010)), ALIGN), (dict(nbytes=100), qg.QG_ERR_SCRATCH_TOO_SMALL)])
def test_backward_refuses(kw, status):
    assert backward(**kw) == status


def test_valid_arguments_reach_the_device_probe():
    """Nothing else is wrong with the calls above: without a device they end at the probe."""
    if torch.cuda.is_available():
        pytest.skip("fake addresses are for machines without a device")
    for call in (quant, scaled, gated8, gated, backward, lambda: scaled(b=P[4]),
                 lambda: gated(g=P[4], u=P[5]), lambda: backward(dx=None),
                 lambda: backward(dwg=None, dwu=None)):
        assert call() in (qg.QG_ERR_CUDA, qg.QG_ERR_NOT_SM100)


def test_backward_workspace_bytes():
    size = qg.qgemm_dense_gated_backward_workspace_bytes
    assert size(0, 8, 8) == size(8, 0, 8) == size(8, 8, 0) == size(8, 8, 12) == 0
    for M, F, K in [(1, 1, 8), (77, 1371, 520), (8192, 11008, 4096), (100000, 28672, 8192)]:
        rows = M * ((F + 7) // 8 * 8) * 2                 # dG, and dU, rows of 16 bytes
        need = size(M, F, K)
        assert 2 * rows <= need <= 2 * (rows + 255) + (64 << 20)
        assert need % 256 == 0


# ---- the binding's own checks (CPU tensors never reach the library) ----------------------------

def test_binding_refuses_cpu_tensors():
    x = torch.zeros(4, 64, dtype=torch.float16)
    q = torch.zeros(4, 64, dtype=torch.int8)
    s = torch.ones(4)
    for call in (lambda: qg.quant_int8_tokens(x), lambda: qg.qgemm_w8a8_scaled(q, q, s, s),
                 lambda: qg.qgemm_w8a8_gated(q, q, q, s, s, s), lambda: qg.qgemm_dense_gated(x, x, x),
                 lambda: qg.qgemm_dense_gated_backward(x, x, x, x, x, x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_binding_refuses_types_and_names():
    x32 = torch.zeros(4, 64)
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        qg.quant_int8_tokens(x32)
    with pytest.raises(TypeError):
        qg.qgemm_dense_gated(x32, x32, x32)
    with pytest.raises(ValueError, match="act"):
        qg.qgemm_dense_gated(x, x, x, act="relu")
    with pytest.raises(ValueError, match="act"):
        qg.qgemm_dense_gated_backward(x, x, x, x, x, x, act="swish")


@pytest.mark.parametrize("shape", [(2 ** 31, 8), (2 ** 32 + 5, 8), (1, 2 ** 32 + 16)])
def test_binding_refuses_sizes_beyond_an_int(shape):
    """Four billion rows would arrive in C as a handful."""
    class Huge:
        dtype = torch.float16
        is_cuda = True

        def __init__(self):
            self.shape = shape

        def dim(self):
            return 2

        def is_contiguous(self):
            return True

    with pytest.raises(ValueError, match="rows or columns"):
        qg.quant_int8_tokens(Huge())
