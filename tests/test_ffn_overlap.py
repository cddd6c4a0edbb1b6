"""Outputs that share memory with an input, with one another or with the workspace, without a GPU: the
kernels read their operands while they write, so such a call would give what the order of its CTAs
happens to leave. It is refused."""
import ctypes

import pytest

import gemv_w4a16_w8a8_b200 as qg

M, F, K = 4, 64, 64
BASE, STEP = 0x1000000, 0x100000                   # addresses that are never dereferenced
QUANT = ("X", "Q", "scales")
SCALED = ("A", "W", "sa", "sw", "bias", "C")
GATED8 = ("A", "Wg", "Wu", "sa", "sg", "su", "H")
GATED = ("X", "Wg", "Wu", "H", "G", "U")
BACKWARD = ("dH", "X", "Wg", "Wu", "G", "U", "dX", "dWg", "dWu", "ws")


def run(names, **at):
    p = {n: BASE + i * STEP for i, n in enumerate(names)}
    p.update({n: p[v] if isinstance(v, str) else p[v[0]] + v[1] for n, v in at.items()})
    a = [ctypes.c_void_p(p[n]) for n in names]
    L = qg.lib()
    if names is QUANT:
        return L.quant_int8_tokens(*a, M, K, 0, None)
    if names is SCALED:
        return L.qgemm_w8a8_scaled(*a, M, F, K, 0, None)
    if names is GATED8:
        return L.qgemm_w8a8_gated(*a, M, F, K, 0, 0, None)
    if names is GATED:
        return L.qgemm_dense_gated(*a, M, F, K, 0, 0, None)
    size = qg.qgemm_dense_gated_backward_workspace_bytes(M, F, K)
    return L.qgemm_dense_gated_backward(*a[:9], M, F, K, 0, 0, a[9], size, None)


@pytest.mark.parametrize("names,outputs", [(QUANT, ("Q", "scales")), (SCALED, ("C",)), (GATED8, ("H",)),
                                           (GATED, ("H", "G", "U")), (BACKWARD, ("dX", "dWg", "dWu", "ws"))])
def test_outputs_apart_from_everything(names, outputs):
    for out in outputs:
        for other in names:
            if other != out:
                assert run(names, **{out: other}) == qg.QG_ERR_INVALID_ARG, (out, other)


@pytest.mark.parametrize("names,at", [
    (QUANT, dict(Q=("X", 2 * M * K - 16))), (QUANT, dict(scales=("Q", M * K - 4))),
    (QUANT, dict(X=("scales", 0))), (SCALED, dict(C=("A", M * K - 16))), (SCALED, dict(bias=("C", 2 * M * F - 2))),
    (SCALED, dict(sa=("C", 16))), (GATED8, dict(H=("Wu", F * K - 16))), (GATED8, dict(su=("H", 2 * M * F - 4))),
    (GATED, dict(G=("H", 2 * M * F - 16))), (GATED, dict(U=("Wg", 16))), (BACKWARD, dict(dX=("dH", 2 * M * F - 16))),
    (BACKWARD, dict(dWu=("dWg", 2 * F * K - 16))), (BACKWARD, dict(ws=("dWu", 2 * F * K - 256)))])
def test_a_part_of_them(names, at):
    assert run(names, **at) == qg.QG_ERR_INVALID_ARG


@pytest.mark.parametrize("names,at", [
    (QUANT, dict(Q=("X", 2 * M * K))), (SCALED, dict(W="A")), (SCALED, dict(sw="sa")), (SCALED, dict(C=("A", M * K))),
    (GATED8, dict(Wu="Wg", su="sg")), (GATED, dict(Wu="Wg")), (GATED, dict(G=("H", 2 * M * F))),
    (BACKWARD, dict(Wu="Wg", U="G", X="dH")), (BACKWARD, dict(dWu=("dWg", 2 * F * K)))])
def test_neighbours_and_shared_inputs_are_taken(names, at):
    import torch
    if torch.cuda.is_available():
        pytest.skip("fake addresses are for machines without a device")
    assert run(names, **at) in (qg.QG_ERR_CUDA, qg.QG_ERR_NOT_SM100)


def test_the_workspace_counts_as_far_as_it_is_used():
    """A large buffer that begins with the workspace's bytes and goes on with other things."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("fake addresses are for machines without a device")
    size = qg.qgemm_dense_gated_backward_workspace_bytes(M, F, K)
    a = [ctypes.c_void_p(BASE + i * STEP) for i in range(9)]
    ws = ctypes.c_void_p(BASE - size)
    call = qg.lib().qgemm_dense_gated_backward
    assert call(*a, M, F, K, 0, 0, ws, 1 << 40, None) in (qg.QG_ERR_CUDA, qg.QG_ERR_NOT_SM100)
