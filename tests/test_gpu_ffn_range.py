"""Gradients whose elementwise half leaves the range of fp16 although they themselves do not: dG = dH U
act'(G) and dU = dH act(G) go to the tensor cores in 16 bits, scaled by one power of two so that the
largest of them (for gelu a bound at most 1.3 times the value of a positive gate) lies between 2^14 and
2^15.

Bound of one rounded value: half a step of its type relative to it, or, where it is so much smaller than
the largest that it becomes a subnormal number after scaling, half of 2^-24 at that scale: at most
2^-25 / 2^14 of the largest. Everything else is counted as in ffn_ref.py."""
import pytest
import torch

import ffn_ref as R
import gemv_w4a16_w8a8_b200 as qg
from test_gpu_ffn import ACTS, DEV, guarded, normal, rng

pytestmark = pytest.mark.gpu
TYPES = [torch.float16, torch.bfloat16]
# dX by the few-token kernel with weights on either side of the MMA, one launch, two launches, in
# parts; F odd, even and a multiple of eight
SHAPES = [(5, 97, 64), (64, 1030, 256), (77, 1371, 520), (65, 640, 1312), (265, 16, 8), (300, 2002, 104),
          (512, 11008, 512), (2049, 520, 136)]


def halves(dH, G, U, act):
    dh, g, u = dH.double(), G.double(), U.double()
    return dh * u * R.slope(g, act), dh * R.value(g, act)


def largest(dH, G, U, act):
    """What the power of two is chosen by: the largest finite |dG| or |dU|; for gelu, of their bounds
    with s = 17/16 / (1 + exp(-1.702 g)) >= Phi(g): |act| <= |g| s, |act'| <= min(1.13, (1 + |g|) s)."""
    if act == "gelu":
        dh, g, u = dH.double(), G.double(), U.double()
        s = 17 / 16 * torch.sigmoid(1.702 * g)
        both = dh * u * ((1 + g.abs()) * s).clamp(max=1.13), dh * g * s
    else:
        both = halves(dH, G, U, act)
    return max(float(t[torch.isfinite(t)].abs().max()) for t in both)


def reference(dH, X, Wg, Wu, G, U, act, rows=slice(None)):
    """ffn_ref.backward with the bound of rounding dG and dU at a common scale; of some tokens."""
    dt, F = X.dtype, Wg.shape[0]
    tiny = 2.0 ** -39 * largest(dH, G, U, act) if dt == torch.float16 else 2.0 ** -134
    dH, X, G, U = (t[rows] for t in (dH, X, G, U))
    M = X.shape[0]
    dh, x, wg, wu, g, u = (t.double() for t in (dH, X, Wg, Wu, G, U))
    s = R.slope(g, act)
    dg, du = halves(dH, G, U, act)
    eg = (dh * u).abs() * (2.0 ** -18 * s.abs() + 2.0 ** -22) + 2.0 ** -22 * dg.abs()
    eu = 2.0 ** -17 * du.abs()
    edg, edu = (e + R.half_step(dt) * (d.abs() + e) + tiny for d, e in ((dg, eg), (du, eu)))

    def product(a, ea, b, n):
        return a @ b, ea @ b.abs() + R.sum_slack(n) * ((a.abs() + ea) @ b.abs())

    (p, ep), (q, eq) = product(dg, edg, wg, 2 * F), product(du, edu, wu, 2 * F)
    out = {"dX": (p + q, R.rounded(p + q, ep + eq, dt))}
    for name, d, e in (("dWg", dg, edg), ("dWu", du, edu)):
        r, er = product(d.T, e.T, x, M)
        out[name] = (r, R.rounded(r, er, dt))
    return out


def case(M, F, K, dtype, dh, u, w, x):
    g = rng(M + F + K)
    return dict(dH=normal((M, F), dh, dtype, g), X=normal((M, K), x, dtype, g),
                Wg=normal((F, K), w, dtype, g), Wu=normal((F, K), w, dtype, g),
                G=normal((M, F), 1.5, dtype, g), U=normal((M, F), u, dtype, g))


def run(c, act):
    M, K = c["X"].shape
    F = c["Wg"].shape[0]
    dtype = c["X"].dtype
    outs = {"dX": guarded((M, K), dtype), "dWg": guarded((F, K), dtype), "dWu": guarded((F, K), dtype)}
    n = qg.qgemm_dense_gated_backward_workspace_bytes(M, F, K)
    ws = torch.full((n + 4096,), 0xFF, dtype=torch.uint8, device=DEV)
    qg.qgemm_dense_gated_backward(**c, act=act, workspace=ws[:n], **{k: v for k, (v, _) in outs.items()})
    qg.qgemm_sync_check()
    assert bool((ws[n:] == 0xFF).all()), "wrote past the workspace"
    for _, guard in outs.values():
        guard()
    return {k: v for k, (v, _) in outs.items()}


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,F,K", SHAPES)
@pytest.mark.parametrize("dh,u,w,x", [
    (400.0, 400.0, 2.0 ** -14, 2.0 ** -14),        # dG around 1e5: beyond 65504 in fp16
    (2.0 ** -13, 2.0 ** -9, 16.0, 64.0)])          # around 2^-22: below fp16's normal numbers
def test_out_of_range(M, F, K, dtype, dh, u, w, x):
    act = ACTS[(M + F) % 3]
    c = case(M, F, K, dtype, dh, u, w, x)
    got, ref = run(c, act), reference(**c, act=act)
    for k, v in got.items():
        R.check(v, ref[k], k)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,F,K", [(3, 20, 16), (200, 333, 72)])
def test_powers_of_two_pass_through(M, F, K, act):
    """dH larger by a power of two: the same bits, larger by it (nothing here becomes subnormal)."""
    c = case(M, F, K, torch.float16, 1.0, 1.0, 0.05, 0.5)
    c["dH"] = (c["dH"].clamp(-3, 3) * 64).round() / 64          # exact at every one of the scales
    base = run(c, act)
    for k in (-4, 3, 7):
        got = run(dict(c, dH=c["dH"] * 2.0 ** k), act)
        for name, v in got.items():
            want = (base[name].double() * 2.0 ** k)
            far = (want.abs() >= 2.0 ** -13) & (base[name].abs() >= 2.0 ** -13)      # normal at either scale
            assert torch.equal(v.double()[far], want[far]), (name, k)


@pytest.mark.parametrize("F", [24, 26, 27])
def test_non_finite_stay_in_their_row_and_column(F):
    """The scale goes by the finite values: a token of infinities leaves the others as they are."""
    M, K = 70, 40
    c = case(M, F, K, torch.float16, 0.25, 1.0, 0.2, 1.0)
    clean = run(c, "silu")
    c["dH"][33] = float("inf")
    c["U"][12, 5] = float("nan")
    got = run(c, "silu")
    assert not bool(torch.isfinite(got["dX"][33]).any()) and bool(got["dX"][12].isnan().all())
    rows = [m for m in range(M) if m not in (12, 33)]
    ref = reference(**c, act="silu", rows=rows)
    R.check(got["dX"][rows], ref["dX"], "dX")
    assert torch.equal(got["dX"][rows].isfinite(), clean["dX"][rows].isfinite())


def test_all_zero():
    c = case(70, 33, 16, torch.float16, 0.0, 1.0, 1.0, 1.0)
    assert all(bool((v == 0).all()) for v in run(c, "gelu").values())


@pytest.mark.parametrize("act", ACTS)
def test_every_gate_alone(act):
    """Each gate by itself decides the power of two: largest dH and U, so that too small a bound of the
    activations (gelu's first pass takes one) overflows, and weights that bring the gradients back."""
    K = 8
    dH = torch.full((1, 1), 60000.0, dtype=torch.float16, device=DEV)
    X = torch.full((1, K), 2.0 ** -20, dtype=torch.float16, device=DEV)
    W = torch.full((1, K), 2.0 ** -20, dtype=torch.float16, device=DEV)
    for g in torch.cat([torch.linspace(-6, 6, 193), torch.tensor([-10.0, 10.0, 30.0, 100.0])]).tolist():
        for u in (60000.0, 0.5):
            c = dict(dH=dH, X=X, Wg=W, Wu=W, G=torch.full_like(dH, g), U=torch.full_like(dH, u))
            got = run(c, act)
            for k, (ref, bound) in reference(**c, act=act).items():
                R.check(got[k], (ref, bound), (g, u, k))
