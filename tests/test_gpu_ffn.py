"""Token quantisation, the scaled W8A8 matmul and the gated feed-forward block on the GPU against
plain 64-bit forms (bounds in ffn_ref.py), over sizes where tiles, splits and alignments end."""
import numpy as np
import pytest
import torch

import ffn_ref as R
import gemv_w4a16_w8a8_b200 as qg

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.float16, torch.bfloat16]
ACTS = ["silu", "gelu", "gelu_tanh"]


def rng(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(shape, spread, dtype, g):
    return (torch.randn(shape, generator=g, device=DEV) * spread).to(dtype)


def codes(rows, cols, g):
    """int8 over the whole range, -128 included."""
    return torch.randint(-128, 128, (rows, cols), generator=g, device=DEV, dtype=torch.int8)


def guarded(shape, dtype):
    """(view, check): rows past the view keep their pattern. The view's storage starts 16-byte aligned."""
    rows, cols = shape
    n = rows * cols
    buf = torch.full((n + 4096,), 7.0, device=DEV).to(dtype)

    def check():
        assert bool((buf[n:] == torch.tensor(7.0, device=DEV).to(dtype)).all()), "wrote past the output"
    return buf[:n].view(rows, cols), check


# ---- quantisation -------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K", [(1, 8), (1, 4096), (3, 24), (5, 264), (7, 2048), (2, 2056), (33, 11008),
                                 (130, 520), (2, 16384), (3, 40008), (1, 131072), (4097, 64)])
def test_quant(M, K, dtype):
    x = normal((M, K), 1.0, dtype, rng(M + K))
    Q, guard = guarded((M, K), torch.int8)
    q, s = qg.quant_int8_tokens(x, Q=Q)
    guard()
    rq, rs = R.quant(x.float().cpu().numpy())
    assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(s.cpu().numpy(), rs)
    # and by what the codes mean: within half a step, and some roundings, of x
    back = q.double() * s.double()[:, None]
    assert bool(((back - x.double()).abs() <= s.double()[:, None] * (0.5 + 127 * 3 * 2.0 ** -24)).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_quant_special_rows(dtype):
    K = 1032
    x = normal((12, K), 1.0, dtype, rng(5))
    x[1] = 0
    x[2] = 0
    x[2, K - 1] = -3.0                       # all but the last
    x[3, 700] = float("inf")
    x[4, 0] = float("nan")
    x[5, K - 1] = float("-inf")
    x[6] = torch.finfo(dtype).max
    x[7] = torch.finfo(dtype).tiny * torch.arange(K, device=DEV).remainder(5).to(dtype)
    x[8] = 0
    x[8, ::3] = 6e-8 if dtype == torch.float16 else 9.2e-41     # the smallest subnormal
    x[9] = 2.0 ** -14 if dtype == torch.float16 else 2.0 ** -61
    x[10] = -torch.arange(K, device=DEV).remainder(128).to(dtype)   # ties and exact codes
    x[10, 3] = 127
    q, s = qg.quant_int8_tokens(x)
    rq, rs = R.quant(x.float().cpu().numpy())
    assert np.array_equal(q.cpu().numpy(), rq)
    assert np.array_equal(s.cpu().numpy(), rs, equal_nan=True)
    assert bool(torch.isnan(s[3:6]).all()) and s[1] == 1


# ---- scaled W8A8 ----------------------------------------------------------------------------------

SCALED_SHAPES = [(1, 1, 16), (1, 256, 4096), (2, 129, 48), (4, 4096, 512), (5, 1000, 1040), (8, 333, 2064),
                 (16, 512, 11008), (17, 130, 64), (31, 777, 4112), (33, 4100, 256), (64, 128, 8192), (77, 1371, 528),
                 (128, 257, 128), (129, 1024, 4096), (255, 640, 272), (300, 2001, 1024), (513, 776, 2064),
                 (1000, 3000, 400), (2049, 1288, 512), (64, 4096, 1024), (65, 4097, 1024), (96, 100, 2048),
                 (3, 100001, 64), (20, 32000, 144), (200, 70, 16384), (700, 200, 4096), (5000, 33, 48)]


def scaled_case(M, N, K, dtype, bias, seed=0):
    g = rng(seed + M + 7 * N + 13 * K)
    A, W = codes(M, K, g), codes(N, K, g)
    sa = torch.rand(M, generator=g, device=DEV) * 0.02 + 1e-4
    sw = (torch.rand(N, generator=g, device=DEV) - 0.5) * 0.02
    b = normal((N,), 1.0, dtype, g) if bias else None
    return A, W, sa, sw, b


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", SCALED_SHAPES)
def test_scaled(M, N, K, dtype):
    bias = (M + N + K // 16) % 2 == 1
    A, W, sa, sw, b = scaled_case(M, N, K, dtype, bias)
    C, guard = guarded((M, N), dtype)
    qg.qgemm_w8a8_scaled(A, W, sa, sw, bias=b, C=C)
    qg.qgemm_sync_check()
    guard()
    R.check(C, R.scaled(A, W, sa, sw, b, dtype))
    # the definition's own binary32 steps give the same bits
    acc = (A.double() @ W.double().T).to(torch.int32).float()
    step = acc * sa[:, None] * sw
    step = step if b is None else step + b.float()
    assert torch.equal(C, step.to(dtype))


def test_scaled_extremes():
    """The largest sums of the largest K, scales that overflow, are zero, infinite and NaN."""
    K = 131056
    A = torch.full((4, K), -128, dtype=torch.int8, device=DEV)
    W = torch.full((40, K), -128, dtype=torch.int8, device=DEV)
    W[20:] = 127
    sa = torch.tensor([2.0 ** -20, 1.0, 0.0, float("nan")], device=DEV)
    sw = torch.full((40,), 2.0 ** -12, device=DEV)
    sw[7] = float("inf")
    C = qg.qgemm_w8a8_scaled(A, W, sa, sw)
    acc = (A.double() @ W.double().T).to(torch.int32).float()
    assert torch.equal(C.isnan(), (acc * sa[:, None] * sw).half().isnan())
    assert torch.equal(C.nan_to_num(1.0), (acc * sa[:, None] * sw).half().nan_to_num(1.0))


def test_scaled_output_past_2_31_elements():
    M, N, K = 140000, 16000, 16
    A, W, sa, sw, _ = scaled_case(M, N, K, torch.float16, False)
    C = qg.qgemm_w8a8_scaled(A, W, sa, sw)
    for m in (0, 67107, 134217, 134218, 139999):          # both sides of element 2^31
        R.check(C[m:m + 1], R.scaled(A[m:m + 1], W, sa[m:m + 1], sw, None, torch.float16), m)


# ---- gated, 8 bits ----------------------------------------------------------------------------------

GATED_SHAPES = [(1, 1, 16), (1, 1376, 4096), (2, 65, 48), (4, 4096, 512), (7, 1000, 1040), (15, 333, 2064), (16, 512, 4096),
                (17, 130, 64), (33, 777, 4112), (64, 128, 8192), (77, 1371, 528), (128, 257, 128), (129, 1024, 1024),
                (255, 640, 272), (300, 2001, 1024), (513, 776, 2064), (2049, 1288, 512)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,F,K", GATED_SHAPES)
def test_gated8(M, F, K, dtype):
    act = ACTS[(M + F) % 3]
    g = rng(M + 3 * F + K)
    A, Wg, Wu = codes(M, K, g), codes(F, K, g), codes(F, K, g)
    s = 1.5 / (74.0 * 74.0 * K ** 0.5)                     # codes have a deviation of 74
    sa = torch.rand(M, generator=g, device=DEV) + 0.5
    sg, su = ((torch.rand(F, generator=g, device=DEV) + 0.5) * s for _ in range(2))
    H, guard = guarded((M, F), dtype)
    qg.qgemm_w8a8_gated(A, Wg, Wu, sa, sg, su, H=H, act=act)
    qg.qgemm_sync_check()
    guard()
    R.check(H, R.gated8(A, Wg, Wu, sa, sg, su, act, dtype))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", TYPES)
def test_gated8_every_activation(act, dtype):
    g = rng(3)
    M, F, K = 40, 200, 256
    A, Wg, Wu = codes(M, K, g), codes(F, K, g), codes(F, K, g)
    sa = torch.ones(M, device=DEV)
    sg = torch.full((F,), 3.0 / (74.0 * 74.0 * 16), device=DEV)
    R.check(qg.qgemm_w8a8_gated(A, Wg, Wu, sa, sg, sg, act=act, out_dtype=dtype),
            R.gated8(A, Wg, Wu, sa, sg, sg, act, dtype))


# ---- gated, 16 bits -----------------------------------------------------------------------------------

DENSE_SHAPES = [(1, 1, 8), (1, 1376, 4096), (2, 65, 24), (3, 4096, 512), (4, 100, 4096), (7, 1000, 1032), (15, 333, 2056),
                (16, 512, 4096), (17, 130, 72), (33, 777, 4104), (64, 128, 8192), (77, 1371, 520), (128, 257, 136),
                (129, 1024, 1024), (255, 640, 264), (300, 2001, 1000), (513, 776, 2056), (2049, 1288, 512)]


@pytest.mark.parametrize("save", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,F,K", DENSE_SHAPES)
def test_gated(M, F, K, dtype, save):
    act = ACTS[(M + F + save) % 3]
    g = rng(M + 3 * F + K)
    X = normal((M, K), 1.0, dtype, g)
    Wg, Wu = (normal((F, K), 1.5 / K ** 0.5, dtype, g) for _ in range(2))
    outs = {n: guarded((M, F), dtype) for n in ("H", "G", "U")}
    kw = {n: v for n, (v, _) in outs.items() if save or n == "H"}
    qg.qgemm_dense_gated(X, Wg, Wu, act=act, **kw)
    qg.qgemm_sync_check()
    ref = R.gated(X, Wg, Wu, act)
    for n, v in kw.items():
        outs[n][1]()
        R.check(v, ref[n], n)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", TYPES)
def test_gated_pre_activations_far_out(act, dtype):
    """Gates from -60 to 60: both tails of every activation."""
    M, F, K = 24, 121, 16
    X = torch.zeros(M, K, device=DEV, dtype=dtype)
    X[:, 0] = torch.linspace(-6, 6, M, device=DEV).to(dtype)
    X[:, 1] = 1
    Wg, Wu = torch.zeros(2, F, K, device=DEV, dtype=dtype)
    Wg[:, 0] = torch.linspace(0, 10, F, device=DEV).to(dtype)
    Wu[:, 1] = 1
    H, G, U = qg.qgemm_dense_gated(X, Wg, Wu, act=act, save_preact=True)
    g = X.double() @ Wg.double().T
    near = g.abs() <= 16
    ref, bound = R.gated(X, Wg, Wu, act)["H"]
    R.check(torch.where(near, H.double(), ref), (ref, bound))
    # beyond: |x| 2^-22 relative for the exponential's argument, and what is below 2^-120 may be 0
    far = (H.double() - ref).abs() <= R.rounded(ref, g.abs() * 2.0 ** -20 * ref.abs() + 2.0 ** -110, dtype)
    assert bool(far[~near].all())


def test_gated_non_finite_stay_in_their_row_and_column():
    M, F, K = 150, 300, 264
    g = rng(1)
    X = normal((M, K), 1.0, torch.bfloat16, g)
    Wg, Wu = (normal((F, K), 0.1, torch.bfloat16, g) for _ in range(2))
    clean = qg.qgemm_dense_gated(X, Wg, Wu)
    X[77, 5] = float("nan")
    Wu[123, 9] = float("inf")
    H = qg.qgemm_dense_gated(X, Wg, Wu)
    assert bool(H[77].isnan().all()) and not bool(torch.isfinite(H[:, 123]).any())
    H[77], H[:, 123] = clean[77], clean[:, 123]
    assert torch.equal(H, clean)


# ---- backward --------------------------------------------------------------------------------------------

BWD_SHAPES = [(1, 1, 8), (1, 256, 512), (2, 65, 24), (3, 100, 40), (16, 512, 1024), (33, 777, 136), (64, 64, 64),
              (77, 1371, 520), (128, 256, 256), (129, 1000, 264), (255, 130, 2056), (300, 2001, 104), (513, 776, 520),
              (1000, 65, 8), (2049, 520, 136), (40, 4103, 72), (4000, 100, 64), (700, 4098, 256), (64, 1030, 2048),
              (8, 9000, 512), (1500, 260, 1032)]


def backward_case(M, F, K, dtype, seed=0):
    g = rng(seed + M + 3 * F + K)
    return dict(dH=normal((M, F), 0.25, dtype, g), X=normal((M, K), 1.0, dtype, g),
                Wg=normal((F, K), 1 / K ** 0.5, dtype, g), Wu=normal((F, K), 1 / K ** 0.5, dtype, g),
                G=normal((M, F), 1.5, dtype, g), U=normal((M, F), 1.0, dtype, g))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,F,K", BWD_SHAPES)
def test_backward(M, F, K, dtype):
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


@pytest.mark.parametrize("act", ACTS)
def test_backward_parts_alone(act):
    """dX alone and the weights' gradients alone are those of the whole call."""
    c = backward_case(70, 200, 136, torch.bfloat16)
    dX, dWg, dWu = qg.qgemm_dense_gated_backward(**c, act=act)
    x, none_g, none_u = qg.qgemm_dense_gated_backward(**c, act=act, need_dw=False)
    assert torch.equal(x, dX) and none_g is None and none_u is None
    none_x, g, u = qg.qgemm_dense_gated_backward(**c, act=act, need_dx=False)
    assert none_x is None and torch.equal(g, dWg) and torch.equal(u, dWu)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", TYPES)
def test_every_gate_value(act, dtype):
    """The activation and its derivative at every 16-bit number up to 100 in size: with dH = U = X = 1
    the weights' gradients are act'(G) and act(G), rounded twice (the second time exactly). Bound:
    2^-18 relative, the exponential's argument (|x| <= 2 |g| (1 + g^2 / 20) where the result is above
    2^-110, so |x| <= 80) by 2^-23 each way, and for a derivative, whose terms may cancel, 2^-22 of
    the larger term."""
    g = torch.arange(-32768, 32768, device=DEV, dtype=torch.int32).to(torch.int16).view(dtype)
    g = g[torch.isfinite(g) & (g.abs() <= 100)]
    F = g.numel()
    g = g.view(1, F)
    one, zero = torch.ones(1, F, device=DEV, dtype=dtype), torch.zeros(F, 8, device=DEV, dtype=dtype)
    X = torch.ones(1, 8, device=DEV, dtype=dtype)
    _, dWg, dWu = qg.qgemm_dense_gated_backward(one, X, zero, zero, g, one, act=act, need_dx=False)
    x = g[0].double()
    arg = torch.where(x < 0, 80 * 2.0 ** -22, 2.0 ** -22)
    v, d = R.value(x, act), R.slope(x, act)
    tail = torch.sigmoid(2.6 * x) * (1 + x.abs()) ** 3       # of the size of the derivative's terms
    R.check(dWu[:, 0], (v, R.rounded(v, v.abs() * (2.0 ** -18 + arg) + 2.0 ** -110, dtype)), "value")
    R.check(dWg[:, 0], (d, R.rounded(d, (d.abs() + tail) * (2.0 ** -18 + arg) + 2.0 ** -110, dtype)), "slope")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", TYPES)
def test_backward_against_differences(act, dtype):
    """Directional differences of the 64-bit forward pass, G and U saved by the library's. The
    bound: the elementwise bounds of the gradients along the direction, what rounding G and U
    moves them (|act''| <= 1.2), and the difference's own t^2 term, estimated from a second t."""
    M, F, K = 20, 72, 40
    g = rng(11)
    X = normal((M, K), 1.0, dtype, g)
    Wg, Wu = (normal((F, K), 1 / K ** 0.5, dtype, g) for _ in range(2))
    dH = normal((M, F), 0.25, dtype, g)
    _, G, U = qg.qgemm_dense_gated(X, Wg, Wu, act=act, save_preact=True)
    grads = qg.qgemm_dense_gated_backward(dH, X, Wg, Wu, G, U, act=act)
    bounds = R.backward(dH, X, Wg, Wu, G, U, act)
    x, wg, wu, dh = (t.double() for t in (X, Wg, Wu, dH))

    def loss(x, wg, wu):
        return float((R.value(x @ wg.T, act) * (x @ wu.T) * dh).sum())

    g64, u64 = x @ wg.T, x @ wu.T
    u = R.half_step(dtype)
    eg = u * 1.01 * g64.abs() + R.sum_slack(K) * (x.abs() @ wg.abs().T)
    eu = u * 1.01 * u64.abs() + R.sum_slack(K) * (x.abs() @ wu.abs().T)
    edg = dh.abs() * (1.13 * eu + 1.2 * (u64.abs() + eu) * eg)      # moves of dG and dU
    edu = dh.abs() * 1.13 * eg
    moved = {"dX": edg @ wg.abs() + edu @ wu.abs(), "dWg": edg.T @ x.abs(), "dWu": edu.T @ x.abs()}
    for i, (name, got) in enumerate(zip(("dX", "dWg", "dWu"), grads)):
        v = torch.randn(got.shape, generator=g, device=DEV).double()
        args = [x, wg, wu]

        def slope(t):
            up, down = list(args), list(args)
            up[i], down[i] = args[i] + t * v, args[i] - t * v
            return (loss(*up) - loss(*down)) / (2 * t)

        d1, d2 = slope(1e-3), slope(2e-3)
        slack = float(((bounds[name][1] + moved[name]) * v.abs()).sum()) + 2 * abs(d1 - d2) + 1e-9
        assert abs(float((got.double() * v).sum()) - d1) <= slack, name


# ---- use: chains, streams, graphs, repetition ------------------------------------------------------------

@pytest.mark.parametrize("M", [1, 9, 200])
def test_8bit_block_in_a_row(M):
    """X -> codes -> gate and up -> codes -> down, each step against its plain form on what the
    step before it gave."""
    g = rng(M)
    K, F = 512, 1376
    X = normal((M, K), 1.0, torch.bfloat16, g)
    weights = []
    for rows, cols in ((F, K), (F, K), (K, F)):
        weights += list(qg.quant_int8_tokens(normal((rows, cols), cols ** -0.5, torch.bfloat16, g)))
    Wg, sg, Wu, su, Wd, sd = weights
    q, s = qg.quant_int8_tokens(X)
    H = qg.qgemm_w8a8_gated(q, Wg, Wu, s, sg, su, out_dtype=torch.bfloat16)
    q2, s2 = qg.quant_int8_tokens(H)
    Y = qg.qgemm_w8a8_scaled(q2, Wd, s2, sd, out_dtype=torch.bfloat16)
    R.check(H, R.gated8(q, Wg, Wu, s, sg, su, "silu", torch.bfloat16))
    rq, rs = R.quant(H.float().cpu().numpy())
    assert np.array_equal(q2.cpu().numpy(), rq) and np.array_equal(s2.cpu().numpy(), rs)
    R.check(Y, R.scaled(q2, Wd, s2, sd, None, torch.bfloat16))


def test_16bit_block_trains():
    """Forward through the down projection and back: the whole block's gradients."""
    g = rng(2)
    M, F, K = 48, 160, 64
    X = normal((M, K), 1.0, torch.float16, g)
    Wg, Wu, Wd = normal((F, K), K ** -0.5, torch.float16, g), normal((F, K), K ** -0.5, torch.float16, g), \
        normal((K, F), F ** -0.5, torch.float16, g)
    H, G, U = qg.qgemm_dense_gated(X, Wg, Wu, save_preact=True)
    Y = qg.qgemm_dense_f16(H, Wd)
    dY = normal((M, K), 0.25, torch.float16, g)
    dH = qg.qgemm_dense_f16(dY, Wd.T.contiguous())
    grads = dict(zip(("dX", "dWg", "dWu"), qg.qgemm_dense_gated_backward(dH, X, Wg, Wu, G, U)))
    ref = R.backward(dH, X, Wg, Wu, G, U, "silu")
    for k, v in grads.items():
        R.check(v, ref[k], k)
    assert bool(torch.isfinite(Y).all())


def every_call(seed, M=37, N=272, K=144):
    """(call, outputs) of every entry point on buffers of its own."""
    g = rng(seed)
    A, W, sa, sw, b = scaled_case(M, N, K, torch.float16, True, seed)
    Wu = codes(N, K, g)
    c = backward_case(M, N, K, torch.bfloat16, seed)
    out = dict(Q=torch.empty(M, K, dtype=torch.int8, device=DEV), s=torch.empty(M, device=DEV),
               C=torch.empty(M, N, dtype=torch.float16, device=DEV),
               H8=torch.empty(M, N, dtype=torch.bfloat16, device=DEV),
               **{n: torch.empty(M, N, dtype=torch.bfloat16, device=DEV) for n in ("H", "G", "U")},
               dX=torch.empty(M, K, dtype=torch.bfloat16, device=DEV),
               dWg=torch.empty(N, K, dtype=torch.bfloat16, device=DEV),
               dWu=torch.empty(N, K, dtype=torch.bfloat16, device=DEV))
    ws = torch.empty(qg.qgemm_dense_gated_backward_workspace_bytes(M, N, K), dtype=torch.uint8, device=DEV)

    def call(stream=None):
        qg.quant_int8_tokens(c["X"], Q=out["Q"], scales=out["s"], stream=stream)
        qg.qgemm_w8a8_scaled(A, W, sa, sw, bias=b, C=out["C"], stream=stream)
        qg.qgemm_w8a8_gated(A, W, Wu, sa, sw, sw, H=out["H8"], stream=stream)
        qg.qgemm_dense_gated(c["X"], c["Wg"], c["Wu"], H=out["H"], G=out["G"], U=out["U"], stream=stream)
        qg.qgemm_dense_gated_backward(**c, dX=out["dX"], dWg=out["dWg"], dWu=out["dWu"], workspace=ws,
                                      stream=stream)
    return call, out


def clear(out):
    for v in out.values():
        v.zero_()


@pytest.mark.parametrize("M,N,K", [(1, 520, 1040), (12, 2000, 2048), (37, 272, 144), (300, 640, 528)])
def test_repeats_bit_for_bit(M, N, K):
    call, out = every_call(1, M, N, K)
    call()
    first = {k: v.clone() for k, v in out.items()}
    for _ in range(3):
        clear(out)
        call()
        assert all(torch.equal(v, first[k]) for k, v in out.items())


def test_other_streams_and_two_at_once():
    (c1, o1), (c2, o2) = every_call(1), every_call(2, M=50)
    c1()
    c2()
    torch.cuda.synchronize()
    want = [{k: v.clone() for k, v in o.items()} for o in (o1, o2)]
    clear(o1)
    clear(o2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        c1(s1)
        c2(s2.cuda_stream)                     # a raw handle
    torch.cuda.synchronize()
    for o, w in zip((o1, o2), want):
        assert all(torch.equal(v, w[k]) for k, v in o.items())
    torch.cuda.synchronize()
    clear(o1)
    torch.cuda.synchronize()
    c1(0)                                      # the legacy default stream, by its handle
    torch.cuda.synchronize()
    assert all(torch.equal(v, want[0][k]) for k, v in o1.items())
    # buffers that the call makes itself belong to the stream that it runs on
    x = torch.ones(4, 64, dtype=torch.float16, device=DEV)
    q, s = qg.quant_int8_tokens(x, stream=s1)
    s1.synchronize()
    assert bool((q == 127).all())


@pytest.mark.parametrize("M", [1, 37, 300])
def test_captured_and_replayed(M):
    call, out = every_call(3, M=M)
    call()
    torch.cuda.synchronize()
    want = {k: v.clone() for k, v in out.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(2):
        clear(out)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(v, want[k]) for k, v in out.items())


def test_binding_refuses_shapes_devices_and_strides():
    g = rng(0)
    A, W, sa, sw, b = scaled_case(4, 64, 64, torch.float16, True)
    for bad in (dict(W=W[:, :48].contiguous()), dict(sa=sa[:3].contiguous()), dict(sw=sw[:5].contiguous()),
                dict(b=b[:9].contiguous()), dict(A=A.T), dict(sa=sa.cpu()),
                dict(C=torch.empty(4, 63, dtype=torch.float16, device=DEV))):
        kw = {**dict(A=A, W=W, sa=sa, sw=sw, b=b, C=None), **bad}
        with pytest.raises(ValueError):
            qg.qgemm_w8a8_scaled(kw["A"], kw["W"], kw["sa"], kw["sw"], bias=kw["b"], C=kw["C"])
    with pytest.raises(TypeError):                       # a bias of another type than the result
        qg.qgemm_w8a8_scaled(A, W, sa, sw, bias=b, out_dtype=torch.bfloat16)
    X = normal((4, 64), 1.0, torch.float16, g)
    with pytest.raises(TypeError):
        qg.qgemm_dense_gated(X, X, X.bfloat16())
    with pytest.raises(ValueError):
        qg.qgemm_dense_gated(X, X, X, G=torch.empty(4, 4, dtype=torch.float16, device=DEV))
    with pytest.raises(ValueError):                      # rows with a stride
        qg.quant_int8_tokens(normal((4, 128), 1.0, torch.float16, g)[:, :64])
    with pytest.raises(qg.QGemmError) as e:
        qg.quant_int8_tokens(X[:, :60].contiguous())
    assert e.value.status == qg.QG_ERR_UNSUPPORTED_SHAPE
    c = backward_case(4, 64, 64, torch.float16)
    with pytest.raises(qg.QGemmError) as e:
        qg.qgemm_dense_gated_backward(**c, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    assert e.value.status == qg.QG_ERR_SCRATCH_TOO_SMALL
