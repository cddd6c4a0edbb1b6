"""Cases for the 8-bit and gated feed-forward operators of the library, with their plain forms.

Five operators of a gated feed-forward block (the sizes are those of the benchmark's LLaMA-style
shapes, K = 4096, F = 11008, 32000 output channels, and of its 16384 x 16384 matmul):

  quant   X [M,K] -> int8 codes [M,K] and one fp32 scale a token:
              amax = max |x|, s = amax / 127 (1 for a row of zeros), q = rint(x * (127 / amax))
          every step a binary32 operation, so that codes are compared as whole numbers
  scaled  C[m,n] = sa[m] * sw[n] * sum_k A[m,k] W[n,k] (+ bias[n])        A, W int8
  gated8  H[m,f] = act(sa[m] sg[f] sum A Wg) * (sa[m] su[f] sum A Wu)     A, Wg, Wu int8
  gated   G = X Wg^T, U = X Wu^T, H = act(G) * U                          16-bit; save: G and U too
  bwd     dG = dH * U * act'(G), dU = dH * act(G),
          dX = dG Wg + dU Wu, dWg = dG^T X, dWu = dU^T X                  G, U as the forward saved

run() computes them with elementary torch operations in 32 bits, rounded once at the end, or,
where `own` is set, calls the library.
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one token before a projection of a decode step: latency alone
        dict(name="quant_decode", op="quant", M=1, K=4096, dtype="fp16"),
        # a long prompt before the down projection
        dict(name="quant_prefill", op="quant", M=16384, K=11008, dtype="bf16"),
        # the down projection of one decoded token
        dict(name="scaled_decode", op="scaled", M=1, N=4096, K=11008, dtype="fp16", bias=False),
        # logits of a batch of 32 decoded tokens
        dict(name="scaled_logits32", op="scaled", M=32, N=32000, K=4096, dtype="bf16", bias=False),
        # a ragged prompt, odd numbers of tokens and of channels, with a bias
        dict(name="scaled_ragged", op="scaled", M=509, N=11007, K=4080, dtype="fp16", bias=True),
        # the benchmark's largest matmul
        dict(name="scaled_prefill", op="scaled", M=16384, N=16384, K=16384, dtype="fp16", bias=False),
        # gate and up projection of one decoded token, 8-bit
        dict(name="gated8_decode", op="gated8", M=1, F=11008, K=4096, dtype="fp16", act="silu"),
        # a prompt's chunk of 512 tokens, 8-bit
        dict(name="gated8_chunk", op="gated8", M=512, F=11008, K=4096, dtype="bf16", act="gelu_tanh"),
        # a decode batch of 16 in 16 bits
        dict(name="gated_batch16", op="gated", M=16, F=11008, K=4096, dtype="fp16", act="silu", save=False),
        # a training step's forward pass, keeping what the backward pass reads
        dict(name="gated_train", op="gated", M=8192, F=11008, K=4096, dtype="bf16", act="silu", save=True),
        # the backward pass of a short odd batch in a small model
        dict(name="bwd_ragged", op="bwd", M=77, F=1371, K=520, dtype="fp16", act="gelu"),
        # the training step's backward pass
        dict(name="bwd_train", op="bwd", M=8192, F=11008, K=4096, dtype="bf16", act="silu"),
    ]


def _size(rng, low, high, multiple=1):
    """A size between low and high, spread over the logarithm, odd ones among them."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return max(multiple, int(v) // multiple * multiple)


def draw(rng):
    op = rng.choice(["quant", "scaled", "gated8", "gated", "bwd"])
    dtype = rng.choice(["fp16", "bf16"])
    act = rng.choice(["silu", "gelu", "gelu_tanh"])
    if op == "quant":
        return dict(op=op, M=_size(rng, 1, 16384), K=_size(rng, 256, 11008, 8), dtype=dtype)
    if op == "scaled":
        return dict(op=op, M=_size(rng, 1, 16384), N=_size(rng, 256, 32000),
                    K=_size(rng, 256, 16384, 16), dtype=dtype, bias=rng.random() < 0.5)
    M, F = _size(rng, 1, 8192), _size(rng, 256, 11008)
    if op == "gated8":
        return dict(op=op, M=M, F=F, K=_size(rng, 256, 4096, 16), dtype=dtype, act=act)
    K = _size(rng, 256, 4096, 8)
    if op == "gated":
        return dict(op=op, M=M, F=F, K=K, dtype=dtype, act=act, save=rng.random() < 0.5)
    return dict(op=op, M=M, F=F, K=K, dtype=dtype, act=act)


# ---- inputs -----------------------------------------------------------------------------------

def _codes(g, rows, cols, spread):
    """int8 codes and scales as a symmetric quantisation of normal rows leaves them: the largest
    of a row near 127, a scale around `spread` / 127 * 4."""
    q = torch.randn(rows, cols, generator=g, device="cuda").mul_(127 / 4.2).round_().clamp_(-127, 127).to(torch.int8)
    s = (torch.rand(rows, generator=g, device="cuda") * 0.5 + 0.75) * (4.2 * spread / 127)
    return q, s


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, M, K, dt = case["op"], case["M"], case["K"], DTYPES[case["dtype"]]

    def normal(rows, cols, spread):
        return (torch.randn(rows, cols, generator=g, device="cuda") * spread).to(dt)

    if op == "quant":
        # activations with a few channels far larger than the rest, as normalised layers leave them
        x = torch.randn(M, K, generator=g, device="cuda")
        x[:, :: 97] *= 8
        return dict(X=x.to(dt))
    if op == "scaled":
        N = case["N"]
        A, sa = _codes(g, M, K, 1.0)
        W, sw = _codes(g, N, K, 1 / math.sqrt(K))
        b = torch.randn(N, generator=g, device="cuda").to(dt) if case["bias"] else None
        return dict(A=A, sa=sa, W=W, sw=sw, bias=b)
    F = case["F"]
    if op == "gated8":
        A, sa = _codes(g, M, K, 1.0)
        Wg, sg = _codes(g, F, K, 1 / math.sqrt(K))
        Wu, su = _codes(g, F, K, 1 / math.sqrt(K))
        return dict(A=A, sa=sa, Wg=Wg, sg=sg, Wu=Wu, su=su)
    X = normal(M, K, 1.0)
    Wg = normal(F, K, 1 / math.sqrt(K))
    Wu = normal(F, K, 1 / math.sqrt(K))
    if op == "gated":
        return dict(X=X, Wg=Wg, Wu=Wu)
    # pre-activations of X Wg^T's distribution, as the forward pass saved them
    return dict(X=X, Wg=Wg, Wu=Wu, G=normal(M, F, 1.0), U=normal(M, F, 1.0), dH=normal(M, F, 0.25))


def prepare(case, seed):
    """The inputs and the buffers that a program keeps from call to call."""
    state = dict(_inputs(case, seed), case=case)
    op, M, K, dt = case["op"], case["M"], case["K"], DTYPES[case["dtype"]]

    def empty(*shape, dtype=dt):
        return torch.empty(shape, dtype=dtype, device="cuda")

    if op == "quant":
        state.update(Q=empty(M, K, dtype=torch.int8), s=empty(M, dtype=torch.float32))
    elif op == "scaled":
        state.update(C=empty(M, case["N"]))
    elif op == "gated8":
        state.update(H=empty(M, case["F"]))
    elif op == "gated":
        state.update(H=empty(M, case["F"]))
        if case["save"]:
            state.update(G=empty(M, case["F"]), U=empty(M, case["F"]))
    else:
        F = case["F"]
        # dG and dU with rows padded to 16 bytes, and up to 64 MiB for sums that are split
        state.update(dX=empty(M, K), dWg=empty(F, K), dWu=empty(F, K),
                     workspace=empty(4 * M * (F + 8) + (64 << 20) + 1024, dtype=torch.uint8))
    return state


# ---- plain forms --------------------------------------------------------------------------------

def _act(g, kind):
    if kind == "silu":
        return g / (1 + torch.exp(-g))
    if kind == "gelu":
        return 0.5 * g * (1 + torch.erf(g * math.sqrt(0.5)))
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))


def _act_grad(g, kind):
    if kind == "silu":
        s = 1 / (1 + torch.exp(-g))
        return s * (1 + g * (1 - s))
    if kind == "gelu":
        return 0.5 * (1 + torch.erf(g * math.sqrt(0.5))) + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def _plain(s):
    case = s["case"]
    op, dt = case["op"], DTYPES[case["dtype"]]
    if op == "quant":
        x = s["X"].float()
        amax = x.abs().amax(1)
        most = torch.full_like(amax, 127.0)
        scale = torch.where(amax > 0, amax / most, torch.ones_like(amax))
        inv = torch.where(amax > 0, most / amax, torch.zeros_like(amax))
        return dict(codes=torch.round(x * inv[:, None]).to(torch.int8), scales=scale)
    if op == "scaled":
        c = (s["A"].float() @ s["W"].float().T) * s["sa"][:, None] * s["sw"]
        if s["bias"] is not None:
            c = c + s["bias"].float()
        return dict(C=c.to(dt))
    if op == "gated8":
        a = s["A"].float()
        g = (a @ s["Wg"].float().T) * s["sa"][:, None] * s["sg"]
        u = (a @ s["Wu"].float().T) * s["sa"][:, None] * s["su"]
        return dict(H=(_act(g, case["act"]) * u).to(dt))
    x, wg, wu = s["X"].float(), s["Wg"].float(), s["Wu"].float()
    if op == "gated":
        g, u = x @ wg.T, x @ wu.T
        h = (_act(g, case["act"]) * u).to(dt)
        return dict(H=h, G=g.to(dt), U=u.to(dt)) if case["save"] else dict(H=h)
    g, u, dh = s["G"].float(), s["U"].float(), s["dH"].float()
    dg, du = dh * u * _act_grad(g, case["act"]), dh * _act(g, case["act"])
    return dict(dX=(dg @ wg + du @ wu).to(dt), dWg=(dg.T @ x).to(dt), dWu=(du.T @ x).to(dt))


def _library(s):
    import gemv_w4a16_w8a8_b200 as qg
    case = s["case"]
    op = case["op"]
    if op == "quant":
        q, scale = qg.quant_int8_tokens(s["X"], Q=s["Q"], scales=s["s"])
        return dict(codes=q, scales=scale)
    if op == "scaled":
        return dict(C=qg.qgemm_w8a8_scaled(s["A"], s["W"], s["sa"], s["sw"], bias=s["bias"], C=s["C"]))
    if op == "gated8":
        return dict(H=qg.qgemm_w8a8_gated(s["A"], s["Wg"], s["Wu"], s["sa"], s["sg"], s["su"],
                                          H=s["H"], act=case["act"]))
    if op == "gated":
        if not case["save"]:
            return dict(H=qg.qgemm_dense_gated(s["X"], s["Wg"], s["Wu"], H=s["H"], act=case["act"]))
        h, g, u = qg.qgemm_dense_gated(s["X"], s["Wg"], s["Wu"], H=s["H"], G=s["G"], U=s["U"],
                                       act=case["act"])
        return dict(H=h, G=g, U=u)
    dx, dwg, dwu = qg.qgemm_dense_gated_backward(
        s["dH"], s["X"], s["Wg"], s["Wu"], s["G"], s["U"], act=case["act"], dX=s["dX"],
        dWg=s["dWg"], dWu=s["dWu"], workspace=s["workspace"])
    return dict(dX=dx, dWg=dwg, dWu=dwu)


def run(state):
    if own:
        return _library(state)
    return _plain(state)


# ---- what a pass cannot do without --------------------------------------------------------------

def work(case):
    op, M, K = case["op"], case["M"], case["K"]
    if op == "quant":
        return dict(bytes=2 * M * K + M * K + 4 * M, flops=3 * M * K)
    if op == "scaled":
        N = case["N"]
        return dict(bytes=M * K + N * K + 2 * M * N + 4 * (M + N) + (2 * N if case["bias"] else 0),
                    flops=2 * M * N * K)
    F = case["F"]
    if op == "gated8":
        return dict(bytes=M * K + 2 * F * K + 2 * M * F + 4 * (M + 2 * F), flops=4 * M * F * K)
    if op == "gated":
        return dict(bytes=2 * (M * K + 2 * F * K + M * F * (3 if case["save"] else 1)),
                    flops=4 * M * F * K)
    return dict(bytes=2 * (3 * M * F + 2 * M * K + 4 * F * K), flops=8 * M * F * K)


# ---- from the definition, in 64 bits -------------------------------------------------------------

def exact(case, seed):
    """float64 from the formulas at the top, through the logistic function and the normal
    distribution's; the codes of quant are whole numbers and have no value of their own here."""
    t = {k: (v.double() if v is not None else None) for k, v in _inputs(case, seed).items()}
    op = case["op"]
    if op == "quant":
        top = torch.linalg.vector_norm(t["X"], ord=math.inf, dim=1)
        return dict(codes=None, scales=torch.where(top == 0, 1.0, top / 127))
    if op == "scaled":
        c = torch.einsum("mk,nk->mn", t["A"], t["W"]).mul_(torch.outer(t["sa"], t["sw"]))
        return dict(C=c if t["bias"] is None else c.add_(t["bias"]))

    root = math.sqrt(2 / math.pi)

    def value(z):
        if case["act"] == "silu":
            return z * torch.special.expit(z)
        if case["act"] == "gelu":
            return z * torch.special.ndtr(z)
        return z * torch.special.expit(2 * root * z * (1 + 0.044715 * z.square()))

    def slope(z):
        if case["act"] == "silu":
            p = torch.special.expit(z)
            return p + z * p * torch.special.expit(-z)
        if case["act"] == "gelu":
            return torch.special.ndtr(z) + z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi)
        w = 2 * root * z * (1 + 0.044715 * z.square())
        p = torch.special.expit(w)
        return p + z * p * torch.special.expit(-w) * 2 * root * (1 + 3 * 0.044715 * z.square())

    if op == "gated8":
        gate = torch.einsum("mk,fk->mf", t["A"] * t["sa"][:, None], t["Wg"] * t["sg"][:, None])
        up = torch.einsum("mk,fk->mf", t["A"] * t["sa"][:, None], t["Wu"] * t["su"][:, None])
        return dict(H=value(gate) * up)
    if op == "gated":
        gate = torch.einsum("mk,fk->mf", t["X"], t["Wg"])
        up = torch.einsum("mk,fk->mf", t["X"], t["Wu"])
        h = value(gate) * up
        return dict(H=h, G=gate, U=up) if case["save"] else dict(H=h)
    down_g = slope(t["G"]) * t["U"] * t["dH"]
    down_u = value(t["G"]) * t["dH"]
    return dict(dX=torch.einsum("mf,fk->mk", down_g, t["Wg"]) + torch.einsum("mf,fk->mk", down_u, t["Wu"]),
                dWg=torch.einsum("mf,mk->fk", down_g, t["X"]),
                dWu=torch.einsum("mf,mk->fk", down_u, t["X"]))
