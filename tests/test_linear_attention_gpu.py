"""Linear attention on the GPU against its 64-bit definition.

Tolerances, before any run.  A bf16 result is one rounding (2^-8 of itself) of
fp32 sums whose terms pass through bf16 once, as an entry of the score matrix or
of the state operand: 2^-8 of the sum of the terms' absolute values, which the
reference computes as `bound`.  States, df and every fp32 result are fp32 sums
of fp32 terms: each of at most T + 256 additions, products and decays along a
path adds 2^-24 of the bound, the decay's logarithm and exponential 2^-21."""
import pytest
import torch

import la_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def api():
    from non_linear_matrix_persistent_b200 import api as a
    return a


def inputs(B, H, T, K, V, G=0, gate="value", start=True, dtype=torch.bfloat16, seed=0):
    g = torch.Generator().manual_seed(seed)
    G = G or H
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = dict(k=n(B, G, T, K) * K ** -0.5, v=n(B, H, T, V) * V ** -0.5, q=n(B, G, T, K) * K ** -0.5, dy=n(B, H, T, V))
    x = {i: t.to(dtype) for i, t in x.items()}
    if gate == "value":
        x["f"] = torch.sigmoid(n(B, H, T) + 2)
    elif gate == "edges":          # discards, keeps everything, underflows, and anything between
        x["f"] = torch.rand(B, H, T, generator=g)
        pick = torch.rand(B, H, T, generator=g)
        x["f"][pick < 0.10] = 0.0
        x["f"][(pick >= 0.10) & (pick < 0.30)] = 1.0
        x["f"][(pick >= 0.30) & (pick < 0.34)] = 1e-30
        x["f"][(pick >= 0.34) & (pick < 0.38)] = 1e-6
    elif gate == "slow":           # 1 - f of about 1e-5: decays that only show over thousands of tokens
        x["f"] = 1.0 - 1e-5 * torch.rand(B, H, T, generator=g)
    elif gate == "logit":
        x["f"] = 3 * n(B, H, T) + 2
    elif gate == "logit_edges":
        x["f"] = 3 * n(B, H, T)
        pick = torch.rand(B, H, T, generator=g)
        x["f"][pick < 0.1] = -200.0
        x["f"][(pick >= 0.1) & (pick < 0.2)] = 200.0
        x["f"][(pick >= 0.2) & (pick < 0.25)] = -30.0
    else:                          # one constant per head
        x["f"] = torch.rand(H, generator=g)
    x["S0"] = n(B, H, K, V) if start else None
    x["dST"] = n(B, H, K, V) if start else None
    return {i: None if t is None else t.to(DEV) for i, t in x.items()}, gate.startswith("logit")


def close(name, got, want, bound, T, dtype):
    assert tuple(got.shape) == tuple(want.shape), name
    assert torch.isfinite(got).all(), name
    slack = (T + 256) * 2.0 ** -24 + 2.0 ** -20
    tol = slack * bound + 1e-37
    if got.dtype == torch.bfloat16:
        assert dtype == torch.bfloat16
        tol = tol + 2.0 ** -8 * (want.abs() + 1.02 * bound)
    err = (got.double() - want).abs() - tol
    assert float(err.max()) <= 0 if err.numel() else True, (name, float(err.max()), int(err.argmax()))


def check(x, logit, bwd=True):
    a = api()
    T, dtype = x["v"].shape[2], x["v"].dtype
    y, ST, ckpt = a.linear_attention(x["k"], x["v"], x["q"], x["f"], x["S0"], want_ckpt=True, f_is_logit=logit)
    args = (x["k"], x["v"], x["q"], x["f"])
    wy, wS, states = ref.forward(*args, x["S0"], logit)
    by, bS, bstates = ref.forward(*args, x["S0"], logit, bound=True)
    close("y", y, wy, by, T, dtype)
    close("ST", ST, wS, bS, T, dtype)
    for c in range(ckpt.shape[2]):
        close("ckpt", ckpt[:, :, c].permute(0, 1, 3, 2, 4).reshape(states[0].shape), states[128 * c], bstates[128 * c], T, dtype)
    if not bwd:
        return y, ST
    got = a.linear_attention_backward(*args, ckpt, x["dy"], x["dST"], f_is_logit=logit)
    want = ref.backward(*args, x["dy"], x["S0"], x["dST"], logit)
    bound = ref.backward(*args, x["dy"], x["S0"], x["dST"], logit, bound=True)
    for n in want:
        close(n, got[n], want[n], bound[n], T * (x["v"].shape[0] if x["f"].dim() == 1 and n == "df" else 1), dtype)
    assert a.device_status() == 0
    return y, ST, got


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 256, 257, 385])
def test_lengths(T):
    check(*inputs(2, 3, T, 64, 64, seed=T))


@pytest.mark.parametrize("K", [16, 32, 64, 128])
@pytest.mark.parametrize("V", [16, 32, 64, 128])
def test_widths(K, V):
    check(*inputs(1, 3, 150, K, V, seed=K + V))


@pytest.mark.parametrize("K,V", [(64, 64), (128, 128), (32, 128)])
@pytest.mark.parametrize("gate", ["edges", "logit", "logit_edges", "head", "slow"])
@pytest.mark.parametrize("T", [1, 9, 290])
def test_gates(K, V, gate, T):
    check(*inputs(2, 2, T, K, V, gate=gate, seed=5))


@pytest.mark.parametrize("f", [1.0, 0.9, 0.2, 0.15, 0.14, 1e-3, 1e-20, 1e-33, 0.0])
@pytest.mark.parametrize("K,V", [(64, 64), (128, 128)])
def test_constant_gates(f, K, V):
    """Decays over a block of 32 tokens on both sides of 2^-90, where the diagonal blocks change their form, and
    gates beneath every floor."""
    x, _ = inputs(1, 2, 200, K, V, gate="head", seed=6)
    x["f"] = torch.full_like(x["f"], f)
    check(x, False)


@pytest.mark.parametrize("K,V", [(64, 128), (128, 64), (128, 128), (32, 64), (64, 64)])
@pytest.mark.parametrize("G", [1, 4])
def test_many_chunks(K, V, G):
    """Several chunks for every schedule, with shared k and q and odd ends, one CTA a pair."""
    check(*inputs(30, 4, 523, K, V, G=G, gate="logit", seed=8))


@pytest.mark.parametrize("K,V", [(64, 128), (128, 64), (128, 128), (64, 64)])
@pytest.mark.parametrize("gate", ["edges", "head"])
def test_segments(K, V, gate):
    """Two pairs over 12 chunks: a segment each, forward and backward."""
    check(*inputs(1, 2, 1500, K, V, G=1, gate=gate, seed=10))


@pytest.mark.parametrize("K,V", [(64, 128), (128, 64), (128, 128), (64, 64)])
def test_segments_of_several_chunks(K, V):
    """37 pairs over 17 chunks with gates close to 1: segments of 5, the last of 2."""
    check(*inputs(1, 37, 2100, K, V, gate="slow", seed=11))


@pytest.mark.parametrize("K,V", [(64, 128), (128, 128), (64, 64)])
def test_buffers_on_16_bytes(K, V):
    """Inputs and outputs that start on 16 bytes and not on 32."""
    a = api()
    x, _ = inputs(1, 2, 140, K, V, seed=12)

    def off(t):
        n = 8 if t.dtype == torch.bfloat16 else 4
        pad = torch.full((t.numel() + 2 * n,), 3.0, dtype=t.dtype, device=DEV)
        v = pad[n:n + t.numel()].view(t.shape)
        v.copy_(t)
        assert v.data_ptr() % 32 == 16
        return v

    args = [off(x[n]) for n in ("k", "v", "q", "f")]
    out = {"y": off(torch.zeros_like(x["v"])), "ST": off(torch.zeros_like(x["S0"]))}
    y, ST, ck = a.linear_attention(*args, off(x["S0"]), want_ckpt=True, out=out)
    y2, ST2, ck2 = a.linear_attention(x["k"], x["v"], x["q"], x["f"], x["S0"], want_ckpt=True)
    assert torch.equal(y, y2) and torch.equal(ST, ST2) and torch.equal(ck, ck2)
    out = {"dk": off(torch.zeros_like(x["k"])), "dv": off(torch.zeros_like(x["v"])), "dq": off(torch.zeros_like(x["q"])),
           "df": off(torch.zeros_like(x["f"])), "dS0": off(torch.zeros_like(x["S0"]))}
    g = a.linear_attention_backward(*args, off(ck), off(x["dy"]), off(x["dST"]), out=out)
    g2 = a.linear_attention_backward(x["k"], x["v"], x["q"], x["f"], ck2, x["dy"], x["dST"])
    assert all(torch.equal(g[n], g2[n]) for n in g2)


def test_a_nan_reaches_what_it_should():
    """A NaN in one pair's v: its later readouts and the states are NaN, other pairs and earlier chunks are not."""
    a = api()
    x, _ = inputs(1, 2, 300, 64, 64, start=False, seed=14)
    x["v"][0, 0, 140, 3] = float("nan")
    y, ST, ck = a.linear_attention(x["k"], x["v"], x["q"], x["f"], want_ckpt=True)
    assert bool(torch.isfinite(y[0, 1]).all()) and bool(torch.isfinite(ST[0, 1]).all())
    assert bool(torch.isfinite(y[0, 0, :128]).all()) and bool(torch.isnan(y[0, 0, 140:, 3]).all())
    assert bool(torch.isnan(ST[0, 0, :, 3]).all())
    g = a.linear_attention_backward(x["k"], x["v"], x["q"], x["f"], ck, x["dy"])
    assert all(bool(torch.isfinite(g[n][0, 1]).all()) for n in g)


def test_strided_inputs_are_refused():
    a = api()
    x, _ = inputs(1, 2, 40, 64, 64, seed=16)
    with pytest.raises(ValueError, match="contiguous"):
        a.linear_attention(x["k"].transpose(2, 3).contiguous().transpose(2, 3), x["v"], x["q"], x["f"])
    with pytest.raises(ValueError, match="shape"):
        a.linear_attention(x["k"], x["v"], x["q"], x["f"][:, :, :39].contiguous())
    with pytest.raises(TypeError):
        a.linear_attention(x["k"], x["v"], x["q"], x["f"].double())
    with pytest.raises(ValueError, match="ckpt"):
        a.linear_attention_backward(x["k"], x["v"], x["q"], x["f"], torch.zeros(1, 2, 1, 64, 64, device=DEV), x["dy"])
    with pytest.raises(RuntimeError, match="UNSUPPORTED"):
        a.linear_attention(x["k"][..., :48].contiguous(), x["v"], x["q"][..., :48].contiguous(), x["f"])


@pytest.mark.parametrize("H,G", [(4, 2), (6, 1), (8, 8)])
@pytest.mark.parametrize("T", [1, 37, 260])
@pytest.mark.parametrize("K,V", [(64, 64), (128, 64)])
def test_shared_k_and_q(H, G, T, K, V):
    check(*inputs(2, H, T, K, V, G=G, seed=7))


@pytest.mark.parametrize("T", [1, 20, 140])
@pytest.mark.parametrize("gate", ["edges", "logit", "head"])
@pytest.mark.parametrize("K,V,G", [(16, 32, 2), (128, 128, 1)])
def test_fp32(T, gate, K, V, G):
    check(*inputs(2, 2, T, K, V, G=G, gate=gate, dtype=torch.float32, seed=9))


@pytest.mark.parametrize("K,V", [(64, 64), (128, 128)])
def test_without_states(K, V):
    """No S0 and no dST: the forward starts from zeros, the backward from dST = 0."""
    check(*inputs(2, 2, 200, K, V, start=False, seed=11))


@pytest.mark.parametrize("B,H,T,K,V", [(1, 1, 3000, 64, 64), (1, 2, 2100, 128, 128), (1, 3, 1500, 32, 16), (40, 8, 130, 64, 64)])
def test_few_pairs_and_many(B, H, T, K, V):
    """One long sequence (split along T) and more pairs than the GPU has processors."""
    check(*inputs(B, H, T, K, V, gate="logit", seed=13))


@pytest.mark.parametrize("T", [1, 2, 5, 33, 64])
@pytest.mark.parametrize("K,V", [(16, 16), (64, 128), (128, 64), (128, 128), (64, 64)])
def test_short_results_are_rounded_once(T, K, V):
    """Up to 64 tokens no bf16 operand adds to the results' own rounding: half a step of bf16, 2^-9 of the value at
    its binade's top and 2^-8 at its bottom, plus 2^-15 of the sums of absolute values for the operands' second terms
    (2^-16 each, two of them in a product's path)."""
    a = api()
    x, logit = inputs(2, 3, T, K, V, G=1, gate="logit", seed=40 + T)
    args = (x["k"], x["v"], x["q"], x["f"])
    y, _, ck = a.linear_attention(*args, x["S0"], want_ckpt=True, f_is_logit=logit)
    got = a.linear_attention_backward(*args, ck, x["dy"], x["dST"], f_is_logit=logit)
    want = ref.backward(*args, x["dy"], x["S0"], x["dST"], logit)
    bound = ref.backward(*args, x["dy"], x["S0"], x["dST"], logit, bound=True)
    got["y"], want["y"] = y, ref.forward(*args, x["S0"], logit)[0]
    bound["y"] = ref.forward(*args, x["S0"], logit, bound=True)[0]
    for n in ("y", "dk", "dv", "dq"):
        err = (got[n].double() - want[n]).abs() - (2.0 ** -8 * want[n].abs() + 2.0 ** -15 * bound[n] + 1e-37)
        assert float(err.max()) <= 0, (n, float(err.max()))


def test_step_matches_scan_and_runs_in_place():
    a = api()
    x, logit = inputs(3, 4, 21, 64, 128, G=2, gate="logit", seed=15)
    wy, wS, _ = ref.forward(x["k"], x["v"], x["q"], x["f"], x["S0"], logit)
    by, bS, _ = ref.forward(x["k"], x["v"], x["q"], x["f"], x["S0"], logit, bound=True)
    S, keep = x["S0"].clone(), x["S0"].clone()
    for t in range(21):
        tok = [x[n][:, :, t].contiguous() for n in ("k", "v", "q", "f")]
        other = torch.full_like(S, float("nan"))
        y2 = a.linear_attention_step(*tok, S, ST=other, f_is_logit=logit)
        y = a.linear_attention_step(*tok, S, f_is_logit=logit)
        assert torch.equal(S, other) and torch.equal(y, y2)
        close("y", y, wy[:, :, t], by[:, :, t], 21, torch.bfloat16)
    close("ST", S, wS, bS, 21, torch.bfloat16)
    # the scan, with the state advanced in place too
    y, ST, _ = a.linear_attention(x["k"], x["v"], x["q"], x["f"], keep, f_is_logit=logit, out={"ST": keep})
    assert ST is keep
    close("ST", keep, wS, bS, 21, torch.bfloat16)
    close("y", y, wy, by, 21, torch.bfloat16)


def test_prompt_continues_from_a_state():
    """Two halves of a prompt, the second from the first's state, give the whole prompt's results."""
    a = api()
    x, _ = inputs(2, 3, 400, 64, 64, seed=17)
    cut = 171
    part = lambda i, j: [x[n][:, :, i:j].contiguous() for n in ("k", "v", "q", "f")]  # noqa: E731
    y1, S, _ = a.linear_attention(*part(0, cut), x["S0"])
    y2, S, _ = a.linear_attention(*part(cut, 400), S)
    wy, wS, _ = ref.forward(x["k"], x["v"], x["q"], x["f"], x["S0"])
    by, bS, _ = ref.forward(x["k"], x["v"], x["q"], x["f"], x["S0"], bound=True)
    close("y", torch.cat([y1, y2], 2), wy, by, 400, torch.bfloat16)
    close("ST", S, wS, bS, 400, torch.bfloat16)


def test_empty():
    a = api()
    x, _ = inputs(2, 3, 0, 64, 64, seed=19)
    y, ST, ckpt = a.linear_attention(x["k"], x["v"], x["q"], x["f"], x["S0"], want_ckpt=True)
    assert y.shape == (2, 3, 0, 64) and torch.equal(ST, x["S0"]) and ckpt.numel() == 0
    g = a.linear_attention_backward(x["k"], x["v"], x["q"], x["f"], ckpt, x["dy"], x["dST"])
    assert torch.equal(g["dS0"], x["dST"]) and g["dk"].numel() == 0
    _, ST, _ = a.linear_attention(x["k"], x["v"], x["q"], x["f"])
    assert float(ST.abs().max()) == 0
    g = a.linear_attention_backward(x["k"], x["v"], x["q"], torch.rand(3, device=DEV), ckpt, x["dy"])
    assert torch.equal(g["df"], torch.zeros(3, device=DEV)) and float(g["dS0"].abs().max()) == 0


def test_results_do_not_depend_on_other_pairs_and_repeat():
    """The same bits every time, nothing written outside the outputs, and gradients in place of dST."""
    a = api()
    x, logit = inputs(2, 3, 333, 64, 64, gate="logit", seed=21)
    args = (x["k"], x["v"], x["q"], x["f"])

    def once():
        pad = torch.full((2 * 3 * 333 * 64 + 4096,), 7.0, dtype=torch.bfloat16, device=DEV)
        n = 2 * 3 * 333 * 64
        y = pad[2048:2048 + n].view(2, 3, 333, 64)
        _, ST, ck = a.linear_attention(*args, x["S0"], want_ckpt=True, f_is_logit=logit, out={"y": y})
        buf = x["dST"].clone()
        g = a.linear_attention_backward(*args, ck, x["dy"], buf, f_is_logit=logit, out={"dS0": buf})
        assert bool((pad[:2048] == 7).all()) and bool((pad[2048 + n:] == 7).all())
        return [y.clone(), ST, ck] + [g[i] for i in sorted(g)]

    first = once()
    for _ in range(3):
        for p, r in zip(once(), first):
            assert torch.equal(p, r)
    ck = first[2]
    g = a.linear_attention_backward(*args, ck, x["dy"], x["dST"], f_is_logit=logit)
    for n, r in zip(sorted(g), first[3:]):
        assert torch.equal(g[n], r), n


def test_streams_and_graphs():
    """Two streams at once, and two captured graphs replayed in turn, give the eager results."""
    a = api()
    cases = [inputs(1, 2, 700, 64, 64, G=1, gate="logit", seed=s) for s in (23, 24)]

    def work(x, logit):
        y, ST, ck = a.linear_attention(x["k"], x["v"], x["q"], x["f"], x["S0"], want_ckpt=True, f_is_logit=logit)
        g = a.linear_attention_backward(x["k"], x["v"], x["q"], x["f"], ck, x["dy"], x["dST"], f_is_logit=logit)
        n, mu, r = a.layer_norm(y, torch.ones(2, 64, device=DEV))
        return [y, ST, n] + [g[i] for i in sorted(g)]

    eager = [work(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = []
    for s, c in zip(streams, cases):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs.append(work(*c))
    torch.cuda.synchronize()
    for e, o in zip(eager, outs):
        assert all(torch.equal(p, r) for p, r in zip(e, o))
    graphs, outs = [], []
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(work(*c))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for e, o in zip(eager, outs):
        assert all(torch.equal(p, r) for p, r in zip(e, o))


def test_gradients_against_differences():
    """fp32 mode: directional derivatives of a loss evaluated by the forward itself, in 64-bit sums."""
    a = api()
    x, _ = inputs(1, 2, 40, 16, 16, dtype=torch.float32, seed=25)
    args = {n: x[n] for n in ("k", "v", "q", "f", "S0")}
    _, _, ck = a.linear_attention(*args.values(), want_ckpt=True)
    g = a.linear_attention_backward(x["k"], x["v"], x["q"], x["f"], ck, x["dy"], x["dST"])

    def loss(kw):
        y, ST, _ = a.linear_attention(*kw.values())
        return float((y.double() * x["dy"].double()).sum() + (ST.double() * x["dST"].double()).sum())

    gen = torch.Generator(device=DEV).manual_seed(1)
    for n in args:
        d = torch.randn(args[n].shape, generator=gen, device=DEV) * (0.05 if n == "f" else 1.0)
        h = 2.0 ** -6
        num = (loss({**args, n: args[n] + h * d}) - loss({**args, n: args[n] - h * d})) / (2 * h)
        ana = float((g["d" + n].double() * d.double()).sum())
        # k, v, q, S0 enter linearly (no truncation error); f as a polynomial, whose h^2 term stays below
        # 1e-3 for steps of 2^-6 · 0.05.  The forward's fp32 rounding, 1e-5 of the loss, is divided by h.
        scale = float((g["d" + n].double().norm() * d.double().norm()))
        assert abs(num - ana) <= 4e-3 * scale, (n, num, ana)


def test_against_the_scan_without_its_tanh():
    """With W = 0 and inputs small enough that tanh(x) = x, the M²RNN scan is linear attention of (1 - f) k."""
    a = api()
    x, _ = inputs(2, 2, 150, 64, 64, dtype=torch.float32, start=False, seed=27)
    k = x["k"] * 1e-3
    f = torch.full_like(x["f"], 0.75)
    W = torch.zeros(2, 64, 64, device=DEV)
    y, HT, _ = a.forward(k, x["v"], x["q"], f, W)
    y2, ST, _ = a.linear_attention(0.25 * k, x["v"], x["q"], f)
    # tanh(x) = x (1 - x^2/3 ...) with |x| <= 1e-3 · |k_i v_j| < 1.5e-3: relative 1e-6, plus fp32 sums of 150 terms
    _, _, b = ref.forward(0.25 * k, x["v"], x["q"], f, bound=True)
    by, _, _ = ref.forward(0.25 * k, x["v"], x["q"], f, bound=True)
    assert bool(((y - y2).abs() <= 2e-5 * by + 1e-12).all())
    assert bool(((HT - ST).abs() <= 2e-5 * b[-1] + 1e-12).all())


def test_block_of_operators_trains():
    """Scan, readout norm, projection and back, as a layer runs them: every gradient against 64-bit autograd."""
    a = api()
    B, H, T, K, V = 2, 4, 200, 64, 64
    x, _ = inputs(B, H, T, K, V, start=False, seed=29)
    gen = torch.Generator(device=DEV).manual_seed(2)
    w = 1 + 0.1 * torch.randn(H, V, generator=gen, device=DEV)
    P = torch.randn(H * V, 32, generator=gen, device=DEV) * (H * V) ** -0.5
    dz = torch.randn(B, T, 32, generator=gen, device=DEV)
    y, ST, ck = a.linear_attention(x["k"], x["v"], x["q"], x["f"], want_ckpt=True)
    n, mean, rstd = a.layer_norm(y, w)
    dn = (dz @ P.t()).view(B, T, H, V).to(torch.bfloat16)
    gn = a.layer_norm_backward(dn, y, w, mean, rstd)
    g = a.linear_attention_backward(x["k"], x["v"], x["q"], x["f"], ck, gn["dx"])
    lv = {i: x[i].double().requires_grad_() for i in ("k", "v", "q", "f")}
    D = torch.cumsum(torch.log(lv["f"]), -1)
    M = torch.exp((D[..., :, None] - D[..., None, :]).tril()).tril()
    yr = ((lv["q"] @ lv["k"].transpose(-1, -2)) * M) @ lv["v"]
    wr = w.double().requires_grad_()
    yt = yr.transpose(1, 2)
    var, mu = torch.var_mean(yt, -1, correction=0, keepdim=True)
    nr = (yt - mu) / torch.sqrt(var + 1e-5) * wr
    (nr * dn.double()).sum().backward()
    got = {"k": g["dk"], "v": g["dv"], "q": g["dq"], "f": g["df"], "w": gn["dweight"]}
    for i, want in {**{i: t.grad for i, t in lv.items()}, "w": wr.grad}.items():
        rel = float((got[i].double() - want).norm() / want.norm())
        # y is rounded to bf16 once (2^-9 rms at most) and enters both the norm's values and dx, which is rounded
        # again; small |y| rows amplify it through rstd: a few roundings, 2^-9 each
        assert rel <= 8 * 2.0 ** -9, (i, rel)
    nr = nr.detach()
    assert float((n.double() - nr).norm() / nr.norm()) <= 4 * 2.0 ** -9
