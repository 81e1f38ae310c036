"""The cases by which the linear-attention scan and the readout norm are measured.

Linear attention with a decay for each head: per batch element b and head h,
    S_t = f_t S_{t-1} + k_t v_tᵀ,    y_t = S_tᵀ q_t,
with the layouts and gates of the M²RNN recurrence (head-first, k and q in G
head groups, f as a value in [0, 1], as a logit, or as one constant per head).
Forms: "step" (one token on a live state), "scan" (a prompt), "train" (a prompt
with checkpoints, then every gradient).

Layer norm and its RMS form: over the last dimension of rows, or per head over
a head-first readout [B, H, T, V], whose result is laid out token-first
[B, T, H, V] as the output projection reads it.  Forms: "norm" (forward) and
"norm_train" (forward, then dx, dweight and dbias).

`run` computes a case in its plain form (elementary torch operations in 32
bits, cumulative logarithms in 64), or, where `own` is true, through the calls
that a user makes.
"""
import math

import torch

own = False

CHUNK = 64          # tokens per chunk of the plain chunked form
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one token of one sequence on the 410M layer's state: pure latency
        _la("step_b1", "step", 1, 16, 1, 64, 64),
        # one token for each of 64 sequences, 7B-MoE layer: reads and writes 134 MB of state twice over
        _la("step_b64_7b", "step", 64, 32, 1, 128, 128, gate="logit"),
        # the 410M layer's prompt batch
        _la("scan_410m", "scan", 8, 16, 2048, 64, 64),
        # one long sequence continued from a state: only 16 (b, h) pairs
        _la("scan_long_b1", "scan", 1, 16, 16384, 64, 64, gate="logit", start=True),
        # the 7B-MoE layer's prompt batch
        _la("scan_7b", "scan", 4, 32, 4096, 128, 128),
        # odd length, shared k and q, K != V, a constant decay for each head
        _la("scan_grouped_odd", "scan", 3, 12, 1037, 128, 64, G=4, gate="head", start=True),
        # the 410M layer's training step
        _la("train_410m", "train", 8, 16, 2048, 64, 64),
        # the 7B-MoE layer's training step, gates as logits
        _la("train_7b", "train", 4, 32, 4096, 128, 128, gate="logit"),
        # the readout norm of one decoded token
        _norm("norm_token", "norm", 1, 16, 1, 64, heads=True, rms=True),
        # the readout norm of the 7B-MoE prompt batch: the M²RNN scan's fp32 readout to the projection's bf16 rows
        _norm("norm_readout_7b", "norm", 4, 32, 4096, 128, heads=True, x="fp32"),
        # the readout norm of the 410M layer, trained
        _norm("norm_train_410m", "norm_train", 8, 16, 2048, 64, heads=True, bias=True),
        # plain rows of a model width, odd count, trained
        _norm("norm_train_rows", "norm_train", 1, 1, 8191, 2048, bias=True),
    ]


def draw(rng):
    def near(lo, hi):   # spread over the logarithm
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    form = rng.choice(["step", "scan", "scan", "train", "train", "norm", "norm_train"])
    if form in ("norm", "norm_train"):
        heads = rng.random() < 0.6
        x = rng.choice(["bf16", "bf16", "fp32"])
        if heads:
            H, V = rng.randint(1, 32), rng.choice([16, 32, 64, 128])
            B = rng.randint(1, 8)
            T = near(1, min(16384, max(1, (1 << 26) // (B * H * V))))
        else:
            B, H, V = 1, 1, near(32, 8192)
            T = near(1, min(65536, (1 << 26) // V))
        c = _norm("", form, B, H, T, V, heads=heads, x=x, rms=rng.random() < 0.4, bias=rng.random() < 0.5)
    else:
        K, V = rng.choice([16, 32, 64, 64, 128, 128]), rng.choice([16, 32, 64, 64, 128, 128])
        G = rng.randint(1, 16)
        H = G * rng.choice([1, 1, 2, 4]) if G <= 8 else G
        gate = rng.choice(["value", "logit", "head"])
        if form == "step":
            B, T = near(1, 64), 1
        else:
            B = rng.randint(1, 8)
            T = near(1, min(16384, max(2, (1 << 26) // (B * H * max(K, V)))))
        c = _la("", form, B, H, T, K, V, G=G, gate=gate, start=rng.random() < 0.5)
    del c["name"]
    return c


def _la(name, form, B, H, T, K, V, G=0, gate="value", start=False):
    return {"name": name, "form": form, "B": B, "H": H, "G": G or H, "T": T, "K": K, "V": V, "gate": gate,
            "start": bool(start or form == "step")}


def _norm(name, form, B, H, T, V, heads=False, x="bf16", rms=False, bias=False):
    return {"name": name, "form": form, "B": B, "H": H, "T": T, "V": V, "heads": heads, "x": x, "rms": rms,
            "bias": bool(bias and not rms)}


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    B, H, T, V = case["B"], case["H"], case["T"], case["V"]
    s = {"case": case}
    if case["form"] in ("norm", "norm_train"):
        # a readout whose heads have different scales and a small offset
        scale = torch.exp(normal(1, H, 1, 1, std=0.5))
        x = (normal(B, H, T, V) * scale + 0.1 * normal(1, H, 1, V)).to(TYPES[case["x"]])
        shape = (H, V) if case["heads"] else (V,)
        s["x"] = x if case["heads"] else x.view(T, V)
        s["weight"] = 1.0 + normal(*shape, std=0.1)
        s["bias"] = normal(*shape, std=0.1) if case["bias"] else None
        if case["form"] == "norm_train":
            s["dy"] = normal(*((B, T, H, V) if case["heads"] else (T, V))).to(torch.bfloat16)
        return s
    G, K = case["G"], case["K"]
    tail = () if case["form"] == "step" else (T,)
    s["k"] = normal(B, G, *tail, K, std=K ** -0.5).to(torch.bfloat16)
    s["v"] = normal(B, H, *tail, V, std=V ** -0.5).to(torch.bfloat16)
    s["q"] = normal(B, G, *tail, K, std=K ** -0.5).to(torch.bfloat16)
    if case["gate"] == "value":        # the repository's gates: f = sigmoid(z + 2)
        s["f"] = torch.sigmoid(normal(B, H, *tail) + 2.0)
    elif case["gate"] == "logit":      # logits about per-head biases with retention times of 2 to 256 steps
        tau = torch.exp(torch.linspace(math.log(2.0), math.log(256.0), H, device="cuda")) if H > 1 else torch.full((1,), 16.0, device="cuda")
        s["f"] = normal(B, H, *tail) + torch.log(tau - 1.0 + 1e-3).view(1, H, *(1 for _ in tail))
    else:                              # one constant per head, retention times of 4 to 1024 steps
        s["f"] = 1.0 - torch.exp(-(math.log(4.0) + torch.rand(H, generator=g, device="cuda") * math.log(256.0)))
    s["S0"] = normal(B, H, K, V, std=0.5) if case["start"] else None
    if case["form"] == "train":
        s["dy"] = normal(B, H, T, V).to(torch.bfloat16)
        s["dST"] = normal(B, H, K, V) if case["start"] else None
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    form = state["case"]["form"]
    if own:
        return _OWN[form](state)
    return _PLAIN[form](state)


def _api():
    from non_linear_matrix_persistent_b200 import api
    return api


def _own_step(s):
    ST = torch.empty_like(s["S0"])      # the state before the token stays, so that a pass can be repeated
    y = _api().linear_attention_step(s["k"], s["v"], s["q"], s["f"], s["S0"], ST=ST, f_is_logit=s["case"]["gate"] == "logit")
    return {"y": y, "ST": ST}


def _own_scan(s):
    y, ST, _ = _api().linear_attention(s["k"], s["v"], s["q"], s["f"], s["S0"], f_is_logit=s["case"]["gate"] == "logit")
    return {"y": y, "ST": ST}


def _own_train(s):
    api, logit = _api(), s["case"]["gate"] == "logit"
    y, ST, ckpt = api.linear_attention(s["k"], s["v"], s["q"], s["f"], s["S0"], want_ckpt=True, f_is_logit=logit)
    grads = api.linear_attention_backward(s["k"], s["v"], s["q"], s["f"], ckpt, s["dy"], s["dST"], f_is_logit=logit)
    return {"y": y, "ST": ST, **grads}


def _own_norm(s):
    y, _, _ = _api().layer_norm(s["x"], s["weight"], s["bias"], rms=s["case"]["rms"], out_dtype=torch.bfloat16)
    return {"y": y}


def _own_norm_train(s):
    api, rms = _api(), s["case"]["rms"]
    y, mean, rstd = api.layer_norm(s["x"], s["weight"], s["bias"], rms=rms, out_dtype=torch.bfloat16)
    g = api.layer_norm_backward(s["dy"], s["x"], s["weight"], mean, rstd, rms=rms)
    return {"y": y, "dx": g["dx"], "dweight": g["dweight"], "dbias": g["dbias"] if s["case"]["bias"] else None}


_OWN = {"step": _own_step, "scan": _own_scan, "train": _own_train, "norm": _own_norm, "norm_train": _own_norm_train}


# ---------------------------------------------------------------- plain forms
def _gate(s):
    """The gates f_t as 64-bit values, broadcast to [B, H, T] (or [B, H])."""
    c = s["case"]
    f = s["f"].double()
    if c["gate"] == "logit":
        return 1.0 / (1.0 + torch.exp(-f))
    if c["gate"] == "head":
        return f.view(1, -1).expand(c["B"], c["H"]) if c["form"] == "step" else f.view(1, -1, 1).expand(c["B"], c["H"], c["T"])
    return f


def _per_head(x, H):
    """[B, G, ...] -> [B, H, ...] in 32 bits: head h reads group h // (H / G)."""
    return x.float().repeat_interleave(H // x.shape[1], 1)


def _plain_step(s):
    H = s["case"]["H"]
    k, v, q, f = _per_head(s["k"], H), s["v"].float(), _per_head(s["q"], H), _gate(s).float()
    S = f[..., None, None] * s["S0"] + k[..., :, None] * v[..., None, :]
    return {"y": (S * q[..., :, None]).sum(-2).to(torch.bfloat16), "ST": S}


def _chunks(x, n):
    """[B, H, T, X] -> [B, H, n, CHUNK, X], zeros behind the last token."""
    B, H, T, X = x.shape
    return torch.nn.functional.pad(x, (0, 0, 0, n * CHUNK - T)).view(B, H, n, CHUNK, X)


def _decays(f, n):
    """Inside chunks: a_t (chunk start to t), b_t (t to chunk end), D_ts (s to t); between chunks: the n by n products."""
    lg = torch.nn.functional.pad(torch.log(f), (0, n * CHUNK - f.shape[-1])).view(*f.shape[:2], n, CHUNK)
    L = lg.cumsum(-1)
    end = L[..., -1:]
    D = torch.exp((L[..., :, None] - L[..., None, :]).tril()).tril().float()
    E = end[..., 0].cumsum(-1)              # log decay from the very start to each chunk's end
    pre = E - end[..., 0]                   # and to each chunk's start
    fwd = torch.exp((pre[..., :, None] - E[..., None, :]).tril(-1)).tril(-1).float()   # chunk j's end -> chunk i's start
    return torch.exp(L).float(), torch.exp(end - L).float(), D, fwd, torch.exp(pre).float(), torch.exp(E[..., -1:] - E).float(), torch.exp(end[..., 0]).float()


def _plain_forward(s):
    c = s["case"]
    B, H, T, K, V = c["B"], c["H"], c["T"], c["K"], c["V"]
    n = -(-T // CHUNK)
    k, v, q = (_chunks(x, n) for x in (_per_head(s["k"], H), s["v"].float(), _per_head(s["q"], H)))
    a, b, D, fwd, pre, post, A = _decays(_gate(s), n)
    add = (k * b[..., None]).transpose(-1, -2) @ v                          # what each chunk adds to the state
    S = (fwd @ add.view(B, H, n, K * V)).view(B, H, n, K, V)                # the states at chunk starts
    if s["S0"] is not None:
        S = S + pre[..., None, None] * s["S0"][:, :, None]
    P = (q @ k.transpose(-1, -2)) * D
    y = P @ v + a[..., None] * (q @ S)
    ST = A[..., -1, None, None] * S[:, :, -1] + add[:, :, -1]
    return k, v, q, a, b, D, fwd, pre, post, A, S, P, y.view(B, H, n * CHUNK, V)[:, :, :T], ST


def _plain_scan(s):
    *_, y, ST = _plain_forward(s)
    return {"y": y.to(torch.bfloat16), "ST": ST}


def _plain_train(s):
    c = s["case"]
    B, H, G, T, K, V = c["B"], c["H"], c["G"], c["T"], c["K"], c["V"]
    k, v, q, a, b, D, fwd, pre, post, A, S, P, y, ST = _plain_forward(s)
    n = k.shape[2]
    dy = _chunks(s["dy"].float(), n)
    back = (q * a[..., None]).transpose(-1, -2) @ dy                        # what each chunk adds to the state's gradient
    E = (fwd.transpose(-1, -2) @ back.view(B, H, n, K * V)).view(B, H, n, K, V)   # the gradients at chunk ends
    dST = s["dST"]
    if dST is not None:
        E = E + post[..., None, None] * dST[:, :, None]
    dS0 = A[..., 0, None, None] * E[:, :, 0] + back[:, :, 0]
    dP = (dy @ v.transpose(-1, -2)) * D                                     # includes the decays
    qi = a[..., None] * (dy @ S.transpose(-1, -2))
    ki = b[..., None] * (v @ E.transpose(-1, -2))
    dq = dP @ k + qi
    dk = dP.transpose(-1, -2) @ q + ki
    dv = P.transpose(-1, -2) @ dy + b[..., None] * (k @ E)
    # f_u df_u: every path from a source s < u to a sink t >= u
    W = dP * (q @ k.transpose(-1, -2))
    over_t = W.flip(-2).cumsum(-2).flip(-2)                                 # over t >= u
    paths = over_t.tril(-1).sum(-1)                                         # over s < u
    paths = paths + (q * qi).sum(-1).flip(-1).cumsum(-1).flip(-1)
    kk = (k * ki).sum(-1)
    paths = paths + kk.cumsum(-1) - kk
    paths = paths + (A * (S * E).sum((-1, -2)))[..., None]
    f = _gate(s)
    df = paths.view(B, H, n * CHUNK)[:, :, :T].double()
    df = df * (1.0 - f) if c["gate"] == "logit" else df / f
    if c["gate"] == "head":
        df = df.sum((0, 2))

    def groups(x):
        return x.view(B, G, H // G, n * CHUNK, K)[:, :, :, :T].sum(2).to(torch.bfloat16)

    return {"y": y.to(torch.bfloat16), "ST": ST, "dk": groups(dk), "dv": dv.view(B, H, n * CHUNK, V)[:, :, :T].to(torch.bfloat16),
            "dq": groups(dq), "df": df.float(), "dS0": dS0}


EPS = 1e-5


def _plain_norm_parts(s):
    c = s["case"]
    x = s["x"].float()
    x = x.transpose(1, 2) if c["heads"] else x
    m = x - x.mean(-1, keepdim=True) if not c["rms"] else x
    r = 1.0 / torch.sqrt((m * m).mean(-1, keepdim=True) + EPS)
    n = m * r
    y = n * s["weight"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return n, r, y.to(torch.bfloat16)


def _plain_norm(s):
    return {"y": _plain_norm_parts(s)[2]}


def _plain_norm_train(s):
    c = s["case"]
    n, r, y = _plain_norm_parts(s)
    dy = s["dy"].float()
    dn = dy * s["weight"]
    dx = dn - n * (dn * n).mean(-1, keepdim=True)
    if not c["rms"]:
        dx = dx - dn.mean(-1, keepdim=True)
    dx = dx * r
    dx = dx.transpose(1, 2).contiguous() if c["heads"] else dx
    rows = (0, 1) if c["heads"] else (0,)
    return {"y": y, "dx": dx.to(s["x"].dtype), "dweight": (dy * n).sum(rows), "dbias": dy.sum(rows) if c["bias"] else None}


_PLAIN = {"step": _plain_step, "scan": _plain_scan, "train": _plain_train, "norm": _plain_norm, "norm_train": _plain_norm_train}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    B, H, T, V = case["B"], case["H"], case["T"], case["V"]
    if case["form"] in ("norm", "norm_train"):
        n, xs = B * H * T * V, 2 if case["x"] == "bf16" else 4
        per = H * V if case["heads"] else V
        params = 4 * per * (2 if case["bias"] else 1)
        if case["form"] == "norm":
            return {"bytes": n * (xs + 2) + params, "flops": 8 * n}
        return {"bytes": n * (xs + 2 + 2 + xs) + 2 * params, "flops": 20 * n}
    G, K = case["G"], case["K"]
    f = H if case["gate"] == "head" else B * H * T
    state = 4 * B * H * K * V
    kq, vy = 2 * B * G * T * K, 2 * B * H * T * V
    if case["form"] == "train":
        states = state * (4 if case["start"] else 2)       # S0, dST in; ST, dS0 out
        return {"bytes": 4 * kq + 4 * vy + 8 * f + states, "flops": 16 * B * H * T * K * V}
    states = state * (2 if case["start"] else 1)
    return {"bytes": 2 * kq + 2 * vy + 4 * f + states, "flops": 4 * B * H * T * K * V}


# ---------------------------------------------------------------- the definition, in 64 bits
def exact(case, seed):
    """The norm's gradients by automatic differentiation.  The scan as the recurrence itself, token by token; its
    backward walks in reverse from states kept at every 64th token."""
    c, s = case, prepare(case, seed)
    if c["form"] in ("norm", "norm_train"):
        return _exact_norm(c, s)
    B, H, G, T, K, V = c["B"], c["H"], c["G"], c["T"], c["K"], c["V"]
    if T * B * H * K * V > 1.5e10:
        return None
    per = [h // (H // G) for h in range(H)]
    lift = (lambda x: x.unsqueeze(2)) if c["form"] == "step" else (lambda x: x)
    k, q, v = lift(s["k"]).double()[:, per], lift(s["q"]).double()[:, per], lift(s["v"]).double()
    raw = s["f"].double()
    raw = raw[None, :, None].expand(B, H, T) if c["gate"] == "head" else lift(raw) if c["form"] == "step" else raw
    f = torch.sigmoid(raw) if c["gate"] == "logit" else raw
    S = s["S0"].double().clone() if s["S0"] is not None else torch.zeros(B, H, K, V, dtype=torch.float64, device="cuda")
    y = torch.empty(B, H, T, V, dtype=torch.float64, device="cuda")
    kept = []
    for t in range(T):
        if t % 64 == 0 and c["form"] == "train":
            kept.append(S.clone())
        S.mul_(f[:, :, t, None, None]).add_(k[:, :, t, :, None] * v[:, :, t, None, :])
        y[:, :, t] = torch.matmul(q[:, :, t, None, :], S)[:, :, 0]
    if c["form"] == "step":
        return {"y": y[:, :, 0], "ST": S}
    if c["form"] == "scan":
        return {"y": y, "ST": S}
    dy = s["dy"].double()
    Gt = s["dST"].double().clone() if s["dST"] is not None else torch.zeros_like(S)
    dk, dq, dv, df = torch.empty_like(k), torch.empty_like(q), torch.empty_like(v), torch.empty_like(f)
    for i in reversed(range(len(kept))):
        P, before = kept[i], []
        for t in range(64 * i, min(T, 64 * i + 64)):
            before.append(P)
            P = f[:, :, t, None, None] * P + k[:, :, t, :, None] * v[:, :, t, None, :]
        after = before[1:] + [P]
        for t in reversed(range(64 * i, min(T, 64 * i + 64))):
            j = t - 64 * i
            dq[:, :, t] = torch.matmul(after[j], dy[:, :, t, :, None])[..., 0]
            Gt.add_(q[:, :, t, :, None] * dy[:, :, t, None, :])
            dk[:, :, t] = torch.matmul(Gt, v[:, :, t, :, None])[..., 0]
            dv[:, :, t] = torch.matmul(k[:, :, t, None, :], Gt)[:, :, 0]
            df[:, :, t] = (Gt * before[j]).sum((-1, -2))
            Gt.mul_(f[:, :, t, None, None])
    if c["gate"] == "logit":
        df = df * f * (1.0 - f)
    if c["gate"] == "head":
        df = df.sum((0, 2))
    return {"y": y, "ST": S, "dk": dk.view(B, G, H // G, T, K).sum(2), "dv": dv, "dq": dq.view(B, G, H // G, T, K).sum(2), "df": df, "dS0": Gt}


def _exact_norm(c, s):
    x = s["x"].double().requires_grad_()
    w = s["weight"].double().requires_grad_()
    b = None if s["bias"] is None else s["bias"].double().requires_grad_()
    z = x.permute(0, 2, 1, 3) if c["heads"] else x
    if c["rms"]:
        z = z / (z.square().mean(-1, keepdim=True) + EPS).sqrt()
    else:
        var, mean = torch.var_mean(z, -1, correction=0, keepdim=True)
        z = (z - mean) / (var + EPS).sqrt()
    y = z * w if b is None else z * w + b
    if c["form"] == "norm":
        return {"y": y.detach()}
    y.backward(s["dy"].double())
    return {"y": y.detach(), "dx": x.grad, "dweight": w.grad, "dbias": None if b is None else b.grad}
