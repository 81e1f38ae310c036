"""Linear attention in 64 bits, token by token from its definition, with the
bounds that the rounding tolerances are built from.

    S_t = f_t S_{t-1} + k_t v_tᵀ,  y_t = S_tᵀ q_t
    G_t = f_{t+1} G_{t+1} + q_t dy_tᵀ  (G_T also dST),  dq_t = S_t dy_t,  dk_t = G_t v_t,
    dv_t = G_tᵀ k_t,  df_t = <G_t, S_{t-1}>,  dS0 = f_1 G_1

`bound=True` runs the same sums on absolute values: what each result's rounding
errors are relative to."""
import torch


def _heads(x, H):
    return x.double().repeat_interleave(H // x.shape[1], 1)


def gates(f, B, H, T, logit):
    f = f.double()
    if f.dim() == 1:
        f = f[None, :, None].expand(B, H, T)
    return torch.sigmoid(f) if logit else f


def forward(k, v, q, f, S0=None, logit=False, bound=False):
    """(y, ST, [S_0 .. S_T])."""
    B, H, T, V = v.shape
    K = k.shape[-1]
    k, v, q = _heads(k, H), v.double(), _heads(q, H)
    S = torch.zeros(B, H, K, V, dtype=torch.float64, device=v.device) if S0 is None else S0.double()
    if bound:
        k, v, q, S = k.abs(), v.abs(), q.abs(), S.abs()
    g = gates(f, B, H, T, logit)
    states, y = [S], torch.zeros(B, H, T, V, dtype=torch.float64, device=v.device)
    for t in range(T):
        S = g[:, :, t, None, None] * S + k[:, :, t, :, None] * v[:, :, t, None, :]
        y[:, :, t] = (q[:, :, t, :, None] * S).sum(-2)
        states.append(S)
    return y, S, states


def backward(k, v, q, f, dy, S0=None, dST=None, logit=False, bound=False):
    B, H, T, V = v.shape
    G, K = k.shape[1], k.shape[-1]
    _, _, states = forward(k, v, q, f, S0, logit, bound)
    kk, vv, qq, dy = _heads(k, H), v.double(), _heads(q, H), dy.double()
    Gr = torch.zeros_like(states[0]) if dST is None else dST.double()
    if bound:
        kk, vv, qq, dy, Gr = kk.abs(), vv.abs(), qq.abs(), dy.abs(), Gr.abs()
    g = gates(f, B, H, T, logit)
    dk, dq, dv, df = torch.zeros_like(kk), torch.zeros_like(qq), torch.zeros_like(vv), torch.zeros_like(g)
    for t in reversed(range(T)):
        Gr = Gr + qq[:, :, t, :, None] * dy[:, :, t, None, :]
        dq[:, :, t] = (states[t + 1] * dy[:, :, t, None, :]).sum(-1)
        dk[:, :, t] = (Gr * vv[:, :, t, None, :]).sum(-1)
        dv[:, :, t] = (Gr * kk[:, :, t, :, None]).sum(-2)
        df[:, :, t] = (Gr * states[t]).sum((-1, -2))
        Gr = g[:, :, t, None, None] * Gr
    if logit:
        df = df * g * (1 - g)
    if f.dim() == 1:
        df = df.sum((0, 2))
    share = lambda x: x.view(B, G, H // G, T, K).sum(2)  # noqa: E731
    return {"dk": share(dk), "dv": dv, "dq": share(dq), "df": df, "dS0": Gr}
