"""The M²RNN update's factor (1 - f_t) in front of the input, put into v: the
gradients of v and f as the header gives them (64 bits, automatic differentiation)."""
import torch

import la_reference as ref


def test_scaled_values_and_their_gradients():
    g = torch.Generator().manual_seed(9)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    B, H, G, T, K, V = 2, 4, 2, 7, 3, 5
    k, q, S0, dy, dST = r(B, G, T, K), r(B, G, T, K), r(B, H, K, V), r(B, H, T, V), r(B, H, K, V)
    v, f = r(B, H, T, V).requires_grad_(), torch.sigmoid(r(B, H, T)).requires_grad_()
    S, ys = S0, []
    for t in range(T):      # S_t = f_t S_{t-1} + (1 - f_t) k_t v_tᵀ
        kt, ft = k[:, :, t].repeat_interleave(H // G, 1), f[:, :, t, None, None]
        S = ft * S + (1 - ft) * kt[..., :, None] * v[:, :, t, None, :]
        ys.append((q[:, :, t].repeat_interleave(H // G, 1)[..., :, None] * S).sum(-2))
    y = torch.stack(ys, 2)
    ((y * dy).sum() + (S * dST).sum()).backward()
    scaled = ((1 - f)[..., None] * v).detach()
    y2, S2, _ = ref.forward(k, scaled, q, f.detach(), S0)
    assert torch.allclose(y2, y, rtol=1e-12, atol=1e-12) and torch.allclose(S2, S, rtol=1e-12, atol=1e-12)
    d = ref.backward(k, scaled, q, f.detach(), dy, S0, dST)
    assert torch.allclose((1 - f.detach())[..., None] * d["dv"], v.grad, rtol=1e-10, atol=1e-12)
    assert torch.allclose(d["df"] - (v.detach() * d["dv"]).sum(-1), f.grad, rtol=1e-10, atol=1e-12)
