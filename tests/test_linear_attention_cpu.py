"""Host-only checks of linear attention and the layer norm: refusals of the C
ABI and of the binding (nothing is launched), and the 64-bit reference against
automatic differentiation and closed forms."""
import pytest
import torch

import la_reference as ref
from non_linear_matrix_persistent_b200 import _lib, api, build


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.lib()


def _dims(B=2, H=4, T=5, K=64, V=64, mode=0, G=0, logit=0, per_head=0):
    return _lib.LaDims(B, H, T, K, V, mode, G, logit, per_head)


def _fwd(L, d, ws_bytes=1 << 40, **ptrs):
    p = dict(k=4096, v=4096, q=4096, f=4096, S0=None, y=4096, ST=None, ckpt=None, ws=4096)
    p.update(ptrs)
    return L.m2rnn_linear_attention_forward(d, *(p[n] for n in ("k", "v", "q", "f", "S0", "y", "ST", "ckpt", "ws")),
                                            ws_bytes, None)


def _bwd(L, d, ws_bytes=1 << 40, **ptrs):
    names = ("k", "v", "q", "f", "ckpt", "dy", "dST", "dk", "dv", "dq", "df", "dS0", "ws")
    p = dict.fromkeys(names, 4096)
    p.update(dST=None)
    p.update(ptrs)
    return L.m2rnn_linear_attention_backward(d, *(p[n] for n in names), ws_bytes, None)


@pytest.mark.parametrize("bad,status", [
    (dict(B=-1), "INVALID_ARG"), (dict(T=-1), "INVALID_ARG"), (dict(mode=2), "INVALID_ARG"),
    (dict(mode=3), "INVALID_ARG"), (dict(mode=-1), "INVALID_ARG"), (dict(G=3), "INVALID_ARG"),
    (dict(G=5), "INVALID_ARG"), (dict(G=-1), "INVALID_ARG"), (dict(logit=2), "INVALID_ARG"),
    (dict(per_head=-1), "INVALID_ARG"), (dict(K=48), "UNSUPPORTED_SHAPE"), (dict(V=256), "UNSUPPORTED_SHAPE"),
    (dict(K=0), "UNSUPPORTED_SHAPE"), (dict(B=1 << 13, H=1 << 12), "UNSUPPORTED_SHAPE")])
def test_linear_attention_refuses_dims(L, bad, status):
    d, want = _dims(**bad), getattr(_lib, "ERR_" + status)
    assert _fwd(L, d) == want and _bwd(L, d) == want
    assert L.m2rnn_linear_attention_workspace(d, 0) == _lib.REFUSED == L.m2rnn_linear_attention_workspace(d, 1)


def test_linear_attention_refuses_pointers(L):
    assert _fwd(L, None) == _lib.ERR_INVALID_ARG and _bwd(L, None) == _lib.ERR_INVALID_ARG
    for n in ("k", "v", "q", "f", "y"):
        assert _fwd(L, _dims(), **{n: None}) == _lib.ERR_INVALID_ARG
    for n in ("k", "v", "q", "f", "ckpt", "dy", "dk", "dv", "dq", "df", "dS0"):
        assert _bwd(L, _dims(), **{n: None}) == _lib.ERR_INVALID_ARG
    for n in ("k", "S0", "ST", "ckpt", "ws"):
        assert _fwd(L, _dims(), **{n: 4104}) == _lib.ERR_MISALIGNED
    for n in ("dy", "dST", "df", "dS0"):
        assert _bwd(L, _dims(), **{n: 4100}) == _lib.ERR_MISALIGNED
    # grouped k / q and per-head gates need partial sums
    for d in (_dims(G=2), _dims(per_head=1)):
        need = L.m2rnn_linear_attention_workspace(d, 1)
        assert 0 < need < _lib.REFUSED
        assert _bwd(L, d, ws_bytes=need - 1) == _lib.ERR_WORKSPACE
        assert _bwd(L, d, ws=None) == _lib.ERR_WORKSPACE


def test_empty_problems_need_no_device(L):
    # no pairs: nothing to write, nothing launched, every pointer may be NULL
    none = dict.fromkeys(("k", "v", "q", "f", "y", "ws"))
    assert _fwd(L, _dims(B=0), **none) == _lib.OK
    none = dict.fromkeys(("k", "v", "q", "f", "ckpt", "dy", "dk", "dv", "dq", "df", "dS0", "ws"))
    assert _bwd(L, _dims(B=0), **none) == _lib.OK
    assert L.m2rnn_linear_attention_workspace(_dims(T=0, G=2, per_head=1), 1) == 0


def test_binding_refuses(L):
    B, H, T, K, V = 1, 2, 3, 64, 64
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t)  # noqa: E731
    k, v, f = z(B, H, T, K), z(B, H, T, V), z(B, H, T, t=torch.float32)
    with pytest.raises(ValueError, match="CUDA"):
        api.linear_attention(k, v, k, f)
    with pytest.raises(TypeError):
        api.linear_attention(k.half(), v.half(), k.half(), f)
    with pytest.raises(ValueError, match="divisor"):
        api.linear_attention(z(B, 3, T, K), v, z(B, 3, T, K), f)
    with pytest.raises(ValueError, match="4 dimensions"):
        api.linear_attention(k[0], v[0], k[0], f)
    with pytest.raises(ValueError, match="3 dimensions"):
        api.linear_attention_step(k, v, k, f, z(B, H, K, V, t=torch.float32))
    with pytest.raises(ValueError, match="state"):
        api.linear_attention_step(k[:, :, 0], v[:, :, 0], k[:, :, 0], f[:, :, 0], None)


def _norm(B=2, H=3, T=5, N=64, x=0, y=0, dx=0, rms=0, eps=1e-5):
    return _lib.NormDims(B, H, T, N, x, y, dx, rms, eps)


def test_layer_norm_refuses(L):
    fwd = lambda d, **p: L.m2rnn_layer_norm_forward(d, *({**dict(x=4096, w=4096, b=4096, y=4096, m=4096, r=4096), **p}[n] for n in "x w b y m r".split()), None)  # noqa: E731
    names = "dy x w m r dx dw db ws".split()
    bwd = lambda d, n=1 << 40, **p: L.m2rnn_layer_norm_backward(d, *({**dict.fromkeys(names, 4096), **p}[i] for i in names), n, None)  # noqa: E731
    for bad in (dict(B=-1), dict(N=0), dict(x=2), dict(y=-1), dict(dx=1), dict(rms=2), dict(eps=-1.0), dict(eps=float("nan"))):
        assert fwd(_norm(**bad)) == _lib.ERR_INVALID_ARG == bwd(_norm(**bad))
        assert L.m2rnn_layer_norm_workspace(_norm(**bad)) == _lib.REFUSED
    assert fwd(None) == _lib.ERR_INVALID_ARG == bwd(None)
    assert fwd(_norm(B=1 << 13, H=1 << 12)) == _lib.ERR_UNSUPPORTED_SHAPE
    assert fwd(_norm(B=1, H=1, T=(1 << 30) + 1, N=1)) == _lib.ERR_UNSUPPORTED_SHAPE
    for n in ("x", "y"):
        assert fwd(_norm(), **{n: None}) == _lib.ERR_INVALID_ARG
    for n in ("x", "w", "b", "y", "m", "r"):
        assert fwd(_norm(), **{n: 4100}) == _lib.ERR_MISALIGNED
    for n in ("dy", "x", "m", "r", "dx"):
        assert bwd(_norm(), **{n: None}) == _lib.ERR_INVALID_ARG
    need = L.m2rnn_layer_norm_workspace(_norm())
    assert bwd(_norm(), need - 1) == _lib.ERR_WORKSPACE == bwd(_norm(), ws=None)
    assert fwd(_norm(T=0), x=None, y=None) == _lib.OK


def test_layer_norm_binding_refuses(L):
    x = torch.zeros(2, 3, 5, 64)
    with pytest.raises(TypeError):
        api.layer_norm(x.half())
    with pytest.raises(ValueError, match="CUDA"):
        api.layer_norm(x)
    with pytest.raises(ValueError, match="weight per head"):
        api.layer_norm(x[0], torch.ones(3, 64))
    with pytest.raises(ValueError, match="empty"):
        api.layer_norm(torch.zeros(3, 0))
    with pytest.raises(ValueError, match="heads=True"):
        api.layer_norm_backward(x[0], x[0], None, x[0, :, :, 0], x[0, :, :, 0], heads=True)


@pytest.mark.parametrize("logit,per_head,start", [(False, False, True), (True, False, True), (False, True, False), (True, True, True)])
def test_reference_gradients_against_differences(logit, per_head, start):
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    B, H, G, T, K, V = 2, 4, 2, 5, 3, 2
    x = dict(k=r(B, G, T, K), v=r(B, H, T, V), q=r(B, G, T, K), f=r(H) if per_head else r(B, H, T),
             S0=r(B, H, K, V) if start else None)
    if not logit:
        x["f"] = torch.sigmoid(x["f"])
        x["f"].view(-1)[1] = 0.0                      # a gate that discards the state
    dy, dST = r(B, H, T, V), r(B, H, K, V)

    def loss(**kw):
        y, ST, _ = ref.forward(**{**x, **kw}, logit=logit)
        return float((y * dy).sum() + (ST * dST).sum())

    grads = ref.backward(x["k"], x["v"], x["q"], x["f"], dy, x["S0"], dST, logit)
    for n, gn in (("k", "dk"), ("v", "dv"), ("q", "dq"), ("f", "df"), ("S0", "dS0")):
        if x[n] is None:
            continue
        for _ in range(4):
            d = r(*x[n].shape)
            h = 1e-5
            num = (loss(**{n: x[n] + h * d}) - loss(**{n: x[n] - h * d})) / (2 * h)
            # central difference of a loss that is a polynomial (or a smooth function) of size O(10): h^2 + rounding/h
            assert abs(num - float((grads[gn] * d).sum())) < 1e-7 * max(1.0, abs(num)), n


def test_reference_closed_forms():
    g = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    k, v, q = r(1, 2, 6, 3), r(1, 2, 6, 2), r(1, 2, 6, 3)
    y, _, _ = ref.forward(k, v, q, torch.zeros(2))             # no memory: y_t = (q_t·k_t) v_t
    assert torch.allclose(y, (q * k).sum(-1, keepdim=True) * v)
    y, _, _ = ref.forward(k, v, q, torch.ones(2))              # no decay: causal sums
    assert torch.allclose(y, (q @ k.transpose(-1, -2)).tril() @ v)
