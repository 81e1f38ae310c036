"""Linear attention and the readout norm with heads sharded over ranks: each
rank's shard gives its slice of the whole problem's results (64-bit reference)."""
import pytest
import torch

import la_reference as ref
from non_linear_matrix_persistent_b200 import parallel

B, H, G, T, K, V = 2, 6, 3, 5, 3, 4


def problem(per_head):
    g = torch.Generator().manual_seed(7)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    f = torch.sigmoid(r(H) if per_head else r(B, H, T))
    return dict(k=r(B, G, T, K), v=r(B, H, T, V), q=r(B, G, T, K), f=f, S0=r(B, H, K, V), dy=r(B, H, T, V), dST=r(B, H, K, V),
                weight=r(H, V), bias=r(H, V), W=None)


def results(x):
    y, ST, _ = ref.forward(x["k"], x["v"], x["q"], x["f"], x["S0"])
    d = ref.backward(x["k"], x["v"], x["q"], x["f"], x["dy"], x["S0"], x["dST"])
    n = torch.nn.functional.layer_norm(y, (V,))
    rstd = 1 / torch.sqrt(y.var(-1, correction=0) + 1e-5)
    rows = (n * x["weight"][:, None] + x["bias"][:, None]).transpose(1, 2)       # token-first
    dweight = (n * x["dy"]).sum((0, 2))
    return dict(d, y=y, ST=ST, n=rows, mean=y.mean(-1), rstd=rstd, dweight=dweight, dbias=x["dy"].sum((0, 2)))


@pytest.mark.parametrize("per_head", [False, True])
def test_shards_give_slices(per_head):
    x = problem(per_head)
    whole = results(x)
    for rank in range(3):
        part = parallel.head_shard({**x, **whole}, rank, 3)
        assert part["W"] is None and all(t is None or t.is_contiguous() for t in part.values())
        assert part["weight"].shape == (2, V) and part["k"].shape[1] == 1
        for n, t in results(part).items():
            assert t.shape == part[n].shape and torch.allclose(t, part[n], rtol=1e-12, atol=1e-13), n


def test_one_token():
    x = problem(True)
    tok = {n: x[n][:, :, 0] for n in ("k", "v", "q")}
    s = parallel.head_shard({**tok, "f": x["f"], "S0": x["S0"]}, 1, 3)
    assert torch.equal(s["k"], tok["k"][:, 1:2]) and torch.equal(s["v"], tok["v"][:, 2:4])
    assert torch.equal(s["f"], x["f"][2:4]) and torch.equal(s["S0"], x["S0"][:, 2:4])


@pytest.mark.parametrize("name,shape", [("weight", (V,)), ("dbias", (V,)), ("bias", (V, H)), ("f", (T,)), ("n", (B, H, T, V)),
                                        ("y", (B, T, H, V)), ("W", (1, V, V)), ("mean", (B,))])
def test_tensors_without_their_heads_are_refused(name, shape):
    with pytest.raises(ValueError, match=name):
        parallel.head_shard({**problem(False), name: torch.zeros(shape)}, 0, 3)
