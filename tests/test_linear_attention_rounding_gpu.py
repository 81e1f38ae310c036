"""bf16 results of linear attention are rounded once, from sums of fp32 accuracy,
at any length.

Tolerances, before any run.  A result's own rounding is half a step of bf16 (at
most 2^-8 of it).  What enters its sums in two bf16 terms is off by 2^-16, twice
in a path: 2^-15 of the sum of the terms' absolute values, which the reference
computes as `bound`; fp32 adds (T + 256) 2^-24 + 2^-20 of it.  Over a whole
tensor rounding errors are spread evenly over their step: the root of the sum of
half² / 3, which for the 9000 and more values here varies by less than 1% (the
mean of N such squares has a relative deviation of 0.9 / sqrt(N)): 10% are
allowed, and the other errors' bound at a quarter (they are as often positive as
negative, and few of them are as large as their bound)."""
import pytest
import torch

import la_reference as ref
from test_linear_attention_gpu import api, inputs

pytestmark = pytest.mark.gpu


def rounded_once(name, got, want, bound, T):
    assert got.dtype == torch.bfloat16 and got.numel() > 9000
    rest = (2.0 ** -15 + 2.0 ** -20 + (T + 256) * 2.0 ** -24) * bound + 1e-37
    err = (got.double() - want).abs()
    assert float((err - (2.0 ** -8 * (want.abs() + rest) + rest)).max()) <= 0, name
    half = torch.exp2(torch.floor(torch.log2(want.abs().clamp_min(1e-37))) - 8)
    most = 1.1 * float((half.square() / 3).sum().sqrt()) + 0.25 * float(rest.norm())
    assert float(err.norm()) <= most, (name, float(err.norm() / want.norm()), most / float(want.norm()))


SHAPES = [(16, 16), (64, 64), (32, 128), (64, 128), (128, 64), (128, 128)]


@pytest.mark.parametrize("K,V", SHAPES)
@pytest.mark.parametrize("B,H,T,G,gate", [(3, 4, 65, 4, "value"), (2, 3, 300, 1, "logit"), (1, 2, 1200, 2, "slow"),
                                          (30, 4, 261, 2, "head"), (2, 4, 200, 4, "edges")])
def test_forward_is_rounded_once(K, V, B, H, T, G, gate):
    x, logit = inputs(B, H, T, K, V, G=G, gate=gate, seed=50 + T)
    args = (x["k"], x["v"], x["q"], x["f"], x["S0"])
    y, _, _ = api().linear_attention(*args, f_is_logit=logit)
    rounded_once("y", y, ref.forward(*args, logit)[0], ref.forward(*args, logit, bound=True)[0], T)


@pytest.mark.parametrize("K,V", SHAPES)
@pytest.mark.parametrize("B,H,T,G,gate", [(3, 4, 65, 4, "value"), (2, 3, 300, 1, "logit"), (1, 2, 1200, 2, "slow"),
                                          (30, 4, 261, 2, "head"), (2, 4, 200, 4, "edges")])
def test_gradients_are_rounded_once(K, V, B, H, T, G, gate):
    x, logit = inputs(B, H, T, K, V, G=G, gate=gate, seed=60 + T)
    args = (x["k"], x["v"], x["q"], x["f"])
    _, _, ck = api().linear_attention(*args, x["S0"], want_ckpt=True, f_is_logit=logit)
    got = api().linear_attention_backward(*args, ck, x["dy"], x["dST"], f_is_logit=logit)
    want = ref.backward(*args, x["dy"], x["S0"], x["dST"], logit)
    bound = ref.backward(*args, x["dy"], x["S0"], x["dST"], logit, bound=True)
    for n in ("dk", "dv", "dq"):
        rounded_once(n, got[n], want[n], bound[n], T)
