"""Many heads: the kernel that sums the weight's and bias's gradients takes any
number of heads that the dims allow, and what it cannot take is refused before
anything is launched."""
import pytest
import torch

from non_linear_matrix_persistent_b200 import _lib, build

NAMES = "dy x w m r dx dw db ws".split()


def test_too_many_sums_are_refused():
    build.build()
    L = _lib.lib()
    bwd = lambda d, **p: L.m2rnn_layer_norm_backward(d, *({**dict.fromkeys(NAMES, 4096), **p}[i] for i in NAMES), 1 << 62, None)  # noqa: E731
    # 2^20 heads of 2^16 columns: 2^32 blocks of 32 columns of dweight and dbias
    d = _lib.NormDims(1, 1 << 20, 1, 1 << 16, 0, 0, 0, 0, 1e-5)
    assert bwd(d) == _lib.ERR_UNSUPPORTED_SHAPE == bwd(d, dw=None) == bwd(d, db=None)
    assert L.m2rnn_layer_norm_workspace(d) == _lib.REFUSED
    # a quarter of the columns: 2^30 blocks, a workspace is wanted
    d = _lib.NormDims(1, 1 << 20, 1, 1 << 14, 0, 0, 0, 0, 1e-5)
    assert 0 < L.m2rnn_layer_norm_workspace(d) < _lib.REFUSED
    assert bwd(d, ws=None) == _lib.ERR_WORKSPACE


@pytest.mark.gpu
@pytest.mark.parametrize("H,T,N", [(65535, 1, 8), (65536, 1, 8), (70000, 2, 5), (1 << 20, 1, 1)])
def test_weight_gradients_of_many_heads(H, T, N):
    from non_linear_matrix_persistent_b200 import api
    g = torch.Generator().manual_seed(H)
    x = torch.randn(1, H, T, N, generator=g).cuda()
    dy = torch.randn(1, T, H, N, generator=g).cuda()
    w = 1 + 0.2 * torch.randn(H, N, generator=g).cuda()
    y, mean, rstd = api.layer_norm(x, w, eps=0.5)
    d = api.layer_norm_backward(dy, x, w, mean, rstd)
    z = x.double().transpose(1, 2)
    n = (z - z.mean(-1, keepdim=True)) / torch.sqrt(z.var(-1, correction=0, keepdim=True) + 0.5)
    # fp32 statistics of at most 8 values of size 1 and sums of at most 2 terms: a few 2^-24 of |x| + 1, at most 2^2 of them
    tol = 2.0 ** -24 * 16 * (z.abs() + 1)
    assert bool(((y.double() - n * w.double()).abs() <= tol * w.double().abs()).all())
    assert bool(((d["dweight"].double() - (dy.double() * n).sum((0, 1))).abs() <= (dy.double().abs() * tol).sum((0, 1))).all())
    assert bool(((d["dbias"].double() - dy.double().sum((0, 1))).abs() <= 2.0 ** -22 * dy.double().abs().sum((0, 1))).all())
    again = api.layer_norm(x, w, eps=0.5)[0]      # a call after it is not told of an old error
    assert torch.equal(again, y)
