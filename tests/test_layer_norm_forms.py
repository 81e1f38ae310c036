"""Which form a norm's backward takes where no weight says it."""
import pytest
import torch

from non_linear_matrix_persistent_b200 import api


def test_ambiguous_and_contradicting_forms_are_refused():
    x = torch.zeros(2, 5, 5, 64)
    stats = torch.zeros(2, 5, 5)
    with pytest.raises(ValueError, match="say which with heads"):       # dy [B, T, H, N] and [B, H, T, N] are the same shape
        api.layer_norm_backward(x, x, None, stats, stats)
    for heads, w in ((True, torch.ones(64)), (False, torch.ones(5, 64))):
        with pytest.raises(ValueError, match="contradicts"):
            api.layer_norm_backward(x, x, w, stats, stats, heads=heads)
    with pytest.raises(ValueError, match="heads=True"):
        api.layer_norm_backward(x[0], x[0], None, stats[0], stats[0], heads=True)
    for args in ((None, None), (None, False), (None, True), (torch.ones(64), False), (torch.ones(5, 64), True)):
        y = x if args != (None, None) else torch.zeros(2, 5, 4, 64)
        with pytest.raises(ValueError, match="CUDA"):                   # what is left to refuse here
            api.layer_norm_backward(y, y, args[0], stats, stats, heads=args[1])


@pytest.mark.gpu
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("shape", [(2, 6, 6, 64), (1, 3, 3, 100), (2, 1, 1, 32), (2, 3, 7, 64)])
def test_readout_and_rows_without_a_weight(shape, rms):
    """A readout's bias makes the forward's form a readout's; its backward, told so, is that of a weight of ones."""
    B, H, T, N = shape
    g = torch.Generator().manual_seed(4)
    x, dy, rows = (torch.randn(*s, generator=g).cuda() for s in (shape, (B, T, H, N), shape))
    y, mean, rstd = api.layer_norm(x, None, torch.zeros(H, N, device="cuda"), rms=rms)
    assert y.shape == (B, T, H, N)
    want = api.layer_norm_backward(dy, x, torch.ones(H, N, device="cuda"), mean, rstd, rms=rms)
    got = api.layer_norm_backward(dy, x, None, mean, rstd, rms=rms, heads=True)
    assert all(torch.equal(got[n], want[n]) for n in want) and got["dweight"].shape == (H, N)
    want = api.layer_norm_backward(rows, x, torch.ones(N, device="cuda"), mean, rstd, rms=rms)
    forms = (False,) if H == T > 1 else (False, None)
    for heads in forms:
        got = api.layer_norm_backward(rows, x, None, mean, rstd, rms=rms, heads=heads)
        assert all(torch.equal(got[n], want[n]) for n in want) and got["dweight"].shape == (N,)
