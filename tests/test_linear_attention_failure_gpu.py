"""A copy that never comes: the bounded waits of the linear-attention kernels
run out, the call reports it, and the next call works.  The failure is made on
the host (m2rnn_debug_set_fault makes the kernels stop fetching after their
first chunk), and no kernel outlives its wait limit."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture
def faulty():
    from non_linear_matrix_persistent_b200 import _lib, api
    api.set_wait_limit_ns(2_000_000)
    yield _lib, api
    _lib.lib().m2rnn_debug_set_fault(0)
    api.set_wait_limit_ns(2_000_000_000)
    api.device_status()


@pytest.mark.parametrize("K,V,H,T", [(64, 64, 150, 900), (64, 64, 2, 20000), (64, 128, 2, 20000), (128, 64, 150, 900),
                                     (128, 128, 150, 900), (128, 128, 2, 20000)])
def test_timeout_is_reported_and_cleared(faulty, K, V, H, T):
    """150 pairs walk all 8 chunks in one CTA each; 2 pairs split 157 chunks into segments of 3 (every walk has a
    second chunk, whose copy does not come)."""
    _lib, api = faulty
    g = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    k, v, q, dy = (n(1, H, T, w).to(torch.bfloat16) for w in (K, V, K, V))
    f = torch.rand(1, H, T, generator=g).cuda()
    y, ST, ck = api.linear_attention(k, v, q, f, want_ckpt=True)
    grads = api.linear_attention_backward(k, v, q, f, ck, dy)
    assert api.device_status() == _lib.OK
    _lib.lib().m2rnn_debug_set_fault(1)
    api.linear_attention(k, v, q, f)
    assert api.device_status() == _lib.ERR_DEVICE_TIMEOUT
    assert api.device_status() == _lib.OK
    api.linear_attention_backward(k, v, q, f, ck, dy)
    assert api.device_status() == _lib.ERR_DEVICE_TIMEOUT
    _lib.lib().m2rnn_debug_set_fault(0)
    api.set_wait_limit_ns(2_000_000_000)
    y2, ST2, ck2 = api.linear_attention(k, v, q, f, want_ckpt=True)
    assert torch.equal(y, y2) and torch.equal(ST, ST2) and torch.equal(ck, ck2)
    grads2 = api.linear_attention_backward(k, v, q, f, ck, dy)
    assert all(torch.equal(grads[i], grads2[i]) for i in grads)
    assert api.device_status() == _lib.OK
