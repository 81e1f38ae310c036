"""Waits that run out at the shortest limit, again and again: every call still
ends and reports it.  The lanes of a warp then give up at the moment at which a
phase may complete for some of them, and have to answer as one: a warp whose
lanes part between the way out and a tensor-memory access or a shuffle would
never end.  The failure is made on the host (the kernels stop fetching after
their first chunk)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture
def faulty():
    from non_linear_matrix_persistent_b200 import _lib, api
    yield _lib, api
    _lib.lib().m2rnn_debug_set_fault(0)
    api.set_wait_limit_ns(2_000_000_000)
    api.device_status()


@pytest.mark.parametrize("K,V", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("H,T", [(150, 600), (2, 20000)])
def test_every_timeout_ends_and_is_reported(faulty, K, V, H, T):
    _lib, api = faulty
    g = torch.Generator().manual_seed(2)
    n = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    k, v, q, dy = (n(1, H, T, w).to(torch.bfloat16) for w in (K, V, K, V))
    f = torch.rand(1, H, T, generator=g).cuda()
    y, ST, ck = api.linear_attention(k, v, q, f, want_ckpt=True)
    grads = api.linear_attention_backward(k, v, q, f, ck, dy)
    assert api.device_status() == _lib.OK
    _lib.lib().m2rnn_debug_set_fault(1)
    for i in range(12):
        api.set_wait_limit_ns(100_000 + 700 * i)
        api.linear_attention(k, v, q, f)
        assert api.device_status() == _lib.ERR_DEVICE_TIMEOUT
        api.linear_attention_backward(k, v, q, f, ck, dy)
        assert api.device_status() == _lib.ERR_DEVICE_TIMEOUT
    _lib.lib().m2rnn_debug_set_fault(0)
    api.set_wait_limit_ns(2_000_000_000)
    y2, ST2, ck2 = api.linear_attention(k, v, q, f, want_ckpt=True)
    grads2 = api.linear_attention_backward(k, v, q, f, ck, dy)
    assert torch.equal(y, y2) and torch.equal(ST, ST2) and torch.equal(ck, ck2)
    assert all(torch.equal(grads[i], grads2[i]) for i in grads)
    assert api.device_status() == _lib.OK
