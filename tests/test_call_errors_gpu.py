"""A call that fails on the host leaves nothing behind for the next one."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_a_failed_call_does_not_fail_the_next():
    """The status call copies and synchronises, which a stream that is being captured refuses (a host-side error)."""
    from non_linear_matrix_persistent_b200 import _lib, api
    rt, L = ctypes.CDLL("libcudart.so.12"), _lib.lib()
    rt.cudaStreamBeginCapture.argtypes = [ctypes.c_void_p, ctypes.c_int]
    rt.cudaStreamEndCapture.argtypes = [ctypes.c_void_p, ctypes.POINTER(ctypes.c_void_p)]
    g = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    k, v = n(1, 2, 40, 64).to(torch.bfloat16), n(1, 2, 40, 64).to(torch.bfloat16)
    f, x = torch.rand(1, 2, 40, generator=g).cuda(), n(5, 64)
    y = api.linear_attention(k, v, k, f)[0]        # (and the kernels' code is loaded)
    z = api.layer_norm(x)[0]
    assert api.device_status() == _lib.OK
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for again in (lambda: torch.equal(api.linear_attention(k, v, k, f)[0], y), lambda: torch.equal(api.layer_norm(x)[0], z),
                  lambda: api.device_status() == _lib.OK):
        torch.cuda.synchronize()
        assert rt.cudaStreamBeginCapture(s.cuda_stream, 1) == 0     # thread-local mode
        assert L.m2rnn_linear_attention_status(s.cuda_stream) == _lib.ERR_CUDA
        graph = ctypes.c_void_p()
        assert rt.cudaStreamEndCapture(s.cuda_stream, ctypes.byref(graph)) != 0 and not graph.value
        rt.cudaGetLastError()                                       # the test's own error
        assert again()
