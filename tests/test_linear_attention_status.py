"""Whose time-outs device_status reports: those of the stream that asks, and of
captured calls, which no stream owns.  (The failures are made on the host: the
kernels stop fetching after their first chunk.)"""
import subprocess
import sys

import pytest
import torch

from non_linear_matrix_persistent_b200 import _lib, build


def test_nothing_to_report_needs_no_device():
    build.build()
    if not torch.cuda.is_available():
        assert _lib.lib().m2rnn_linear_attention_status(None) == _lib.OK


@pytest.fixture
def faulty():
    from non_linear_matrix_persistent_b200 import api
    g = torch.Generator().manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=g).cuda().to(torch.bfloat16)  # noqa: E731
    x = n(1, 150, 300, 64), n(1, 150, 300, 64), n(1, 150, 300, 64), torch.rand(1, 150, 300, generator=g).cuda()
    torch.cuda.synchronize()
    api.set_wait_limit_ns(1_000_000)
    yield api, x, _lib.lib().m2rnn_debug_set_fault
    _lib.lib().m2rnn_debug_set_fault(0)
    api.set_wait_limit_ns(2_000_000_000)
    torch.cuda.synchronize()
    api.device_status()


@pytest.mark.gpu
def test_each_stream_is_told_of_its_own_calls(faulty):
    api, x, fault = faulty
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(b):
        api.linear_attention(*x)
    with torch.cuda.stream(a):
        fault(1)
        api.linear_attention(*x)
        fault(0)
    torch.cuda.synchronize()
    with torch.cuda.stream(b):
        assert api.device_status() == _lib.OK
    assert api.device_status() == _lib.OK
    with torch.cuda.stream(a):
        assert api.device_status() == _lib.ERR_DEVICE_TIMEOUT
        assert api.device_status() == _lib.OK


def in_a_process_of_its_own(code):
    r = subprocess.run([sys.executable, "-c", "import ctypes, torch\nfrom non_linear_matrix_persistent_b200 import _lib, api\n"
                        "rt = ctypes.CDLL('libcudart.so.12')\n" + code + "\nprint('done')"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "done" in r.stdout, r.stderr[-2000:]


@pytest.mark.gpu
def test_a_stream_without_calls_is_not_waited_for():
    """A step's kernel waits for nothing and has no status; calls on another stream are not this one's."""
    in_a_process_of_its_own("""
x = [torch.zeros(1, 2, 300, 64, dtype=torch.bfloat16, device="cuda") for _ in range(3)] + [torch.ones(1, 2, 300, device="cuda")]
api.linear_attention(*x)
assert api.device_status() == _lib.OK
done = torch.cuda.Event()
with torch.cuda.stream(torch.cuda.Stream()):
    api.linear_attention_step(*(t[:, :, 0].contiguous() for t in x), torch.zeros(1, 2, 64, 64, device="cuda"))
    torch.cuda.current_stream().synchronize()
    torch.cuda._sleep(400_000_000)       # a fifth of a second
    done.record()
    assert api.device_status() == _lib.OK
    assert not done.query()
    done.synchronize()
""")


@pytest.mark.gpu
def test_captured_calls_are_reported_to_the_stream_that_asks(faulty):
    api, x, fault = faulty
    graph = torch.cuda.CUDAGraph()
    fault(1)
    with torch.cuda.graph(graph):
        api.linear_attention(*x)
    fault(0)
    assert api.device_status() == _lib.OK
    for s in (torch.cuda.current_stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            graph.replay()
            assert api.device_status() == _lib.ERR_DEVICE_TIMEOUT
            assert api.device_status() == _lib.OK


@pytest.mark.gpu
def test_more_streams_than_words():
    """300 streams: the last ones share a status, none goes unreported (words are not given back)."""
    in_a_process_of_its_own("""
x = [torch.zeros(1, 2, 300, 64, dtype=torch.bfloat16, device="cuda") for _ in range(3)] + [torch.ones(1, 2, 300, device="cuda")]
torch.cuda.synchronize()
api.set_wait_limit_ns(1000000)
for i in range(300):
    s = ctypes.c_void_p()
    assert rt.cudaStreamCreateWithFlags(ctypes.byref(s), 1) == 0
    with torch.cuda.stream(torch.cuda.ExternalStream(s.value)):
        api.linear_attention_backward(*x, torch.zeros(1, 2, 3, 16, 64, 4, device="cuda"), x[1])
        torch.cuda.current_stream().synchronize()
        if i in (5, 254, 255, 299):
            many = [t.repeat(1, 75, *[1] * (t.dim() - 2)) for t in x]
            _lib.lib().m2rnn_debug_set_fault(1)
            api.linear_attention(*many)
            _lib.lib().m2rnn_debug_set_fault(0)
            torch.cuda.current_stream().synchronize()
            assert api.device_status() == _lib.ERR_DEVICE_TIMEOUT, i
        assert api.device_status() == _lib.OK, i
""")
