"""Python binding of libm2rnn.so over torch tensors (argument marshalling only).

Every step of the recurrence runs in the CUDA library; torch only provides
device memory and the current stream.  Names follow include/m2rnn.h.

  y, HT, ckpt = forward(k, v, q, f, W, H0=None, ckpt_stride=8, want_ckpt=False)
  grads       = backward(k, v, q, f, W, ckpt, dy, dHT=None, ckpt_stride=8)
  y_t         = step(k_t, v_t, q_t, f_t, W, H)        # one decode step, H updated in place
  b           = decay_logit_bias(H)                   # per-head gate-logit bias at initialisation
  y, ST, ckpt = linear_attention(k, v, q, f, S0=None, want_ckpt=False)   # S_t = f_t S_{t-1} + k_t v_tᵀ
  grads       = linear_attention_backward(k, v, q, f, ckpt, dy, dST=None)
  y_t         = linear_attention_step(k_t, v_t, q_t, f_t, S)             # one decode step, S updated in place
  n, mu, r    = layer_norm(y, weight, bias)           # readout [B, H, T, V] -> normalised rows [B, T, H, V]
  grads       = layer_norm_backward(dn, y, weight, mu, r)

k and q may carry fewer heads than v (G dividing H: grouped k / q, head h
uses group h // (H // G)); dk and dq then have G heads too.  With
f_is_logit=True, f holds gate logits a_t (f_t = sigmoid(a_t), evaluated in
the kernels) and backward returns dL/da_t as df.

bf16 k/v/q/W select the tensor-core mode (M2RNN_MODE_BF16_TC); fp32 select
the fp32 debug mode; forward(..., fast_tanh=True) and forward(...,
mma_sync=True) select the forward-only alternatives.  Tensors must be
contiguous CUDA tensors with the head-first layouts of the header.

The default checkpoint stride, 8, is the longest chunk that the V = 64
tensor-core backward keeps in tensor memory for K = 64 and 128 (16 for
K = 32); longer strides (up to 16) run the general-shape backward.
"""
from __future__ import annotations

import functools
from typing import Dict, Optional, Tuple

import torch

from . import _lib
from ._lib import Dims, M2RNNError

_workspaces: Dict[Tuple[int, int], torch.Tensor] = {}

# Tokens between the states that linear_attention keeps for its backward.
LA_CHUNK = 128


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _mode(k: torch.Tensor) -> int:
    if k.dtype == torch.bfloat16:
        return _lib.MODE_BF16_TC
    if k.dtype == torch.float32:
        return _lib.MODE_FP32_DEBUG
    raise TypeError("k/v/q/W must be bfloat16 (tensor-core mode) or float32 (debug mode), got %s" % k.dtype)


def _check(name, t, shape, dtype, device):
    if t is None:
        return
    if not t.is_cuda or t.device != device:
        raise ValueError("%s must be a CUDA tensor on %s" % (name, device))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.dtype != dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def dims_of(k: torch.Tensor, v: torch.Tensor, ckpt_stride: int = 8, f_is_logit: bool = False) -> Dims:
    """Dims of a call: H from v, the k / q head groups G from k."""
    B, G, T, K = k.shape
    H = v.shape[1]
    if G < 1 or H % G != 0:
        if H > 0 or G > 0:
            raise ValueError("k has %d heads: it must have H = %d heads or a divisor of H" % (G, H))
    return Dims(B, H, T, K, v.shape[-1], _mode(k), ckpt_stride, G if G != H else 0, int(bool(f_is_logit)))


def _ws_key(device) -> Tuple[int, int]:
    """Workspaces are cached per (device, stream): calls that the library
    orders on one stream may share one, calls on different streams may
    overlap on the GPU and must not."""
    index = device.index if device.index is not None else torch.cuda.current_device()
    return index, _stream(torch.device("cuda", index))


def workspace(d: Dims, backward: bool, device) -> torch.Tensor:
    """Zero-initialised device workspace (cached per device and current
    stream, grown on demand)."""
    need = _lib.lib().m2rnn_workspace_size(d, 1 if backward else 0)
    if need == 0:
        raise M2RNNError(_lib.ERR_INVALID_ARG, "m2rnn_workspace_size")
    key = _ws_key(device)
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < need:
        ws = torch.zeros(need, dtype=torch.uint8, device=device)
        _workspaces[key] = ws
    return ws


def num_checkpoints(T: int, ckpt_stride: int) -> int:
    return (T + ckpt_stride - 1) // ckpt_stride


def forward(k, v, q, f, W, H0=None, *, ckpt_stride: int = 8, want_ckpt: bool = False,
            want_HT: bool = True, out: Optional[dict] = None, fast_tanh: bool = False,
            mma_sync: bool = False, f_is_logit: bool = False):
    """Runs the forward scan.  Returns (y, HT or None, ckpt or None).

    Two bf16-only alternatives to the default tensor-core forward:
    fast_tanh selects M2RNN_MODE_BF16_TC_FAST_TANH (the single-SFU
    tanh.approx.f32, for inference; its checkpoints are not meant for the
    backward); mma_sync selects M2RNN_MODE_BF16_MMA_SYNC (the register-resident
    forward for V = 64, K <= 64; its checkpoints feed the backward as usual)."""
    dev = k.device
    d = dims_of(k, v, ckpt_stride, f_is_logit)
    if fast_tanh or mma_sync:
        if d.mode != _lib.MODE_BF16_TC:
            raise TypeError("fast_tanh / mma_sync need bf16 inputs (the tensor-core mode)")
        if fast_tanh and mma_sync:
            raise ValueError("choose one of fast_tanh and mma_sync")
        d.mode = _lib.MODE_BF16_TC_FAST_TANH if fast_tanh else _lib.MODE_BF16_MMA_SYNC
    B, H, T, K, V = d.B, d.H, d.T, d.K, d.V
    lp = k.dtype
    G = d.qk_heads or H
    _check("k", k, (B, G, T, K), lp, dev)
    _check("v", v, (B, H, T, V), lp, dev)
    _check("q", q, (B, G, T, K), lp, dev)
    _check("f", f, (B, H, T), torch.float32, dev)
    _check("W", W, (H, V, V), lp, dev)
    _check("H0", H0, (B, H, K, V), torch.float32, dev)
    out = out or {}
    y = out.get("y")
    if y is None:
        y = torch.empty(B, H, T, V, dtype=torch.float32, device=dev)
    HT = out.get("HT") if want_HT else None
    if want_HT and HT is None:
        HT = torch.empty(B, H, K, V, dtype=torch.float32, device=dev)
    ckpt = out.get("ckpt") if want_ckpt else None
    if want_ckpt and ckpt is None:
        ckpt = torch.empty(B, H, num_checkpoints(T, ckpt_stride), K, V, dtype=torch.float32, device=dev)
    ws = workspace(d, False, dev)
    st = _lib.lib().m2rnn_forward(d, _ptr(k), _ptr(v), _ptr(q), _ptr(f), _ptr(W), _ptr(H0), _ptr(y), _ptr(HT),
                                  _ptr(ckpt), _ptr(ws), ws.numel(), _stream(dev))
    if st != _lib.OK:
        raise M2RNNError(st, "m2rnn_forward")
    return y, HT, ckpt


def step(k, v, q, f, W, H, *, y: Optional[torch.Tensor] = None, f_is_logit: bool = False):
    """One decode step, in place: advances the fp32 state H [B, H, K, V] by one
    step of the recurrence with k, q [B, H, K] (or [B, G, K], grouped), v
    [B, H, V] and f [B, H], and returns y [B, H, V].  It is the forward with
    T = 1 and the state buffer passed as both H0 and H_T (the ABI allows that
    alias), so T calls give the scan's outputs bit for bit."""
    B, _, K = k.shape
    Hh, V = v.shape[1], v.shape[-1]
    if H is None:
        raise ValueError("step needs the state buffer H (it is updated in place)")
    _check("H", H, (B, Hh, K, V), torch.float32, k.device)
    if y is None:
        y = torch.empty(B, Hh, V, dtype=torch.float32, device=k.device)
    forward(k.unsqueeze(2), v.unsqueeze(2), q.unsqueeze(2), f.unsqueeze(2), W, H, ckpt_stride=1,
            out={"y": y.view(B, Hh, 1, V), "HT": H}, f_is_logit=f_is_logit)
    return y


def backward(k, v, q, f, W, ckpt, dy, dHT=None, *, ckpt_stride: int = 8, out: Optional[dict] = None,
             f_is_logit: bool = False):
    """BPTT from the forward's checkpoints.  Returns dict dk, dv, dq, df, dW, dH0 (fp32)."""
    dev = k.device
    d = dims_of(k, v, ckpt_stride, f_is_logit)
    B, H, T, K, V = d.B, d.H, d.T, d.K, d.V
    lp = k.dtype
    G = d.qk_heads or H
    _check("k", k, (B, G, T, K), lp, dev)
    _check("v", v, (B, H, T, V), lp, dev)
    _check("q", q, (B, G, T, K), lp, dev)
    _check("f", f, (B, H, T), torch.float32, dev)
    _check("W", W, (H, V, V), lp, dev)
    _check("ckpt", ckpt, (B, H, num_checkpoints(T, ckpt_stride), K, V), torch.float32, dev)
    _check("dy", dy, (B, H, T, V), lp, dev)
    _check("dHT", dHT, (B, H, K, V), torch.float32, dev)
    out = dict(out or {})
    shapes = {"dk": (B, G, T, K), "dv": (B, H, T, V), "dq": (B, G, T, K), "df": (B, H, T),
              "dW": (H, V, V), "dH0": (B, H, K, V)}
    for n, s in shapes.items():
        if out.get(n) is None:
            out[n] = torch.empty(*s, dtype=torch.float32, device=dev)
    ws = workspace(d, True, dev)
    st = _lib.lib().m2rnn_backward(d, _ptr(k), _ptr(v), _ptr(q), _ptr(f), _ptr(W), _ptr(ckpt), _ptr(dy),
                                   _ptr(dHT), _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dq"]), _ptr(out["df"]),
                                   _ptr(out["dW"]), _ptr(out["dH0"]), _ptr(ws), ws.numel(), _stream(dev))
    if st != _lib.OK:
        raise M2RNNError(st, "m2rnn_backward")
    return out


def device_status(device=None) -> int:
    """Synchronises the current stream and returns (and clears) the device
    status of the workspace cached for that stream, and that of the
    linear-attention calls made on it or captured into graphs on this device.
    Returns at once where there are neither."""
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    key = _ws_key(dev)
    ws = _workspaces.get(key)
    st = _lib.OK if ws is None else _lib.lib().m2rnn_get_device_status(_ptr(ws), _stream(dev))
    with torch.cuda.device(dev):
        other = _lib.lib().m2rnn_linear_attention_status(_stream(dev))
    return st if st != _lib.OK else other


def set_wait_limit_ns(ns: int) -> None:
    _lib.lib().m2rnn_set_wait_limit_ns(int(ns))


def decay_logit_bias(H: int, tau_min: float = 2.0, tau_max: float = 256.0) -> torch.Tensor:
    """Per-head bias of the gate logit at initialisation, shape [H] (fp32, CPU).

    The pages parameterise the forget gate as f_t = ψ(x_t) in [0, 1] and start
    the heads with different decay rates (gist.science technical summary of
    "M²RNN", §2.1, forget gate), without giving the form.  This library's
    reading: ψ ends in the logistic function of a logit a_t = (projection of
    x_t) + b_h, and at initialisation, where the projection contributes about
    nothing, head h retains f_h = 1 / (1 + exp(-b_h)) of its state per step.
    The heads' retention times tau_h = 1 / (1 - f_h) are spaced geometrically
    from tau_min to tau_max steps, so b_h = log(tau_h - 1).  Pass logits built
    on it with f_is_logit=True."""
    if H < 1 or not (1.0 < tau_min <= tau_max):
        raise ValueError("need H >= 1 and 1 < tau_min <= tau_max")
    h = torch.arange(H, dtype=torch.float64)
    frac = h / (H - 1) if H > 1 else torch.zeros(1, dtype=torch.float64)
    tau = tau_min * (tau_max / tau_min) ** frac
    return torch.log(tau - 1.0).float()


# ------------------------------------------------------------------ linear attention

# What a call needs besides its tensors, by its shape and flags: the C dims and
# the bytes of workspace forward and backward.  (A decode step takes a few
# microseconds on the GPU; asking again each time costs as much on the host.)
_la_plans: Dict[tuple, tuple] = {}


def _la_plan(B, H, G, T, K, V, mode, f_is_logit, per_head):
    key = (B, H, G, T, K, V, mode, f_is_logit, per_head)
    plan = _la_plans.get(key)
    if plan is None:
        if G != H and (G < 1 or H % G != 0):
            raise ValueError("k has %d heads: it must have H = %d heads or a divisor of H" % (G, H))
        d = _lib.LaDims(B, H, T, K, V, mode, G if G != H else 0, int(f_is_logit), int(per_head))
        L = _lib.lib()
        plan = (d, L.m2rnn_linear_attention_workspace(d, 0), L.m2rnn_linear_attention_workspace(d, 1))
        if plan[1] == _lib.REFUSED:
            raise M2RNNError(_lib.ERR_UNSUPPORTED_SHAPE, "m2rnn_linear_attention (K = %d, V = %d)" % (K, V))
        if len(_la_plans) >= 4096:
            _la_plans.clear()
        _la_plans[key] = plan
    return plan


def _same(name, t, shape, dtype, device):
    """_check, in one expression where nothing is wrong."""
    if not (t.shape == shape and t.dtype is dtype and t.device == device and t.is_contiguous() and t.is_cuda):
        _check(name, t, shape, dtype, device)


def _out(out, name, like, shape, dtype):
    """The buffer out[name], checked, or a new one on like's device."""
    t = None if out is None else out.get(name)
    if t is None:
        return like.new_empty(shape, dtype=dtype)
    _same(name, t, shape, dtype, like.device)
    return t


def _scratch(need: int, like) -> Tuple[Optional[torch.Tensor], int]:
    """Workspace of one call and its address, from torch's allocator: calls on
    different streams, and captured graphs, never share one."""
    if not need:
        return None, 0
    t = like.new_empty(need, dtype=torch.uint8)
    return t, t.data_ptr()


# The current stream's handle and the current device by the calls beneath
# torch.cuda.current_stream and current_device, whose Python objects cost 3 us.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_raw_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call(what: str, device, fn, *args) -> None:
    """Calls the library on the device of the tensors, on its current stream."""
    index = device.index
    if index != _raw_device():
        with torch.cuda.device(device):
            st = fn(*args, _raw_stream(index))
    else:
        st = fn(*args, _raw_stream(index))
    if st != _lib.OK:
        raise M2RNNError(st, what)


def _la_inputs(k, v, q, f, S, f_is_logit, tokens):
    """Checks the inputs of a call (tokens: 4-dimensional k, q, v; else one
    token's, 3-dimensional) and gives its plan."""
    dims = 4 if tokens else 3
    if k.dim() != dims or v.dim() != dims:
        raise ValueError("k and v must have %d dimensions (batch, heads, %swidth), got %d and %d"
                         % (dims, "tokens, " if tokens else "", k.dim(), v.dim()))
    if tokens:
        B, G, T, K = k.shape
        _, H, _, V = v.shape
        vs, fs = (B, H, T, V), (B, H, T)
    else:
        B, G, K = k.shape
        _, H, V = v.shape
        T, vs, fs = 1, (B, H, V), (B, H)
    dev, lp = k.device, k.dtype
    mode = _mode(k)
    per_head = f.dim() == 1
    plan = _la_plan(B, H, G, T, K, V, mode, bool(f_is_logit), per_head)
    _same("k", k, k.shape, lp, dev)
    _same("v", v, vs, lp, dev)
    _same("q", q, k.shape, lp, dev)
    _same("f", f, (H,) if per_head else fs, torch.float32, dev)
    if S is not None:
        _same("S0", S, (B, H, K, V), torch.float32, dev)
    return plan, B, H, T, K, V


def linear_attention(k, v, q, f, S0=None, *, want_ST: bool = True, want_ckpt: bool = False,
                     f_is_logit: bool = False, out: Optional[dict] = None):
    """Linear attention with a decay for each head, over a whole sequence:
    S_t = f_t S_{t-1} + k_t v_tᵀ, y_t = S_tᵀ q_t.  Returns (y, ST or None, ckpt or None).
    (Unlike the M²RNN scan's, the input has no factor 1 - f_t: where it is wanted,
    v is scaled by it, and the sum of -v·dv over the last dimension added to df.)

    k, q [B, G, T, K] and v [B, H, T, V] (bf16, or fp32 for the debug mode),
    f [B, H, T] fp32 in [0, 1] (or logits, with f_is_logit) or [H], one
    constant for each head; S0 [B, H, K, V] fp32 (None: zeros).  y has the
    inputs' type, ST [B, H, K, V] is fp32.  ckpt [B, H, ceil(T/128), V/4, K, 4]
    holds the states that linear_attention_backward starts from (element (i, j)
    of a state at [j // 4, i, j % 4]).  `out` may hold buffers for y, ST and
    ckpt; ST may be S0's, and no other is an input's.  Padding holds finite values: a NaN in a bf16 token
    may reach the earlier tokens of its 128-token chunk too."""
    (d, need, _), B, H, T, K, V = _la_inputs(k, v, q, f, S0, f_is_logit, True)
    y = _out(out, "y", k, (B, H, T, V), k.dtype)
    ST = _out(out, "ST", k, (B, H, K, V), torch.float32) if want_ST else None
    ckpt = _out(out, "ckpt", k, (B, H, num_checkpoints(T, LA_CHUNK), V // 4, K, 4), torch.float32) if want_ckpt else None
    ws, wp = _scratch(need, k)
    _call("m2rnn_linear_attention_forward", k.device, _lib.lib().m2rnn_linear_attention_forward, d, k.data_ptr(),
          v.data_ptr(), q.data_ptr(), f.data_ptr(), _ptr(S0), y.data_ptr(), _ptr(ST), _ptr(ckpt), wp, need)
    return y, ST, ckpt


def linear_attention_step(k, v, q, f, S, *, ST: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                          f_is_logit: bool = False):
    """One decode step: advances the fp32 state S [B, H, K, V] by one token with
    k, q [B, G, K], v [B, H, V] and f [B, H] (or [H]), in place, or into ST
    where that is given.  Returns y [B, H, V]."""
    if S is None:
        raise ValueError("linear_attention_step needs the state buffer S")
    (d, need, _), B, H, _, K, V = _la_inputs(k, v, q, f, S, f_is_logit, False)
    if ST is None:
        ST = S
    else:
        _same("ST", ST, (B, H, K, V), torch.float32, k.device)
    if y is None:
        y = torch.empty_like(v)
    else:
        _same("y", y, (B, H, V), k.dtype, k.device)
    ws, wp = _scratch(need, k)
    _call("m2rnn_linear_attention_forward", k.device, _lib.lib().m2rnn_linear_attention_forward, d, k.data_ptr(),
          v.data_ptr(), q.data_ptr(), f.data_ptr(), S.data_ptr(), y.data_ptr(), ST.data_ptr(), None, wp, need)
    return y


def linear_attention_backward(k, v, q, f, ckpt, dy, dST=None, *, f_is_logit: bool = False,
                              out: Optional[dict] = None) -> dict:
    """Gradients of linear_attention from the checkpoints of its forward.
    Returns dict dk, dv, dq (the inputs' type), df (fp32, f's shape), dS0 (fp32).
    dk and dq of shared k and q are the sums over each group's heads."""
    (d, _, need), B, H, T, K, V = _la_inputs(k, v, q, f, None, f_is_logit, True)
    dev, lp = k.device, k.dtype
    _same("dy", dy, (B, H, T, V), lp, dev)
    if dST is not None:
        _same("dST", dST, (B, H, K, V), torch.float32, dev)
    if ckpt is None:
        raise ValueError("linear_attention_backward needs the checkpoints of linear_attention(..., want_ckpt=True)")
    _same("ckpt", ckpt, (B, H, num_checkpoints(T, LA_CHUNK), V // 4, K, 4), torch.float32, dev)
    g = dict(out or {})
    for n, shape, t in (("dk", k.shape, lp), ("dv", v.shape, lp), ("dq", k.shape, lp), ("df", f.shape, torch.float32),
                        ("dS0", (B, H, K, V), torch.float32)):
        g[n] = _out(g, n, k, shape, t)
    ws, wp = _scratch(need, k)
    _call("m2rnn_linear_attention_backward", dev, _lib.lib().m2rnn_linear_attention_backward, d, k.data_ptr(),
          v.data_ptr(), q.data_ptr(), f.data_ptr(), ckpt.data_ptr(), dy.data_ptr(), _ptr(dST), g["dk"].data_ptr(),
          g["dv"].data_ptr(), g["dq"].data_ptr(), g["df"].data_ptr(), g["dS0"].data_ptr(), wp, need)
    return g


# ------------------------------------------------------------------ layer norm

_NORM_TYPES = {torch.bfloat16: 0, torch.float32: 1}


@functools.lru_cache(maxsize=4096)
def _norm_dims(*fields):
    """The C dims of a shape: making them anew costs 1 us a call."""
    return _lib.NormDims(*fields)


def _norm_shape(x, weight, bias, heads=None):
    """(B, H, T, N) of a call, and whether x is a head-first readout: by the
    weight (or bias), or where there is none by `heads`."""
    first = weight if weight is not None else bias
    if first is not None:
        if heads is not None and bool(heads) != (first.dim() == 2):
            raise ValueError("heads=%s contradicts a weight of %d dimensions" % (bool(heads), first.dim()))
        heads = first.dim() == 2
    if x.dtype not in _NORM_TYPES:
        raise TypeError("x must be bfloat16 or float32, got %s" % x.dtype)
    if heads:
        if x.dim() != 4:
            raise ValueError("a norm with one weight per head%s takes x [B, H, T, N], got %d dimensions"
                             % (" (heads=True)" if first is None else "", x.dim()))
        B, H, T, N = x.shape
    else:
        if x.dim() < 1:
            raise ValueError("x must have at least one dimension")
        N = x.shape[-1]
        B, H, T = 1, 1, x.numel() // N if N else 0
    if N < 1:
        raise ValueError("the last dimension of x is empty")
    if T > 1 << 30:
        raise ValueError("x has %d rows: at most 2^30 in one call" % T)
    dev = x.device
    _same("x", x, x.shape, x.dtype, dev)
    ps = (H, N) if heads else (N,)
    if weight is not None:
        _same("weight", weight, ps, torch.float32, dev)
    if bias is not None:
        _same("bias", bias, ps, torch.float32, dev)
    return B, H, T, N, bool(heads)


def layer_norm(x, weight=None, bias=None, *, eps: float = 1e-5, rms: bool = False,
               out_dtype: Optional[torch.dtype] = None, out: Optional[dict] = None):
    """Layer norm over the last dimension (with rms=True, its RMS form).
    Returns (y, mean, rstd); mean is None with rms=True.

    weight and bias [H, N] (fp32): x is a readout [B, H, T, N] as forward and
    linear_attention give it, normalised per head, and y is token-first,
    [B, T, H, N]: the rows of the output projection.  weight and bias [N] or
    None: plain rows, y has x's shape.  x is bf16 or fp32; y has type out_dtype
    (x's by default).  mean and rstd (fp32, x's leading shape) feed
    layer_norm_backward.  `out` may hold buffers for y, mean and rstd (none of
    them x's)."""
    B, H, T, N, heads = _norm_shape(x, weight, bias)
    yt = x.dtype if out_dtype is None else out_dtype
    if yt not in _NORM_TYPES:
        raise TypeError("out_dtype must be bfloat16 or float32, got %s" % yt)
    lead = x.shape[:-1]
    y = _out(out, "y", x, (B, T, H, N) if heads else x.shape, yt)
    rstd = _out(out, "rstd", x, lead, torch.float32)
    mean = None if rms else _out(out, "mean", x, lead, torch.float32)
    d = _norm_dims(B, H, T, N, _NORM_TYPES[x.dtype], _NORM_TYPES[yt], 0, 1 if rms else 0, float(eps))
    _call("m2rnn_layer_norm_forward", x.device, _lib.lib().m2rnn_layer_norm_forward, d, x.data_ptr(), _ptr(weight),
          _ptr(bias), y.data_ptr(), _ptr(mean), rstd.data_ptr())
    return y, mean, rstd


def layer_norm_backward(dy, x, weight, mean, rstd, *, rms: bool = False, heads: Optional[bool] = None,
                        dx_dtype: Optional[torch.dtype] = None, out: Optional[dict] = None) -> dict:
    """Gradients of layer_norm: dict dx (x's shape; type dx_dtype, x's by
    default), dweight and dbias (fp32, in weight's shape).  dy has y's shape
    and type.  With weight=None, `heads` says which form x was in: a readout
    with dy [B, T, H, N] (True), or plain rows (False, and what None takes
    unless dy's shape fits both)."""
    if weight is None and heads is None and x.dim() == 4 and x.shape[1] == x.shape[2] > 1:
        raise ValueError("without a weight, x of shape %s may be a readout or plain rows: say which with heads=True "
                         "or heads=False" % (tuple(x.shape),))
    B, H, T, N, per_head = _norm_shape(x, weight, None, heads)
    dev = x.device
    dt = x.dtype if dx_dtype is None else dx_dtype
    if dy.dtype not in _NORM_TYPES or dt not in _NORM_TYPES or (dt == torch.float32 and x.dtype != torch.float32):
        raise TypeError("dy must be bfloat16 or float32 and dx bfloat16 or x's type, got %s and %s" % (dy.dtype, dt))
    _same("dy", dy, (B, T, H, N) if per_head else x.shape, dy.dtype, dev)
    lead = x.shape[:-1]
    if rstd is None or (mean is None and not rms):
        raise ValueError("layer_norm_backward needs the forward's rstd, and its mean unless rms=True")
    _same("rstd", rstd, lead, torch.float32, dev)
    if not rms:
        _same("mean", mean, lead, torch.float32, dev)
    g = dict(out or {})
    shape = (H, N) if per_head else (N,)
    for n, sh, t in (("dx", x.shape, dt), ("dweight", shape, torch.float32), ("dbias", shape, torch.float32)):
        g[n] = _out(g, n, x, sh, t)
    d = _norm_dims(B, H, T, N, _NORM_TYPES[x.dtype], _NORM_TYPES[dy.dtype], _NORM_TYPES[dt], 1 if rms else 0, 0.0)
    L = _lib.lib()
    need = L.m2rnn_layer_norm_workspace(d)
    if need == _lib.REFUSED:
        raise M2RNNError(_lib.ERR_UNSUPPORTED_SHAPE, "m2rnn_layer_norm_backward")
    ws, wp = _scratch(need, x)
    _call("m2rnn_layer_norm_backward", dev, L.m2rnn_layer_norm_backward, d, dy.data_ptr(), x.data_ptr(), _ptr(weight),
          None if rms else mean.data_ptr(), rstd.data_ptr(), g["dx"].data_ptr(), g["dweight"].data_ptr(),
          g["dbias"].data_ptr(), wp, need)
    return g
