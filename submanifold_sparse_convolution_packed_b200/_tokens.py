"""Binding of the token-wise layers of include/smc.h: layer norm, rotary
positions, attention.  As in ``_binding``: argument checks and pointers only,
every step runs in the library's kernels, and there is no fallback.  None of the
calls is recorded by autograd: results never require gradients, and the
gradients are calls of their own."""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Sequence, Tuple

import torch

from . import _binding
from ._binding import _DTYPES, ACTS, _check

# The current stream's handle and the current device without the Python objects
# around them: those took 8 of a small call's 25 microseconds on the host.
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device

ROTARY_LAYOUTS = {"interleaved": 0, "half": 1}


def lib() -> ctypes.CDLL:
    return _binding._lib or _binding.lib()


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _device_of(first: torch.Tensor, *others: Optional[torch.Tensor]) -> int:
    d = first.get_device()
    for t in others:
        if t is not None and t.get_device() != d:
            d = -1
    if d < 0:
        raise ValueError("all tensors must be on one CUDA device")
    return d


def _act(act: Optional[str]) -> int:
    if act not in ACTS:
        raise ValueError(f"act must be one of {list(ACTS)}")
    return ACTS[act]


def _result(out: Optional[torch.Tensor], shape, dtype, device, what: str, dense: bool = True) -> torch.Tensor:
    """`out`, checked, or a new tensor."""
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if tuple(out.shape) != tuple(shape) or out.dtype != dtype:
        raise ValueError(f"{what} must be {list(shape)} of {dtype}")
    if dense and not out.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if not dense and out.dim() and out.shape[-1] > 1 and out.stride(-1) != 1:
        raise ValueError(f"{what} must be dense along its last axis")
    return out


def _last_dense(t: torch.Tensor) -> torch.Tensor:
    return t if t.is_contiguous() or t.shape[-1] <= 1 or t.stride(-1) == 1 else t.contiguous()


_Two = ctypes.c_int64 * 2


def _strides(t: torch.Tensor):
    """Of rows and heads; None (dense) spares the conversion."""
    if t.is_contiguous():
        return None
    s = t.stride()
    return _Two(s[0], s[1])


class _On:
    """Makes a device and a stream the current ones: the stream then owns the
    tensors made inside, as the caching allocator needs.  Calls on the current
    device and stream go without (a switch takes longer than a launch).  A
    stream of another device is refused: the call would leave it for the
    tensors' own."""

    def __init__(self, device: int, stream):
        if stream is not None and stream.device.index != device:
            raise ValueError("stream must belong to the tensors' device")
        self.inner = [torch.cuda.device(device)]
        if stream is not None:
            self.inner.append(torch.cuda.stream(stream))

    def __enter__(self):
        for c in self.inner:
            c.__enter__()

    def __exit__(self, *error):
        for c in reversed(self.inner):
            c.__exit__(*error)


def layer_norm(x: torch.Tensor, gamma: Optional[torch.Tensor] = None, beta: Optional[torch.Tensor] = None,
               eps: float = 1e-5, act: Optional[str] = None, out: Optional[torch.Tensor] = None,
               stats: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """act(gamma * (x - mean) * rstd + beta) over each row's channels
    (smc_layer_norm): x [N, C], gamma / beta [C] of x's dtype or None, act in
    {None, "relu", "silu"}.  `out` may be x.  `stats` (float32 [N, 2]), if
    given, receives (mean, rstd), which layer_norm_backward takes."""
    if x.dtype not in _DTYPES or x.dim() != 2:
        raise TypeError("x must be a 2-D float32 / bfloat16 / float16 tensor")
    a = _act(act)
    n, c = x.shape
    for t in (gamma, beta):
        if t is not None and (t.dtype != x.dtype or t.shape != (c,)):
            raise ValueError("gamma and beta must be [C] of the x dtype")
    if stats is not None:
        _result(stats, (n, 2), torch.float32, x.device, "stats")
    if out is not None:
        _result(out, (n, c), x.dtype, x.device, "out")
        if out.data_ptr() == x.data_ptr() and not x.is_contiguous():
            raise ValueError("out may be x only if x is contiguous")
    dev = _device_of(x, gamma, beta, out, stats)
    if stream is not None or dev != _current_device():
        with _On(dev, stream):
            return layer_norm(x, gamma, beta, eps, act, out, stats)
    x = x.contiguous()
    gamma, beta = gamma if gamma is None else gamma.contiguous(), beta if beta is None else beta.contiguous()
    if out is None:
        out = torch.empty_like(x)
    _check(lib().smc_layer_norm(x.data_ptr(), n, c, _ptr(gamma), _ptr(beta), eps, a, out.data_ptr(), _ptr(stats),
                                _DTYPES[x.dtype], _current_stream(dev)), "smc_layer_norm")
    return out


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, stats: torch.Tensor, gamma: Optional[torch.Tensor] = None,
                        beta: Optional[torch.Tensor] = None, act: Optional[str] = None,
                        dx: Optional[torch.Tensor] = None, dgamma: Optional[torch.Tensor] = None,
                        dbeta: Optional[torch.Tensor] = None, stream=None
                        ) -> Tuple[torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Gradients of layer_norm (smc_layer_norm_backward): (dx, dgamma, dbeta)
    for dy [N, C], with the forward call's x, stats, gamma, beta and act.
    dgamma / dbeta are None where gamma / beta are (unless buffers for them
    are given).  dx may be dy or x.  Deterministic."""
    if x.dtype not in _DTYPES or x.dim() != 2:
        raise TypeError("x must be a 2-D float32 / bfloat16 / float16 tensor")
    a = _act(act)
    n, c = x.shape
    if dy.shape != x.shape or dy.dtype != x.dtype:
        raise ValueError("dy must be [N, C] of the x dtype")
    if stats.shape != (n, 2) or stats.dtype != torch.float32:
        raise ValueError("stats must be the forward call's float32 [N, 2]")
    for t in (gamma, beta):
        if t is not None and (t.dtype != x.dtype or t.shape != (c,)):
            raise ValueError("gamma and beta must be [C] of the x dtype")
    if dx is not None:
        _result(dx, (n, c), x.dtype, x.device, "dx")
        for t in (x, dy):
            if dx.data_ptr() == t.data_ptr() and not t.is_contiguous():
                raise ValueError("dx may be x or dy only if that is contiguous")
    for t, what in ((dgamma, "dgamma"), (dbeta, "dbeta")):
        if t is not None:
            _result(t, (c,), x.dtype, x.device, what)
    dev = _device_of(x, dy, stats, gamma, beta, dx, dgamma, dbeta)
    if stream is not None or dev != _current_device():
        with _On(dev, stream):
            return layer_norm_backward(dy, x, stats, gamma, beta, act, dx, dgamma, dbeta)
    dy, x, stats = dy.contiguous(), x.contiguous(), stats.contiguous()
    gamma, beta = gamma if gamma is None else gamma.contiguous(), beta if beta is None else beta.contiguous()
    if dx is None:
        dx = torch.empty_like(x)
    if dgamma is None and gamma is not None:
        dgamma = torch.empty_like(gamma)
    if dbeta is None and beta is not None:
        dbeta = torch.empty_like(beta)
    _check(lib().smc_layer_norm_backward(dy.data_ptr(), x.data_ptr(), n, c, stats.data_ptr(), _ptr(gamma), _ptr(beta),
                                         a, dx.data_ptr(), _ptr(dgamma), _ptr(dbeta), _DTYPES[x.dtype],
                                         _current_stream(dev)), "smc_layer_norm_backward")
    return dx, dgamma, dbeta


def rotary_freqs(pairs: int, axes: int = 1, base: float = 10000.0, factor: float = 1.0, scaling: str = "linear",
                 original: Optional[int] = None, device=None) -> Tuple[torch.Tensor, float]:
    """Frequencies for rotary: (float64 [axes, pairs], scale), f_i =
    base^(-i / pairs) on every axis, stretched to `factor` times the length:

    * "linear": every frequency divided by factor;
    * "ntk": the base raised to base * factor^(pairs / (pairs - 1)), which
      keeps the fastest pair and divides the slowest by factor;
    * "yarn": pairs up to the last that turns 32 times or more over the
      `original` length (or the first pair) keep their frequency, those from
      the first place at one turn or less on are divided by factor, a linear
      ramp in the pair index between, also where no pair is that slow;
      scale = 0.1 ln(factor) + 1.
    """
    if pairs < 1 or axes < 1 or not base > 1.0 or not factor >= 1.0:
        raise ValueError("need pairs >= 1, axes >= 1, base > 1 and factor >= 1")
    if scaling not in ("linear", "ntk", "yarn"):
        raise ValueError("scaling must be 'linear', 'ntk' or 'yarn'")
    scale = 1.0
    i = torch.arange(pairs, dtype=torch.float64)
    if scaling == "ntk" and pairs > 1:
        base = base * factor ** (pairs / (pairs - 1))
    f = base ** (-i / pairs)
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        if not original or original < 1:
            raise ValueError("yarn needs the original length")

        def index(turns):  # the place, whole or not, of a pair that turns this often over the original length
            return pairs * math.log(original / (turns * 2 * math.pi)) / math.log(base)

        # hi may lie behind the last pair; before the first, every pair turns less than once
        lo, hi = max(math.floor(index(32.0)), 0), math.ceil(index(1.0))
        stretch = ((i - lo) / (hi - lo)).clamp(0.0, 1.0) if hi > lo else torch.ones_like(i)
        f = f * (1 - stretch) + f / factor * stretch
        scale = 0.1 * math.log(factor) + 1.0
    return f.expand(axes, -1).contiguous().to(device), scale


def rotary(x: torch.Tensor, positions: torch.Tensor, freqs: torch.Tensor, layout: str = "interleaved",
           scale: float = 1.0, inverse: bool = False, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Rotary positions (smc_rotary): x [N, H, D] turned by positions [N, A]
    (int32; e.g. ``coords[:, 1:]``, any strides) times freqs (float64 [A, F],
    see rotary_freqs); layout "interleaved" or "half" over the first 2 A F
    channels of each head.  inverse=True is the gradient.  x may be a view
    (a slice of a packed projection); `out` may be x."""
    if x.dtype not in _DTYPES or x.dim() != 3:
        raise TypeError("x must be a 3-D float32 / bfloat16 / float16 tensor [N, H, D]")
    if layout not in ROTARY_LAYOUTS:
        raise ValueError(f"layout must be one of {list(ROTARY_LAYOUTS)}")
    n, h, d = x.shape
    if positions.dtype != torch.int32 or positions.dim() != 2 or positions.shape[0] != n:
        raise ValueError("positions must be int32 [N, axes]")
    if freqs.dtype != torch.float64 or freqs.dim() != 2 or freqs.shape[0] != positions.shape[1]:
        raise ValueError("freqs must be float64 [axes, F]")
    if h < 1 or freqs.numel() < 1 or 2 * freqs.numel() > d:
        raise ValueError("freqs must hold 1 to D / 2 pairs")
    if out is not None:
        _result(out, (n, h, d), x.dtype, x.device, "out", dense=False)
        if out.data_ptr() == x.data_ptr() and d > 1 and x.stride(-1) != 1:
            raise ValueError("out may be x only if x is dense along its last axis")
    dev = _device_of(x, positions, freqs, out)
    if stream is not None or dev != _current_device():
        with _On(dev, stream):
            return rotary(x, positions, freqs, layout, scale, inverse, out)
    x, freqs = _last_dense(x), freqs.contiguous()
    if out is None:
        out = x.new_empty((n, h, d))
    axes, f = freqs.shape
    _check(lib().smc_rotary(x.data_ptr(), _strides(x), n, h, d, positions.data_ptr(), _strides(positions),
                            freqs.data_ptr(), axes, f, ROTARY_LAYOUTS[layout], scale, 1 if inverse else 0,
                            out.data_ptr(), _strides(out), _DTYPES[x.dtype], _current_stream(dev)), "smc_rotary")
    return out


def _attention_sizes(q, k, v, offsets, k_offsets, scale):
    """The checked sizes (n, h, d, m, hk, items), k_offsets and scale."""
    dtype = q.dtype
    if dtype not in _DTYPES or q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise TypeError("q, k and v must be 3-D float32 / bfloat16 / float16 tensors [rows, heads, dim]")
    if k.dtype != dtype or v.dtype != dtype:
        raise TypeError("q, k and v must share one dtype")
    n, h, d = q.shape
    m, hk, dk = ks = k.shape
    if v.shape != ks or dk != d:
        raise ValueError("k and v must be [M, kv_heads, D] with q's D")
    if d < 1:
        raise ValueError("a head must have channels")
    if h < 1 or hk < 1 or h % hk != 0:
        raise ValueError("the heads of q must be a multiple of those of k and v")
    if k_offsets is None:
        if m != n:
            raise ValueError("k_offsets are needed where k has other rows than q")
        k_offsets = offsets
    for o in (offsets,) if k_offsets is offsets else (offsets, k_offsets):
        if o.dtype != torch.int32 or o.dim() != 1 or o.shape[0] < 1 or o.shape != offsets.shape:
            raise ValueError("offsets must be int32 [items + 1], the same items for q and k")
    if scale is None:
        scale = d ** -0.5
    if not (0.0 < scale < math.inf):
        raise ValueError("scale must be positive and finite")
    return (n, h, d, m, hk, offsets.shape[0] - 1), k_offsets, float(scale)


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, offsets: torch.Tensor,
              k_offsets: Optional[torch.Tensor] = None, scale: Optional[float] = None, causal: bool = False,
              out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention within each item (smc_attention): q [N, H, D], k / v
    [M, Hkv, D] (views are fine, H a multiple of Hkv, D <= 128), `offsets`
    int32 [items + 1] row bounds on the device, `k_offsets` those of the keys
    where they differ.  For rows in item order,
    ``torch.searchsorted(coords[:, 0].contiguous(), torch.arange(batch + 1,
    dtype=torch.int32, device=coords.device), out_int32=True)`` gives them.
    scale defaults to D ** -0.5; causal lets the last query see every key.
    `lse` (float32 [N, H]), if given, receives the log sum of exponentials,
    which attention_backward takes.  A query without keys gets zeros; rows
    outside every item are left as they were (unset in a new tensor).
    bf16 / fp16 run on the tensor cores where D is a multiple of 8, every tensor
    starts on 16 bytes and the strides are positive multiples of 8 (one k or v head
    expanded to all is not: give its dense copy, or fewer kv_heads); anything else
    is right, but about 24 times slower over long items."""
    (n, h, d, m, hk, items), k_offsets, scale = _attention_sizes(q, k, v, offsets, k_offsets, scale)
    if out is not None:
        _result(out, (n, h, d), q.dtype, q.device, "out")
    if lse is not None:
        _result(lse, (n, h), torch.float32, q.device, "lse")
    dev = _device_of(q, k, v, offsets, k_offsets, out, lse)
    if stream is not None or dev != _current_device():
        with _On(dev, stream):
            return attention(q, k, v, offsets, k_offsets, scale, causal, out, lse)
    q, k, v = _last_dense(q), _last_dense(k), _last_dense(v)
    offsets, k_offsets = offsets.contiguous(), k_offsets.contiguous()
    if out is None:
        out = q.new_empty((n, h, d))
    _check(lib().smc_attention(q.data_ptr(), _strides(q), k.data_ptr(), _strides(k), v.data_ptr(), _strides(v),
                               offsets.data_ptr(), k_offsets.data_ptr(), items, n, m, h, hk, d, scale,
                               1 if causal else 0, out.data_ptr(), _ptr(lse), _DTYPES[q.dtype], _current_stream(dev)),
           "smc_attention")
    return out


def attention_backward(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                       lse: torch.Tensor, offsets: torch.Tensor, k_offsets: Optional[torch.Tensor] = None,
                       scale: Optional[float] = None, causal: bool = False, dq: Optional[torch.Tensor] = None,
                       dk: Optional[torch.Tensor] = None, dv: Optional[torch.Tensor] = None, stream=None
                       ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Gradients of attention (smc_attention_backward): (dq, dk, dv) for dout
    [N, H, D], with the forward call's arguments, its out and its lse.  The
    gradients of shared key/value heads are summed.  dq, dk, dv may be given,
    also as views of one packed buffer.  Deterministic.  The tensor cores take the
    shapes that attention names, dout and the gradients included."""
    (n, h, d, m, hk, items), k_offsets, scale = _attention_sizes(q, k, v, offsets, k_offsets, scale)
    if dout.shape != q.shape or dout.dtype != q.dtype or out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("dout and out must be [N, H, D] of q's dtype")
    if lse.shape != (n, h) or lse.dtype != torch.float32:
        raise ValueError("lse must be the forward call's float32 [N, H]")
    shapes = ((dq, (n, h, d), "dq"), (dk, (m, hk, d), "dk"), (dv, (m, hk, d), "dv"))
    for t, shape, what in shapes:
        if t is not None:
            _result(t, shape, q.dtype, q.device, what, dense=False)
    dev = _device_of(q, k, v, dout, out, lse, offsets, k_offsets, dq, dk, dv)
    if stream is not None or dev != _current_device():
        with _On(dev, stream):
            return attention_backward(dout, q, k, v, out, lse, offsets, k_offsets, scale, causal, dq, dk, dv)
    q, k, v, dout = _last_dense(q), _last_dense(k), _last_dense(v), _last_dense(dout)
    out, lse = out.contiguous(), lse.contiguous()
    offsets, k_offsets = offsets.contiguous(), k_offsets.contiguous()
    if dq is None:
        dq = q.new_empty((n, h, d))
    if dk is None:
        dk = q.new_empty((m, hk, d))
    if dv is None:
        dv = q.new_empty((m, hk, d))
    _check(lib().smc_attention_backward(dout.data_ptr(), _strides(dout), q.data_ptr(), _strides(q), k.data_ptr(),
                                        _strides(k), v.data_ptr(), _strides(v), out.data_ptr(), lse.data_ptr(),
                                        offsets.data_ptr(), k_offsets.data_ptr(), items, n, m, h, hk, d, scale,
                                        1 if causal else 0, dq.data_ptr(), _strides(dq), dk.data_ptr(), _strides(dk),
                                        dv.data_ptr(), _strides(dv), _DTYPES[q.dtype], _current_stream(dev)),
           "smc_attention_backward")
    return dq, dk, dv
