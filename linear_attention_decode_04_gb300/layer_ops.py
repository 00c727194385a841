"""Python binding of the operators between and behind the layers of a serving
step:

- ``kda_add_norm`` (``include/kda_add_norm.h``): addition to the residual
  stream, root-mean-square norm, output in bf16 and in 8 bits with row scales;
- ``kda_linear`` (``include/kda_linear.h``): matrix products of bf16 or 8-bit
  rows with scales, bias, activation and residual in the epilogue;
- ``kda_logprobs`` (``include/kda_logprobs.h``): log probabilities of given
  tokens, entropy and the likeliest alternatives.

Prepared calls and functions as in ``step_ops``.
"""
from __future__ import annotations

import ctypes

import torch

from .binding import _check, _dense, _rows
from .step_ops import _Args, _Call, _err, _p, _shaped

KDA_ADD_NORM_NO_NORM = 1
ADD_NORM_MAX_D = 32768
KDA_LINEAR_E4M3, KDA_LINEAR_OUT_F32, KDA_LINEAR_EARLY_WEIGHT = 1, 2, 4
ACTIVATIONS = {None: 0, "silu": 1, "gelu": 2, "silu_gated": 3}
KDA_LOGPROBS_BF16 = 1
LOGPROBS_MAX_TOP = 32

_i32, _i64, _u32, _f32, _ptr = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_float, ctypes.c_void_p


class KdaAddNormArgs(_Args):
    """Mirror of ``KdaAddNormArgs`` (field order and types must match)."""
    _fields_ = [("struct_size", _u32), ("T", _i32), ("D", _i32), ("flags", _u32), ("eps", _f32), ("x", _ptr),
                ("x_row_stride", _i64), ("residual", _ptr), ("residual_row_stride", _i64), ("weight", _ptr),
                ("residual_out", _ptr), ("residual_out_row_stride", _i64), ("out", _ptr), ("out_row_stride", _i64),
                ("out_q", _ptr), ("out_q_row_stride", _i64), ("out_scale", _ptr)]


class KdaLinearArgs(_Args):
    """Mirror of ``KdaLinearArgs``."""
    _fields_ = [("struct_size", _u32), ("M", _i32), ("N", _i32), ("K", _i32), ("activation", _i32), ("flags", _u32),
                ("x", _ptr), ("x_row_stride", _i64), ("weight", _ptr), ("weight_row_stride", _i64), ("x_scale", _ptr),
                ("weight_scale", _ptr), ("bias", _ptr), ("residual", _ptr), ("residual_row_stride", _i64),
                ("out", _ptr), ("out_row_stride", _i64), ("err_flag", _ptr)]


class KdaLogprobsArgs(_Args):
    """Mirror of ``KdaLogprobsArgs``."""
    _fields_ = [("struct_size", _u32), ("R", _i32), ("V", _i32), ("num_top", _i32), ("flags", _u32), ("logits", _ptr),
                ("logits_row_stride", _i64), ("tokens", _ptr), ("logprobs", _ptr), ("ranks", _ptr), ("entropy", _ptr),
                ("top_ids", _ptr), ("top_logprobs", _ptr), ("err_flag", _ptr)]


def _span(t: torch.Tensor) -> tuple[int, int]:
    """First byte and end of the memory that a row-strided tensor's elements lie in."""
    n = 1 + sum((s - 1) * st for s, st in zip(t.shape, t.stride())) if t.numel() else 0
    return t.data_ptr(), t.data_ptr() + n * t.element_size()


def _apart(result: torch.Tensor, name: str, other: torch.Tensor | None, other_name: str):
    """Refuses a result whose memory interleaves with another tensor's.  (Columns of the same wider rows are apart:
    they have one row stride, and their columns do not meet.)"""
    if other is None or not result.numel() or not other.numel():
        return
    (a, b), (c, d) = _span(result), _span(other)
    if b <= c or d <= a:
        return
    if result.dim() == 2 and other.dim() == 2:
        pitch = result.stride(0) * result.element_size()
        wide = result.shape[1] * result.element_size(), other.shape[1] * other.element_size()
        if pitch == other.stride(0) * other.element_size():
            off = (c - a) % pitch
            if off >= wide[0] and off + wide[1] <= pitch:
                return
    raise ValueError(f"{name} overlaps {other_name}")


def _same_place(a: torch.Tensor | None, b: torch.Tensor | None) -> bool:
    return (a is not None and b is not None and a.data_ptr() == b.data_ptr() and a.dtype == b.dtype
            and a.shape == b.shape and a.stride() == b.stride())


# ------------------------------------------------------------- norm with residual
class KdaAddNormCall(_Call):
    """A prepared ``kda_add_norm`` call: h = x + residual, y = h / rms(h) *
    weight.

      x            bf16 [T, D] (rows may be strided, as all rows here)
      residual     bf16 [T, D] or None
      weight       fp32 [D] or None (ones)
      residual_out bf16 [T, D] or None: h; may be ``residual`` or ``x`` itself
      out          bf16 [T, D] or None: y; may be ``x`` or ``residual`` itself
      out_q, out_scale  float8_e4m3fn [T, D] and fp32 [T], or None: y in 8
                   bits, with the scale of each row, as ``kda_linear`` takes it
      norm         False leaves the norm out (y = h): 8-bit rows of what a
                   layer gives"""

    def __init__(self, x, *, weight=None, residual=None, residual_out=None, out=None, out_q=None, out_scale=None,
                 eps: float = 1e-6, norm: bool = True):
        _check(x, "x", torch.bfloat16, None)
        if x.dim() != 2:
            raise ValueError(f"x must be [T, D] (got {tuple(x.shape)})")
        dev, (T, D) = x.device, x.shape
        if D < 8 or D % 8 or D > ADD_NORM_MAX_D:
            raise ValueError(f"D must be a multiple of 8 up to {ADD_NORM_MAX_D} (got {D})")
        if not norm and weight is not None:
            raise ValueError("weight without the norm")
        if (out_q is None) != (out_scale is None):
            raise ValueError("out_q and out_scale go together")
        if out is None and out_q is None and residual_out is None:
            raise ValueError("a result is needed: residual_out, out, or out_q with out_scale")
        rows = lambda t, name: _rows(t, name, T, D) if T > 1 else D * (_rows(t, name, T, D) > 0)  # noqa: E731
        strides = {"x": rows(x, "x")}
        tensors = dict(residual=residual, residual_out=residual_out, out=out, out_q=out_q)
        for name, t in tensors.items():
            if t is not None:
                _check(t, name, torch.float8_e4m3fn if name == "out_q" else torch.bfloat16, dev)
                strides[name] = rows(t, name)
                if t.shape[1] != D:
                    raise ValueError(f"{name} must be [{T}, {D}] (got {tuple(t.shape)})")
        if weight is not None:
            _shaped(weight, "weight", torch.float32, dev, (D,))
        if out_scale is not None:
            _shaped(out_scale, "out_scale", torch.float32, dev, (T,))
        results = [(n, t) for n, t in (("residual_out", residual_out), ("out", out), ("out_q", out_q),
                                       ("out_scale", out_scale)) if t is not None]
        for i, (name, t) in enumerate(results):
            for other_name, other in (("x", x), ("residual", residual)):
                if not _same_place(t, other):
                    _apart(t, name, other, other_name)
            _apart(t, name, weight, "weight")
            for other_name, other in results[:i]:
                _apart(t, name, other, other_name)
        s = lambda name: strides.get(name, 0)  # noqa: E731
        args = KdaAddNormArgs(
            T=T, D=D, flags=0 if norm else KDA_ADD_NORM_NO_NORM, eps=float(eps), x=_p(x), x_row_stride=s("x"),
            residual=_p(residual), residual_row_stride=s("residual"), weight=_p(weight),
            residual_out=_p(residual_out), residual_out_row_stride=s("residual_out"), out=_p(out),
            out_row_stride=s("out"), out_q=_p(out_q), out_q_row_stride=s("out_q"), out_scale=_p(out_scale))
        self._prepare("kda_add_norm", args, dev, (x, weight, residual, residual_out, out, out_q, out_scale))


def kda_add_norm(x, *, weight=None, residual=None, residual_out=None, out=None, out_q=None, out_scale=None,
                 eps: float = 1e-6, norm: bool = True, stream: torch.cuda.Stream | None = None) -> None:
    """Residual addition, root-mean-square norm, and output in bf16 and / or 8
    bits (see ``KdaAddNormCall``)."""
    KdaAddNormCall(x, weight=weight, residual=residual, residual_out=residual_out, out=out, out_q=out_q,
                   out_scale=out_scale, eps=eps, norm=norm)(stream)


# ----------------------------------------------------------------- matrix products
class KdaLinearCall(_Call):
    """A prepared ``kda_linear`` call: out = act(x @ weight^T * scales + bias) +
    residual.

      x            [M, K] bf16, or float8_e4m3fn with x_scale fp32 [M]
      weight       [N, K] of the same type, float8_e4m3fn with weight_scale
                   fp32 [N]; rows of x and weight may be strided, by multiples
                   of 16 bytes
      out          bf16 or fp32 [M, N] ([M, N / 2] gated); rows may be strided
      bias         fp32 [N] or None
      residual     bf16, of out's shape, or None; may be ``out`` itself
      activation   None, "silu", "gelu", or "silu_gated" (silu of the first
                   half of the N channels times the second)
      early_weight weight, its scale and bias are not written by the kernel
                   directly ahead of the call in its stream: the call may
                   read them while that still runs (not before whatever is
                   ahead of that kernel has ended)"""

    def __init__(self, x, weight, out, *, x_scale=None, weight_scale=None, bias=None, residual=None,
                 activation: str | None = None, early_weight: bool = False, err_flag=None):
        if activation not in ACTIVATIONS:
            raise ValueError(f"activation must be one of {tuple(ACTIVATIONS)} (got {activation!r})")
        if not isinstance(x, torch.Tensor) or x.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
            raise TypeError("x must be a bfloat16 or float8_e4m3fn tensor")
        dev, dt = x.device, x.dtype
        _check(x, "x", dt, None)
        _check(weight, "weight", dt, dev)
        if x.dim() != 2 or weight.dim() != 2 or weight.shape[1] != x.shape[1] or x.shape[1] < 1 or weight.shape[0] < 1:
            raise ValueError(f"x must be [M, K] and weight [N, K] (got {tuple(x.shape)} and {tuple(weight.shape)})")
        (M, K), N = x.shape, weight.shape[0]
        gated = activation == "silu_gated"
        if gated and N % 2:
            raise ValueError(f"a gated product needs an even number of weight rows (got {N})")
        width = N // 2 if gated else N
        x_stride, w_stride = _rows(x, "x", M, K), _rows(weight, "weight", N, K)
        # (one row has any stride: the next multiple of 16 bytes will do)
        each = 16 // x.element_size()
        x_stride = x_stride if M > 1 else -(-K // each) * each
        w_stride = w_stride if N > 1 else -(-K // each) * each
        e4m3 = dt == torch.float8_e4m3fn
        if (x_scale is not None) != e4m3 or (weight_scale is not None) != e4m3:
            raise ValueError("x_scale and weight_scale go with float8_e4m3fn operands, and only with them")
        if e4m3:
            _shaped(x_scale, "x_scale", torch.float32, dev, (M,))
            _shaped(weight_scale, "weight_scale", torch.float32, dev, (N,))
        if bias is not None:
            _shaped(bias, "bias", torch.float32, dev, (N,))
        if not isinstance(out, torch.Tensor) or out.dtype not in (torch.bfloat16, torch.float32):
            raise TypeError("out must be a bfloat16 or float32 tensor")
        _check(out, "out", out.dtype, dev)
        out_stride = _rows(out, "out", M, width)
        if out.shape[1] != width:
            raise ValueError(f"out must be [{M}, {width}] (got {tuple(out.shape)})")
        res_stride = 0
        if residual is not None:
            _check(residual, "residual", torch.bfloat16, dev)
            res_stride = _rows(residual, "residual", M, width)
            if residual.shape[1] != width:
                raise ValueError(f"residual must be [{M}, {width}] (got {tuple(residual.shape)})")
        _err(err_flag, dev)
        for name, t in (("x", x), ("weight", weight), ("x_scale", x_scale), ("weight_scale", weight_scale),
                        ("bias", bias), ("residual", residual)):
            if not (t is residual and _same_place(out, residual)):
                _apart(out, "out", t, name)
        args = KdaLinearArgs(
            M=M, N=N, K=K, activation=ACTIVATIONS[activation],
            flags=(KDA_LINEAR_E4M3 if e4m3 else 0) | (KDA_LINEAR_OUT_F32 if out.dtype == torch.float32 else 0)
            | (KDA_LINEAR_EARLY_WEIGHT if early_weight else 0),
            x=_p(x), x_row_stride=x_stride, weight=_p(weight), weight_row_stride=w_stride, x_scale=_p(x_scale),
            weight_scale=_p(weight_scale), bias=_p(bias), residual=_p(residual), residual_row_stride=res_stride,
            out=_p(out), out_row_stride=out_stride, err_flag=_p(err_flag))
        self._prepare("kda_linear", args, dev,
                      (x, weight, out, x_scale, weight_scale, bias, residual, err_flag))


def kda_linear(x, weight, out, *, x_scale=None, weight_scale=None, bias=None, residual=None,
               activation: str | None = None, early_weight: bool = False, err_flag=None,
               stream: torch.cuda.Stream | None = None) -> None:
    """Matrix product with scales, bias, activation and residual, to ``out``
    (see ``KdaLinearCall``)."""
    KdaLinearCall(x, weight, out, x_scale=x_scale, weight_scale=weight_scale, bias=bias, residual=residual,
                  activation=activation, early_weight=early_weight, err_flag=err_flag)(stream)


# --------------------------------------------------------------- log probabilities
class KdaLogprobsCall(_Call):
    """A prepared ``kda_logprobs`` call.

      logits   fp32 or bf16 [..., V] (one or more leading dimensions whose
               rows have one stride between them, unit inner stride)
      tokens   int32 [...] of the leading dimensions (as verification's
               ``tokens``: rows whose token is < 0 are not read), or None
      num_top  likeliest alternatives per row, 0 .. 32

    Results in tensors that the call owns, of the leading dimensions:
    ``logprobs`` fp32 and ``ranks`` int32 (None without tokens), ``entropy``
    fp32, ``top_ids`` int32 and ``top_logprobs`` fp32 [..., num_top]."""

    def __init__(self, logits, tokens=None, *, num_top: int = 0, err_flag=None):
        if not isinstance(logits, torch.Tensor) or logits.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError("logits must be a float32 or bfloat16 tensor")
        _check(logits, "logits", logits.dtype, None)
        if logits.dim() < 2 or logits.shape[-1] < 1:
            raise ValueError(f"logits must be [..., V] (got {tuple(logits.shape)})")
        dev, lead, V = logits.device, tuple(logits.shape[:-1]), logits.shape[-1]
        if V > 1 and logits.stride(-1) != 1:
            raise ValueError("logits need a unit inner stride")
        stride, want, rows = V, None, 1
        for n, st in zip(reversed(lead), reversed(logits.stride()[:-1])):   # innermost first
            if n > 1:
                if want is None:
                    stride = st
                elif st != want:
                    raise ValueError(f"logits: rows must have one stride (got strides {logits.stride()})")
                want = st * n
            rows *= n
        if rows > 1 and stride < V:
            raise ValueError(f"logits: rows must have one stride of at least V (got strides {logits.stride()})")
        num_top = int(num_top)
        if not 0 <= num_top <= LOGPROBS_MAX_TOP:
            raise ValueError(f"num_top must be 0 .. {LOGPROBS_MAX_TOP} (got {num_top})")
        if tokens is not None:
            _shaped(tokens, "tokens", torch.int32, dev, lead)
        _err(err_flag, dev)
        i32, f32 = dict(dtype=torch.int32, device=dev), dict(dtype=torch.float32, device=dev)
        self.logprobs = self.ranks = None
        if tokens is not None:
            self.logprobs, self.ranks = torch.empty(lead, **f32), torch.empty(lead, **i32)
        self.entropy = torch.empty(lead, **f32)
        self.top_ids, self.top_logprobs = torch.empty(*lead, num_top, **i32), torch.empty(*lead, num_top, **f32)
        args = KdaLogprobsArgs(
            R=rows, V=V, num_top=num_top, flags=KDA_LOGPROBS_BF16 if logits.dtype == torch.bfloat16 else 0,
            logits=_p(logits), logits_row_stride=stride, tokens=_p(tokens), logprobs=_p(self.logprobs),
            ranks=_p(self.ranks), entropy=_p(self.entropy), top_ids=_p(self.top_ids) if num_top else None,
            top_logprobs=_p(self.top_logprobs) if num_top else None, err_flag=_p(err_flag))
        own = tuple(t for t in (self.logprobs, self.ranks, self.entropy, self.top_ids, self.top_logprobs)
                    if t is not None and t.numel())
        self._prepare("kda_logprobs", args, dev, (logits, tokens, err_flag), own)


def kda_logprobs(logits, tokens=None, *, num_top: int = 0, err_flag=None, stream: torch.cuda.Stream | None = None):
    """Returns ``(logprobs, ranks, entropy, top_ids, top_logprobs)`` (see
    ``KdaLogprobsCall``)."""
    with torch.cuda.stream(stream):
        c = KdaLogprobsCall(logits, tokens, num_top=num_top, err_flag=err_flag)
        c(stream)
    return c.logprobs, c.ranks, c.entropy, c.top_ids, c.top_logprobs
