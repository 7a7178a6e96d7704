"""Operators of the descriptor network and its training: attention, rotary positions, norms, gated layer, matching loss.

The maps that this package matches come from a transformer over image patches whose descriptor head is trained by a
symmetric softmax loss over matched descriptors ("MASt3R" note on cv-learn.com, section 手法とアーキテクチャ). Each operator here
has a forward and a backward function over the C ABI (``include/ddm.h`` documents them) and a differentiable one for
torch's autograd: :func:`attention`, :func:`rotary`, :func:`layer_norm`, :func:`residual_norm`, :func:`gated_linear`,
:func:`matching_loss`.

Packed sets: sequences of different lengths lie one after another along the first axis; ``cu`` (int32, device) holds
the B + 1 places where they begin and end. The lengths stay on the device: no call waits for it.
"""
from __future__ import annotations

import ctypes as C
import functools
import math

import torch
from torch.autograd.function import once_differentiable

import dense_descriptor_matching_amd as _api     # the package itself: its library handle, checks and errors

_DT = _api._DT


def declare(lib):
    P, I, I64, SZ, F = C.c_void_p, C.c_int, C.c_int64, C.c_size_t, C.c_double
    view = [P, I64, I64]
    sizes = [P, P, I, I, I, I, I, I, I, I, F]              # cu_q, cu_k, B, Tq, Tk, Hq, Hkv, D, dtype, causal, scale
    for f in (lib.ddm_attention_forward_workspace_bytes, lib.ddm_attention_backward_workspace_bytes):
        f.argtypes, f.restype = [I] * 7, SZ
    lib.ddm_attention_forward.argtypes = view * 3 + sizes + [P, P, P, SZ, P]
    lib.ddm_attention_backward.argtypes = view * 4 + [P, P] + sizes + [P, P, P, P, SZ, P]
    lib.ddm_layer_norm_forward.argtypes = [P, I64, P, P, I64, I, I, I, F, P, P, P, P]
    lib.ddm_layer_norm_backward_workspace_bytes.argtypes = [I64, I, I]
    lib.ddm_layer_norm_backward_workspace_bytes.restype = SZ
    lib.ddm_layer_norm_backward.argtypes = [P, P, I64, P, P, P, I64, I, I, I, P, P, P, P, SZ, P]
    for f in (lib.ddm_matching_loss_forward_workspace_bytes, lib.ddm_matching_loss_backward_workspace_bytes,
              lib.ddm_matching_loss_workspace_bytes):
        f.argtypes, f.restype = [I] * 4, SZ
    lib.ddm_matching_loss_forward.argtypes = [P, P, P, I, I, I, I, F, P, P, P, P, SZ, P]
    lib.ddm_matching_loss_backward.argtypes = [P, P, P, P, P, P, I, I, I, I, F, P, P, P, SZ, P]
    heads = [P, I64, I64, I]
    lib.ddm_rotary.argtypes = heads * 2 + [P, P, I, I, I, I, I, I, I, F, P, I64, I64, P, I64, I64, P]
    rows = [P, I64]
    lib.ddm_residual_norm_forward.argtypes = rows * 3 + [P] * 5 + [I64, I, I, I, I, I, F, P, P, P, P]
    lib.ddm_residual_norm_backward_workspace_bytes.argtypes = [I64, I, I, I]
    lib.ddm_residual_norm_backward.argtypes = [P, P] + rows * 3 + [P] * 5 + [I64, I, I, I, I, I] + [P] * 9 + [SZ, P]
    lib.ddm_gated_linear_forward.argtypes = rows + [P, P, I64, I, I, I, I, P, P, P, SZ, P]
    lib.ddm_gated_linear_backward.argtypes = [P] + rows + [P, P, I64, I, I, I, I, P, P, P, P, SZ, P]
    for f in (lib.ddm_gated_linear_forward_workspace_bytes, lib.ddm_gated_linear_backward_workspace_bytes):
        f.argtypes = [I64, I, I, I]
    lib.ddm_gated_linear_repack_bytes.argtypes = [I64, I, I]
    for f in (lib.ddm_residual_norm_backward_workspace_bytes, lib.ddm_gated_linear_repack_bytes, lib.ddm_gated_linear_forward_workspace_bytes,
              lib.ddm_gated_linear_backward_workspace_bytes):
        f.restype = SZ
    for f in (lib.ddm_attention_forward, lib.ddm_attention_backward, lib.ddm_layer_norm_forward,
              lib.ddm_layer_norm_backward, lib.ddm_matching_loss_forward, lib.ddm_matching_loss_backward, lib.ddm_rotary,
              lib.ddm_residual_norm_forward, lib.ddm_residual_norm_backward, lib.ddm_gated_linear_forward,
              lib.ddm_gated_linear_backward):
        f.restype = I


def _call(dev, what, *args):
    """Enqueue on the tensors' device and its current stream."""
    f, at = getattr(_api.lib(), what), dev.index
    if torch.cuda.current_device() == at:
        rc = f(*args, torch.cuda.current_stream(at).cuda_stream)
    else:
        with torch.cuda.device(dev):
            rc = f(*args, torch.cuda.current_stream(at).cuda_stream)
    if rc != 0:
        raise _api.DDMError(rc, what)


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(what, *sizes):
    """The library's workspace size for these sizes (a pure function of them)."""
    n = getattr(_api.lib(), what)(*sizes)
    if n == 0:
        raise _api.DDMError(-4, f"{what} (sizes outside the limits stated in include/ddm.h)")
    return n


def _tensor(t, name, dtype=None, dev=None, shape=None, contiguous=True):
    """t, checked: a device tensor of the dtype (None: any supported), device and shape asked for."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a device tensor")
    if dtype is None:
        if t.dtype not in _DT:
            raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    elif t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if dev is not None and t.device != dev:
        raise ValueError(f"tensors on {dev} and {t.device}: one device per call")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _cu(cu, name, dev):
    """(number of sequences, pointer) of a packed set's boundaries."""
    if cu is None:
        return 1, None
    _tensor(cu, name, torch.int32, dev)
    if cu.dim() != 1 or cu.numel() < 2:
        raise ValueError(f"{name} must hold at least two boundaries in one dimension")
    return cu.numel() - 1, cu.data_ptr()


# ---------------------------------------------------------------------------------------------------- attention
def _heads_view(t, name):
    """Strides (tokens, heads) of [T, H, D] rows that are whole 16-byte pieces."""
    ts, hs, es = t.stride()
    T, H, D = t.shape
    e = t.element_size()
    ts, hs = ts if T > 1 else 0, hs if H > 1 else 0
    if (es != 1 and D > 1) or ts * e % 16 or hs * e % 16 or t.data_ptr() % 16:
        raise ValueError(f"{name}: the last dimension must be contiguous and its rows on 16-byte boundaries")
    return t.data_ptr(), ts, hs


def _attention_sizes(q, k, v, cu_q, cu_k, scale):
    _tensor(q, "q", contiguous=False)
    dev, dt = q.device, q.dtype
    _tensor(k, "k", dt, dev, contiguous=False)
    _tensor(v, "v", dt, dev, contiguous=False)
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k and v must be [tokens, heads, head dimension]")
    Tq, Hq, D = q.shape
    Tk, Hkv, Dk = k.shape
    if v.shape != k.shape or Dk != D:
        raise ValueError("k and v must share their shape, and its head dimension with q")
    if Hkv == 0 or Hq % Hkv:
        raise ValueError("the number of query heads must be a multiple of the number of key heads")
    if (cu_q is None) != (cu_k is None):
        raise ValueError("cu_q and cu_k come together")
    B, pq = _cu(cu_q, "cu_q", dev)
    Bk, pk = _cu(cu_k, "cu_k", dev)
    if B != Bk:
        raise ValueError("cu_q and cu_k must hold the same number of sequences")
    return (B, Tq, Tk, Hq, Hkv, D, _DT[dt]), pq, pk, float(D ** -0.5 if scale is None else scale)


def attention_forward(q, k, v, cu_q=None, cu_k=None, *, causal: bool = False, scale: float | None = None):
    """Attention of packed sequences: q [Tq, Hq, D], k, v [Tk, Hkv, D]; query head h uses key head h // (Hq // Hkv).

    A query sees the keys of its sequence, with ``causal`` up to its own position counted from the sequences' ends.
    ``scale`` defaults to D ** -0.5. Returns (out [Tq, Hq, D], lse float32 [Tq, Hq]); a query that sees no key gets 0 and
    -inf, one with a score of NaN gets NaN in both. The tensors may be views (of a packed qkv projection, say) whose rows
    are whole 16-byte pieces."""
    sizes, pq, pk, scale = _attention_sizes(q, k, v, cu_q, cu_k, scale)
    nbytes = _workspace_bytes("ddm_attention_forward_workspace_bytes", *sizes)
    out = torch.empty_like(q, memory_format=torch.contiguous_format)
    lse = q.new_empty(q.shape[:2], dtype=torch.float32)
    ws = q.new_empty(nbytes, dtype=torch.uint8)
    _call(q.device, "ddm_attention_forward", *_heads_view(q, "q"), *_heads_view(k, "k"), *_heads_view(v, "v"), pq, pk,
          *sizes, int(causal), scale, out.data_ptr(), lse.data_ptr(), ws.data_ptr(), nbytes)
    return out, lse


def attention_backward(dout, q, k, v, out, lse, cu_q=None, cu_k=None, *, causal: bool = False,
                       scale: float | None = None):
    """Gradients (dq, dk, dv) of :func:`attention_forward` by its out, from that call's inputs, out and lse."""
    sizes, pq, pk, scale = _attention_sizes(q, k, v, cu_q, cu_k, scale)
    _tensor(dout, "dout", q.dtype, q.device, q.shape, contiguous=False)
    _tensor(out, "out", q.dtype, q.device, q.shape)
    _tensor(lse, "lse", torch.float32, q.device, q.shape[:2])
    nbytes = _workspace_bytes("ddm_attention_backward_workspace_bytes", *sizes)
    dq, dk, dv = (torch.empty_like(t, memory_format=torch.contiguous_format) for t in (q, k, v))
    ws = q.new_empty(nbytes, dtype=torch.uint8)
    _call(q.device, "ddm_attention_backward", *_heads_view(dout, "dout"), *_heads_view(q, "q"), *_heads_view(k, "k"),
          *_heads_view(v, "v"), out.data_ptr(), lse.data_ptr(), pq, pk, *sizes, int(causal), scale, dq.data_ptr(),
          dk.data_ptr(), dv.data_ptr(), ws.data_ptr(), nbytes)
    return dq, dk, dv


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cu_q, cu_k, causal, scale):
        out, lse = attention_forward(q, k, v, cu_q, cu_k, causal=causal, scale=scale)
        ctx.save_for_backward(q, k, v, out, lse, cu_q, cu_k)
        ctx.options = dict(causal=causal, scale=scale)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        q, k, v, out, lse, cu_q, cu_k = ctx.saved_tensors
        dout = dout.contiguous()
        if dout.data_ptr() % 16:            # a view of a larger gradient
            dout = dout.clone()
        return attention_backward(dout, q, k, v, out, lse, cu_q, cu_k, **ctx.options) + (None,) * 4


def attention(q, k, v, cu_q=None, cu_k=None, *, causal: bool = False, scale: float | None = None):
    """Differentiable :func:`attention_forward`; returns out alone."""
    return _Attention.apply(q, k, v, cu_q, cu_k, causal, scale)


# --------------------------------------------------------------------------------------------------- layer norm
def _norm_rows(x, weight, bias):
    """x as rows of its last dimension: (rows, columns, row stride, wtype)."""
    _tensor(x, "x", contiguous=False)
    if x.dim() == 0 or x.shape[-1] == 0:
        raise ValueError("x must have a last dimension of at least one")
    cols = x.shape[-1]
    if not x.is_contiguous() and not (x.dim() == 2 and x.stride(1) == 1 and x.stride(0) >= cols):
        raise ValueError("x must be contiguous, or two-dimensional with contiguous rows")
    wtype = torch.float32
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            wtype = _tensor(t, name, None, x.device, x.shape[-1:]).dtype
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise TypeError("weight and bias must share their dtype")
    if wtype not in (torch.float32, x.dtype):
        raise TypeError("weight and bias must be float32 or of x's dtype")
    ldx = x.stride(0) if x.dim() == 2 and x.shape[0] > 1 else cols
    return x.numel() // cols, cols, ldx, wtype


def _at(t):
    return None if t is None else t.data_ptr()


def layer_norm_forward(x, weight=None, bias=None, *, eps: float = 1e-6):
    """Layer norm over the last dimension. Returns (y like x, mean, rstd float32 over the rows)."""
    N, cols, ldx, wtype = _norm_rows(x, weight, bias)
    y = torch.empty_like(x, memory_format=torch.contiguous_format)
    mean = x.new_empty(x.shape[:-1], dtype=torch.float32)
    rstd = torch.empty_like(mean)
    _call(x.device, "ddm_layer_norm_forward", x.data_ptr(), ldx, _at(weight), _at(bias), N, cols, _DT[x.dtype],
          _DT[wtype], float(eps), y.data_ptr(), mean.data_ptr(), rstd.data_ptr())
    return y, mean, rstd


def layer_norm_backward(dy, x, weight, mean, rstd, *, wtype=None, need_dx: bool = True, need_dweight: bool = True,
                        need_dbias: bool = True):
    """Gradients (dx, dweight, dbias) of :func:`layer_norm_forward` by its y; None for those not wanted. ``wtype`` is the
    dtype of dweight and dbias where there is no weight (float32 by default)."""
    N, cols, ldx, wt = _norm_rows(x, weight, None)
    wt = wt if weight is not None or wtype is None else wtype
    if wt not in (torch.float32, x.dtype):
        raise TypeError("wtype must be float32 or x's dtype")
    _tensor(dy, "dy", x.dtype, x.device, x.shape)
    _tensor(mean, "mean", torch.float32, x.device, x.shape[:-1])
    _tensor(rstd, "rstd", torch.float32, x.device, x.shape[:-1])
    dx = torch.empty_like(x, memory_format=torch.contiguous_format) if need_dx else None
    dw = x.new_empty(cols, dtype=wt) if need_dweight else None
    db = x.new_empty(cols, dtype=wt) if need_dbias else None
    nbytes = _workspace_bytes("ddm_layer_norm_backward_workspace_bytes", N, cols, _DT[x.dtype])
    ws = x.new_empty(nbytes, dtype=torch.uint8)
    _call(x.device, "ddm_layer_norm_backward", dy.data_ptr(), x.data_ptr(), ldx, _at(weight), mean.data_ptr(),
          rstd.data_ptr(), N, cols, _DT[x.dtype], _DT[wt], _at(dx), _at(dw), _at(db), ws.data_ptr(), nbytes)
    return dx, dw, db


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = layer_norm_forward(x, weight, bias, eps=eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.wtype = None if bias is None else bias.dtype
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        return layer_norm_backward(dy.contiguous(), x, weight, mean, rstd, wtype=ctx.wtype, need_dx=need[0],
                                   need_dweight=need[1], need_dbias=need[2]) + (None,)


def layer_norm(x, weight=None, bias=None, *, eps: float = 1e-6):
    """Differentiable :func:`layer_norm_forward`; returns y alone."""
    return _LayerNorm.apply(x, weight, bias, eps)


# ------------------------------------------------------------------------------------------------------- rotary
def rotary_frequencies(pairs: int, base: float = 10000.0, *, scaling: str | None = None, factor: float = 1.0,
                       length: int | None = None, slow: float = 1.0, fast: float = 32.0, device=None):
    """Frequencies base ** (-i / pairs) of the pairs of an axis, float64 [pairs], as :func:`rotary` takes them.

    ``scaling`` fits them to positions ``factor`` times as far as those trained on: "linear" divides all by the factor; "base"
    raises the base so that the last pair's is divided by it and the first's stays; "ramp" divides those of pairs that turn at
    most ``slow`` times over ``length`` positions, keeps those that turn ``fast`` times or more, and mixes between them in
    proportion to the turns (a magnitude of 0.1 log(factor) + 1 goes with it)."""
    if pairs < 1 or not base > 0 or not factor > 0:
        raise ValueError("pairs, base and factor must be positive")
    if scaling == "base" and pairs > 1:
        base = base * factor ** (pairs / (pairs - 1))
    f = base ** (-torch.arange(pairs, dtype=torch.float64) / pairs)
    if scaling == "linear":
        f = f / factor
    elif scaling == "ramp":
        if length is None or not 0 <= slow < fast:
            raise ValueError("ramp needs the length trained on, and slow below fast")
        keep = ((length * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
    elif scaling not in (None, "base"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return f.to(device)


def _rotary_heads(t, name):
    if t is None:
        return None, 0, 0, 0
    if t.stride(2) != 1 and t.shape[2] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return t.data_ptr(), t.stride(0), t.stride(1), t.shape[1]


def _rotary(q, k, positions, frequencies, interleaved, magnitude, inverse, out, names):
    _tensor(q, names[0], contiguous=False)
    if q.dim() != 3:
        raise ValueError(f"{names[0]} must be [tokens, heads, head dimension]")
    dev, (T, _, D) = q.device, q.shape
    if k is not None:
        _tensor(k, names[1], q.dtype, dev, contiguous=False)
        if k.dim() != 3 or k.shape[0] != T or k.shape[2] != D:
            raise ValueError(f"{names[1]} must share its tokens and its head dimension with {names[0]}")
    _tensor(frequencies, "frequencies", torch.float64, dev)
    if frequencies.dim() not in (1, 2) or frequencies.numel() == 0:
        raise ValueError("frequencies must be [pairs] or [axes, pairs]")
    axes, pairs = (1, *frequencies.shape) if frequencies.dim() == 1 else frequencies.shape
    _tensor(positions, "positions", torch.int32, dev)
    if tuple(positions.shape) not in ((T, axes),) + (((T,),) if axes == 1 else ()):
        raise ValueError(f"positions must be [{T}, {axes}], one place on each axis a token, not {list(positions.shape)}")
    if 2 * axes * pairs > D:
        raise ValueError(f"{axes} axes of {pairs} pairs do not fit into heads of {D}")
    if out is None:
        qo = torch.empty_like(q, memory_format=torch.contiguous_format)
        ko = None if k is None else torch.empty_like(k, memory_format=torch.contiguous_format)
    else:
        qo, ko = out
        for t, s, name in ((qo, q, "out[0]"), (ko, k, "out[1]")):
            if (t is None) != (s is None):
                raise ValueError("out must hold one tensor for each of q and k")
            if t is not None:
                _tensor(t, name, q.dtype, dev, s.shape, contiguous=False)
        if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (q, k, qo, ko)):
            raise RuntimeError("out= has no gradient, but one of the tensors requires it: use rotary, or torch.no_grad()")
    qv, kv, qw, kw = (_rotary_heads(t, n) for t, n in ((q, names[0]), (k, names[1]), (qo, "out[0]"), (ko, "out[1]")))
    _call(dev, "ddm_rotary", *qv, *kv, positions.data_ptr(), frequencies.data_ptr(), T, D, axes, pairs, _DT[q.dtype],
          int(interleaved), int(inverse), float(magnitude), *qw[:3], *kw[:3])
    if out is not None:                     # a backward pass that was to read what stood there raises
        torch.autograd.graph.increment_version([t for t in (qo, ko) if t is not None])
    return qo, ko


def rotary_forward(q, k, positions, frequencies, *, interleaved: bool = False, magnitude: float = 1.0, out=None):
    """Rotary positions of queries q [T, Hq, D] and keys k [T, Hk, D] (or None) of the same tokens; returns both.

    ``positions`` int32 [T], or [T, axes] (row and column of an image patch); ``frequencies`` float64 [pairs] or [axes, pairs]
    (:func:`rotary_frequencies`). The first 2 axes pairs elements of a head are turned, axis by axis, the rest stays: element i of an
    axis' 2 pairs goes with i + pairs, or, ``interleaved``, 2i with 2i + 1, by the angle position * frequency, times ``magnitude``.
    The tensors may be views (of a packed qkv projection, say) with contiguous heads. ``out`` holds tensors to write to, q and k
    themselves (each in its own place) or others that overlap neither them nor one another; as with torch's own ``out=``, none of the tensors may require a gradient then, unless gradients are off."""
    return _rotary(q, k, positions, frequencies, interleaved, magnitude, False, out, ("q", "k"))


def rotary_backward(dq, dk, positions, frequencies, *, interleaved: bool = False, magnitude: float = 1.0, out=None):
    """Gradients of :func:`rotary_forward` by q and k, from those by its outputs."""
    return _rotary(dq, dk, positions, frequencies, interleaved, magnitude, True, out, ("dq", "dk"))


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, positions, frequencies, interleaved, magnitude):
        ctx.save_for_backward(positions, frequencies)
        ctx.options = dict(interleaved=interleaved, magnitude=magnitude)
        ctx.set_materialize_grads(False)
        q, k = rotary_forward(q, k, positions, frequencies, **ctx.options)
        return q if k is None else (q, k)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk=None):
        given = [t.contiguous() for t in (dq, dk) if t is not None]
        if not given:
            return (None,) * 6
        if len(given) == 2:
            dq, dk = rotary_backward(*given, *ctx.saved_tensors, **ctx.options)
        else:
            got, _ = rotary_backward(given[0], None, *ctx.saved_tensors, **ctx.options)
            dq, dk = (got, None) if dq is not None else (None, got)
        return dq, dk, None, None, None, None


def rotary(q, k, positions, frequencies, *, interleaved: bool = False, magnitude: float = 1.0):
    """Differentiable (by q and k) :func:`rotary_forward`; without k it returns q alone."""
    if torch.is_grad_enabled() and any(isinstance(t, torch.Tensor) and t.requires_grad for t in (frequencies, magnitude)):
        raise ValueError("frequencies and magnitude get no gradient: give them detached")
    return _Rotary.apply(q, k, positions, frequencies, interleaved, magnitude)


# ------------------------------------------------------------------------------------------------ residual norm
def _rows(t, name, like=None):
    """(pointer, row stride) of t as rows of its last dimension."""
    if t is None:
        return None, 0
    if like is not None:
        _tensor(t, name, like.dtype, like.device, like.shape, contiguous=False)
    cols = t.shape[-1]
    if t.is_contiguous():
        return t.data_ptr(), cols
    if t.dim() != 2 or t.stride(1) != 1 or t.stride(0) < cols:
        raise ValueError(f"{name} must be contiguous, or two-dimensional with contiguous rows")
    return t.data_ptr(), t.stride(0) if t.shape[0] > 1 else cols


def _residual_sizes(x, branch, gate, params, branch_norm):
    _tensor(x, "x", contiguous=False)
    if x.dim() == 0 or x.shape[-1] == 0:
        raise ValueError("x must have a last dimension of at least one")
    wtype = None
    for name, t in params.items():
        if t is None:
            continue
        _tensor(t, name, None, x.device, x.shape[-1:])
        if t.dtype not in (torch.float32, x.dtype) or wtype not in (None, t.dtype):
            raise TypeError("scale, weights and biases must share their dtype, float32 or x's")
        if name.startswith("branch") and not branch_norm:
            raise ValueError(f"{name} goes with branch_norm")
        wtype = t.dtype
    views = *_rows(x, "x", x), *_rows(branch, "branch", x), *_rows(gate, "gate", x)
    return x.numel() // x.shape[-1], x.shape[-1], wtype or torch.float32, views


def residual_norm_forward(x, branch, weight=None, bias=None, *, scale=None, gate=None, branch_norm: bool = False,
                          branch_weight=None, branch_bias=None, rms: bool = False, eps: float = 1e-6):
    """The sum of a residual stream and a block's branch, and its norm, over the last dimension:

        t = branch, or with ``branch_norm`` norm(branch) * branch_weight + branch_bias
        s = x + scale * sigmoid(gate) * t,    y = norm(s) * weight + bias

    norm is a layer norm, with ``rms`` one without means. x, branch and gate share shape and type; the others have one value a column.
    Returns (s, y, stats): stats float32 [2, rows...] holds the means and 1 / deviations of s, with ``branch_norm`` [4, rows...] and
    those of the branch. y is taken of s before it is rounded."""
    params = dict(scale=scale, branch_weight=branch_weight, branch_bias=branch_bias, weight=weight, bias=bias)
    N, cols, wtype, views = _residual_sizes(x, branch, gate, params, branch_norm)
    s, y = (torch.empty_like(x, memory_format=torch.contiguous_format) for _ in range(2))
    stats = x.new_empty((4 if branch_norm else 2,) + x.shape[:-1], dtype=torch.float32)
    _call(x.device, "ddm_residual_norm_forward", *views, *map(_at, params.values()), N, cols, _DT[x.dtype], _DT[wtype],
          int(branch_norm), int(rms), float(eps), s.data_ptr(), y.data_ptr(), stats.data_ptr())
    return s, y, stats


_RESIDUAL_GRADIENTS = ("dx", "dbranch", "dweight", "dbias", "dscale", "dgate", "dbranch_weight", "dbranch_bias")


def residual_norm_backward(dy, ds, x, branch, stats, weight=None, *, scale=None, gate=None, branch_norm: bool = False,
                           branch_weight=None, branch_bias=None, rms: bool = False, wtype=None, needs=None):
    """Gradients (dx, dbranch, dweight, dbias, dscale, dgate, dbranch_weight, dbranch_bias) of :func:`residual_norm_forward` by its
    outputs' gradients dy and ds (None for zeros), from its inputs and stats. ``needs`` names those that are wanted, the others are
    None; by default all but dscale without a scale, dgate without a gate and the branch's without ``branch_norm``. ``wtype`` is
    the parameters' dtype where none of them is given (float32 by default)."""
    params = dict(scale=scale, branch_weight=branch_weight, branch_bias=branch_bias, weight=weight)
    N, cols, wt, views = _residual_sizes(x, branch, gate, params, branch_norm)
    if wtype is not None and all(t is None for t in params.values()):
        wt = wtype
    if wt not in (torch.float32, x.dtype):
        raise TypeError("wtype must be float32 or x's dtype")
    for t, name in ((dy, "dy"), (ds, "ds")):
        if t is not None:
            _tensor(t, name, x.dtype, x.device, x.shape)
    _tensor(stats, "stats", torch.float32, x.device, (4 if branch_norm else 2,) + x.shape[:-1])
    if needs is None:
        needs = {"dx", "dbranch", "dweight", "dbias"}
        needs |= ({"dscale"} if scale is not None else set()) | ({"dgate"} if gate is not None else set())
        needs |= {"dbranch_weight", "dbranch_bias"} if branch_norm else set()
    needs = set(needs)
    if needs - set(_RESIDUAL_GRADIENTS):
        raise ValueError(f"unknown gradients {sorted(needs - set(_RESIDUAL_GRADIENTS))}")
    if ("dgate" in needs and gate is None) or (not branch_norm and needs & {"dbranch_weight", "dbranch_bias"}):
        raise ValueError("a gradient by what the call does not have")
    got = {n: None if n not in needs else
           torch.empty_like(x, memory_format=torch.contiguous_format) if n in ("dx", "dbranch", "dgate") else
           x.new_empty(cols, dtype=wt) for n in _RESIDUAL_GRADIENTS}
    nbytes, ws = 0, None
    if needs - {"dx", "dbranch", "dgate"}:
        nbytes = _workspace_bytes("ddm_residual_norm_backward_workspace_bytes", N, cols, _DT[x.dtype], int(branch_norm))
        ws = x.new_empty(nbytes, dtype=torch.uint8)
    _call(x.device, "ddm_residual_norm_backward", _at(dy), _at(ds), *views, *map(_at, params.values()), stats.data_ptr(), N, cols,
          _DT[x.dtype], _DT[wt], int(branch_norm), int(rms),
          *(_at(got[n]) for n in ("dx", "dbranch", "dgate", "dscale", "dbranch_weight", "dbranch_bias", "dweight", "dbias")),
          _at(ws), nbytes)
    return tuple(got[n] for n in _RESIDUAL_GRADIENTS)


class _ResidualNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, branch, weight, bias, scale, gate, branch_weight, branch_bias, branch_norm, rms, eps):
        s, y, stats = residual_norm_forward(x, branch, weight, bias, scale=scale, gate=gate, branch_norm=branch_norm,
                                            branch_weight=branch_weight, branch_bias=branch_bias, rms=rms, eps=eps)
        ctx.save_for_backward(x, branch, weight, scale, gate, branch_weight, branch_bias, stats)
        ctx.options = dict(branch_norm=branch_norm, rms=rms, wtype=None if bias is None else bias.dtype)
        ctx.set_materialize_grads(False)
        return s, y

    @staticmethod
    @once_differentiable
    def backward(ctx, ds, dy):
        x, branch, weight, scale, gate, branch_weight, branch_bias, stats = ctx.saved_tensors
        if ds is None and dy is None:
            return (None,) * 11
        ds, dy = (None if t is None else t.contiguous() for t in (ds, dy))
        needs = {n for n, wanted in zip(_RESIDUAL_GRADIENTS, ctx.needs_input_grad) if wanted}
        return residual_norm_backward(dy, ds, x, branch, stats, weight, scale=scale, gate=gate, branch_weight=branch_weight,
                                      branch_bias=branch_bias, needs=needs, **ctx.options) + (None,) * 3


def residual_norm(x, branch, weight=None, bias=None, *, scale=None, gate=None, branch_norm: bool = False, branch_weight=None,
                  branch_bias=None, rms: bool = False, eps: float = 1e-6):
    """Differentiable :func:`residual_norm_forward`; returns (s, y)."""
    return _ResidualNorm.apply(x, branch, weight, bias, scale, gate, branch_weight, branch_bias, branch_norm, rms, eps)


# ------------------------------------------------------------------------------------------------- gated linear
ACTIVATIONS = {"silu": 0, "gelu": 1, "sigmoid": 2}


def _gated_sizes(x, weight, activation):
    _tensor(x, "x", contiguous=False)
    if x.dim() == 0 or x.shape[-1] == 0:
        raise ValueError("x must have a last dimension of at least one")
    _tensor(weight, "weight", x.dtype, x.device)
    if weight.dim() != 2 or weight.shape[1] != x.shape[-1] or weight.shape[0] % 2 or weight.shape[0] == 0:
        raise ValueError("weight must be [2 * hidden, columns of x]: the gate's rows, then the other projection's")
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}")
    return x.numel() // x.shape[-1], x.shape[-1], weight.shape[0] // 2, _DT[x.dtype]


def _gated_call(x, weight, what, *args):
    try:
        _call(x.device, what, *args)
    except _api.DDMError as e:
        if e.status == -1 and weight.data_ptr() % 16 and weight.shape[1] * weight.itemsize % 16 == 0:
            raise _api.DDMError(-1, f"{what}: a weight off a 16-byte boundary, with rows of whole 16-byte pieces (clone it)") from None
        raise


@functools.lru_cache(maxsize=1024)
def _gated_bytes(what, copy, N, C, F, dtype):
    """The workspace's bytes, with room for a copy of x or without."""
    nbytes = _workspace_bytes(what, N, C, F, dtype)
    return nbytes if copy or N == 0 else max(nbytes - _workspace_bytes("ddm_gated_linear_repack_bytes", N, C, dtype), 16)


def _copied(view, x):
    """Whether x's rows are copied first: they are not whole 16-byte pieces."""
    e = x.itemsize
    return (view[0] | view[1] * e | x.shape[-1] * e) % 16 != 0


def gated_linear_forward(x, weight, bias=None, *, activation: str = "silu", keep: bool = False):
    """Gated linear layer h = act(x Wg^T + bg) * (x Wu^T + bu) of x [..., C]: weight [2F, C] holds the F rows of Wg and then those of Wu,
    bias [2F] likewise. Returns (h [..., F], kept): kept [..., 2F] is what :func:`gated_linear_backward` needs with ``keep``, else
    None. ``activation``: "silu" g * sigmoid(g), "gelu" g * Phi(g), "sigmoid". x is contiguous or two-dimensional with contiguous rows;
    a weight whose rows are whole 16-byte pieces begins on such a boundary."""
    sizes = _gated_sizes(x, weight, activation)
    F = sizes[2]
    if bias is not None:
        _tensor(bias, "bias", x.dtype, x.device, (2 * F,))
    view = _rows(x, "x")
    nbytes = _gated_bytes("ddm_gated_linear_forward_workspace_bytes", _copied(view, x), *sizes)
    h = x.new_empty(x.shape[:-1] + (F,))
    kept = x.new_empty(x.shape[:-1] + (2 * F,)) if keep else None
    ws = x.new_empty(nbytes, dtype=torch.uint8)
    _gated_call(x, weight, "ddm_gated_linear_forward", *view, weight.data_ptr(), _at(bias), *sizes, ACTIVATIONS[activation],
                h.data_ptr(), _at(kept), ws.data_ptr(), nbytes)
    return h, kept


def gated_linear_backward(dh, x, weight, kept, *, activation: str = "silu", need_dx: bool = True, need_dweight: bool = True,
                          need_dbias: bool = True):
    """Gradients (dx, dweight, dbias) of :func:`gated_linear_forward` by its h; None for those not wanted. The projections (kept) and
    their gradients are rounded to x's type between the products, the latter wherever they lie (in float16 in units that fit the largest).
    A projection beyond 65504 is infinite in a float16 kept, and what the gradient has through it is infinite or NaN."""
    sizes = _gated_sizes(x, weight, activation)
    F = sizes[2]
    _tensor(dh, "dh", x.dtype, x.device, x.shape[:-1] + (F,))
    _tensor(kept, "kept", x.dtype, x.device, x.shape[:-1] + (2 * F,))
    view = _rows(x, "x")
    nbytes = _gated_bytes("ddm_gated_linear_backward_workspace_bytes", _copied(view, x), *sizes)
    dx = torch.empty_like(x, memory_format=torch.contiguous_format) if need_dx else None
    dw = torch.empty_like(weight) if need_dweight else None
    db = x.new_empty(2 * F) if need_dbias else None
    ws = x.new_empty(nbytes, dtype=torch.uint8)
    _gated_call(x, weight, "ddm_gated_linear_backward", dh.data_ptr(), *view, weight.data_ptr(), kept.data_ptr(), *sizes,
                ACTIVATIONS[activation], _at(dx), _at(dw), _at(db), ws.data_ptr(), nbytes)
    return dx, dw, db


class _GatedLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, activation, keep):
        h, kept = gated_linear_forward(x, weight, bias, activation=activation, keep=keep)
        ctx.save_for_backward(x, weight, kept)
        ctx.activation = activation
        return h

    @staticmethod
    @once_differentiable
    def backward(ctx, dh):
        x, weight, kept = ctx.saved_tensors
        need = ctx.needs_input_grad
        return gated_linear_backward(dh.contiguous(), x, weight, kept, activation=ctx.activation, need_dx=need[0], need_dweight=need[1],
                                     need_dbias=need[2]) + (None,) * 2


def gated_linear(x, weight, bias=None, *, activation: str = "silu"):
    """Differentiable :func:`gated_linear_forward`; returns h alone. What a gradient needs is kept only where one may be asked
    for: not under ``torch.no_grad()``."""
    # asked here: within apply the mode is off, and needs_input_grad follows requires_grad alone
    keep = torch.is_grad_enabled() and any(isinstance(t, torch.Tensor) and t.requires_grad for t in (x, weight, bias))
    return _GatedLinear.apply(x, weight, bias, activation, keep)


# ------------------------------------------------------------------------------------------------- matching loss
def _match_sizes(a, b, cu, what):
    _tensor(a, "a")
    _tensor(b, "b", a.dtype, a.device, a.shape)
    if a.dim() != 2:
        raise ValueError("a and b must be [matches, d]")
    B, pcu = _cu(cu, "cu", a.device)
    P, d = a.shape
    sizes = (B, P, d, _DT[a.dtype])
    return sizes, pcu, _workspace_bytes(f"ddm_matching_loss_{what}_workspace_bytes", *sizes)


def matching_loss_forward(a, b, cu=None, *, temperature: float = 0.07):
    """Symmetric softmax loss of matched descriptors a, b [P, d]: row p of one is to find row p of the other among the
    rows of its set (an image pair's matches; ``cu`` bounds the sets). Returns (loss, lse_a, lse_b), float32 [P]. Rows outside
    every set have loss 0; NaN in a descriptor makes all losses of its set NaN."""
    sizes, pcu, nbytes = _match_sizes(a, b, cu, "forward")
    loss = a.new_empty(a.shape[:1], dtype=torch.float32)
    lse_a, lse_b = torch.empty_like(loss), torch.empty_like(loss)
    ws = a.new_empty(nbytes, dtype=torch.uint8)
    _call(a.device, "ddm_matching_loss_forward", a.data_ptr(), b.data_ptr(), pcu, *sizes, float(temperature),
          loss.data_ptr(), lse_a.data_ptr(), lse_b.data_ptr(), ws.data_ptr(), nbytes)
    return loss, lse_a, lse_b


def matching_loss_backward(dloss, a, b, lse_a, lse_b, cu=None, *, temperature: float = 0.07):
    """Gradients (da, db) of :func:`matching_loss_forward` for dloss, the gradient by each match's loss (float32 [P])."""
    sizes, pcu, nbytes = _match_sizes(a, b, cu, "backward")
    for t, name in ((dloss, "dloss"), (lse_a, "lse_a"), (lse_b, "lse_b")):
        _tensor(t, name, torch.float32, a.device, a.shape[:1])
    da, db = torch.empty_like(a), torch.empty_like(b)
    ws = a.new_empty(nbytes, dtype=torch.uint8)
    _call(a.device, "ddm_matching_loss_backward", dloss.data_ptr(), a.data_ptr(), b.data_ptr(), lse_a.data_ptr(),
          lse_b.data_ptr(), pcu, *sizes, float(temperature), da.data_ptr(), db.data_ptr(), ws.data_ptr(), nbytes)
    return da, db


class _MatchingLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, a, b, cu, temperature):
        loss, lse_a, lse_b = matching_loss_forward(a, b, cu, temperature=temperature)
        ctx.save_for_backward(a, b, lse_a, lse_b, cu)
        ctx.temperature = temperature
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss):
        a, b, lse_a, lse_b, cu = ctx.saved_tensors
        return matching_loss_backward(dloss.contiguous(), a, b, lse_a, lse_b, cu, temperature=ctx.temperature) + (None,) * 2


def matching_loss(a, b, cu=None, *, temperature: float = 0.07):
    """Differentiable :func:`matching_loss_forward`; returns the loss of each match (take its mean over a batch)."""
    return _MatchingLoss.apply(a, b, cu, temperature)
