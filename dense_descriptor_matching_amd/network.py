"""Operators of the descriptor network and its training: attention, layer norm, matching loss.

The maps that this package matches come from a transformer over image patches whose descriptor head is trained by a
symmetric softmax loss over matched descriptors ("MASt3R" note on cv-learn.com, section 手法とアーキテクチャ). Each operator here
has a forward and a backward function over the C ABI (``include/ddm.h`` documents them) and a differentiable one for
torch's autograd: :func:`attention`, :func:`layer_norm`, :func:`matching_loss`.

Packed sets: sequences of different lengths lie one after another along the first axis; ``cu`` (int32, device) holds
the B + 1 places where they begin and end. The lengths stay on the device: no call waits for it.
"""
from __future__ import annotations

import ctypes as C
import functools

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
    for f in (lib.ddm_attention_forward, lib.ddm_attention_backward, lib.ddm_layer_norm_forward,
              lib.ddm_layer_norm_backward, lib.ddm_matching_loss_forward, lib.ddm_matching_loss_backward):
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
