"""Sequence operators of librecis.so: dense embedding tables for small
vocabularies, layer norm, attention of a bag's queries over the bag's keys, and
SequenceAttention, the attention pooling of a table's bags built from them.

As in recis.py, this is argument marshalling: the arithmetic runs in the CUDA
library, forward and backward are separate calls, and there is no CPU fallback.
Calls are asynchronous on `stream` (the current stream of the tensors' device
by default); outputs and scratch are allocated by torch for that stream, so the
calls may be captured into CUDA graphs (after a first call on the device).
Inputs used on another stream than the one they were made on are the caller's to
order.  Errors found on the device (a token out of range, malformed offsets) are
raised by sequence_status_sync.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import recis as _r

TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
NO_TOKEN = -1  # the default padding token


class AttendArgs(ctypes.Structure):
    _fields_ = ([("type", ctypes.c_int32), ("D", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32)]
                + [(n, ctypes.c_int64) for n in ("B", "Tq", "Tk", "max_q", "max_k")]
                + [("scale", ctypes.c_double)]
                + [(n, ctypes.c_void_p) for n in ("q_offsets", "k_offsets", "key_mask", "q", "k", "v")]
                + [(n, ctypes.c_int64) for n in ("q_stride", "q_head_stride", "k_stride", "k_head_stride",
                                                 "v_stride", "v_head_stride")]
                + [("out", ctypes.c_void_p), ("out_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64),
                   ("lse", ctypes.c_void_p), ("grad_out", ctypes.c_void_p), ("grad_out_stride", ctypes.c_int64),
                   ("grad_out_head_stride", ctypes.c_int64)]
                + [(n, ctypes.c_void_p) for n in ("grad_q", "grad_k", "grad_v")]
                + [(n, ctypes.c_int64) for n in ("grad_q_stride", "grad_q_head_stride", "grad_k_stride",
                                                 "grad_k_head_stride", "grad_v_stride", "grad_v_head_stride")])


def _elsewhere(stream, *tensors) -> bool:
    """Whether the call runs on another device or stream than the current one.
    Every tensor (None: left out) is on the first one's device."""
    index = tensors[0].get_device()  # -1: not a GPU's
    for t in tensors:
        if t is not None and (t.get_device() != index or index < 0):
            raise ValueError(f"expected CUDA tensors on one device, got {t.device} beside {tensors[0].device}")
    if stream is None:
        return index != torch.cuda.current_device()
    if stream.device != tensors[0].device:
        raise ValueError(f"the stream belongs to {stream.device}, the tensors to {tensors[0].device}")
    return True


def _on(stream, t: torch.Tensor):
    """The context that makes the call's stream, and with it its device, current."""
    return torch.cuda.stream(torch.cuda.current_stream(t.device) if stream is None else stream)


def _raw(dev: torch.device) -> int:
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _type(t: torch.Tensor, name: str, types=TYPES) -> int:
    code = types.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: expected one of {', '.join(str(d) for d in types)}, got {t.dtype}")
    return code


def _int64(t: torch.Tensor, name: str) -> torch.Tensor:
    if t.dtype != torch.int64:
        raise TypeError(f"{name}: expected {torch.int64}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    return t


def _rows(t: torch.Tensor, name: str, D: Optional[int] = None):
    """(rows, D, row stride) of a tensor seen as rows of its last dimension."""
    shape = t.shape
    if not shape:
        raise ValueError(f"{name}: expected rows, got a scalar")
    width = shape[-1]
    if (D is None or width == D) and width and t.is_contiguous():
        return t.numel() // width, width, width
    if D is not None and width != D:
        raise ValueError(f"{name}: expected rows of {D}, got {width}")
    n = t.numel() // width if width else 0
    if n <= 1 or t.is_contiguous():
        if width > 1 and t.stride(-1) != 1:
            raise ValueError(f"{name}: the elements of a row must be contiguous")
        return n, width, width
    if width > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    step = None
    span = 0
    for size, stride in zip(reversed(shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if step is None:
            step = stride
        elif stride != span:
            raise ValueError(f"{name}: the rows must be evenly spaced")
        span = stride * size
    if step < width:
        raise ValueError(f"{name}: rows overlap (an expanded tensor?)")
    return n, width, step


def _out(out, name, like, shape, dtype):
    """The output given, or a new contiguous one beside the tensor `like`, of
    `shape` (None: like's)."""
    if shape is None:
        if out is None and like.is_contiguous():
            return torch.empty_like(like, dtype=dtype)
        shape = like.shape
    if out is None:
        return like.new_empty(shape, dtype=dtype)
    if out.shape != shape or out.dtype != dtype:
        raise ValueError(f"{name}: expected {tuple(shape)} of {dtype}, got {tuple(out.shape)} of {out.dtype}")
    return out


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None or t.numel() == 0 else t.data_ptr()


def _scratch(nbytes: int, device) -> Optional[torch.Tensor]:
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def sequence_status_sync(stream=None):
    """recis_sequence_status_sync: waits for the stream and raises what earlier
    sequence calls on its device found."""
    s = torch.cuda.current_stream() if stream is None else stream
    with torch.cuda.device(s.device):
        _r._check(_r.load().recis_sequence_status_sync(s.cuda_stream), "recis_sequence_status_sync")


# ------------------------------------------------------------------ dense embedding
def embed_lookup(weight: torch.Tensor, tokens: torch.Tensor, scale: float = 1.0, padding: int = NO_TOKEN,
                 out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """recis_embed_lookup: scale * weight[tokens], shape tokens.shape + [D]; the
    padding token reads as zeros.  out_dtype: weight's by default."""
    if weight.dim() != 2 or not weight.is_contiguous():
        raise ValueError("weight: expected a contiguous [V, D] tensor")
    wt = _type(weight, "weight")
    tokens = _int64(tokens, "tokens")
    V, D = weight.shape
    if _elsewhere(stream, weight, tokens, out):
        with _on(stream, weight):
            return embed_lookup(weight, tokens, scale, padding, out_dtype, out)
    dev = weight.device
    out = _out(out, "out", weight, (*tokens.shape, D), out_dtype or (weight.dtype if out is None else out.dtype))
    ot = _type(out, "out")
    _, _, stride = _rows(out, "out", D)
    _r._check(_r.load().recis_embed_lookup(weight.data_ptr(), wt, V, D, _ptr(tokens), tokens.numel(), scale, padding,
                                           _ptr(out), ot, stride, _raw(dev)), "recis_embed_lookup")
    return out


def embed_grad(tokens: torch.Tensor, grad_out: torch.Tensor, num_rows: int, scale: float = 1.0,
               padding: int = NO_TOKEN, dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
               accumulate: bool = False, stream=None) -> torch.Tensor:
    """recis_embed_grad: the gradient [num_rows, D] of embed_lookup's weight, of
    `dtype` (fp32 by default).  accumulate: added to `out`."""
    gt = _type(grad_out, "grad_out")
    tokens = _int64(tokens, "tokens")
    if grad_out.shape[:-1] != tokens.shape:
        raise ValueError(f"grad_out: expected {tuple(tokens.shape)} + [D], got {tuple(grad_out.shape)}")
    if accumulate and out is None:
        raise ValueError("accumulate needs the tensor to add to (out)")
    _, D, grad_stride = _rows(grad_out, "grad_out")
    if _elsewhere(stream, grad_out, tokens, out):
        with _on(stream, grad_out):
            return embed_grad(tokens, grad_out, num_rows, scale, padding, dtype, out, accumulate)
    L, dev, n = _r.load(), grad_out.device, tokens.numel()
    out = _out(out, "out", grad_out, (num_rows, D), dtype or (torch.float32 if out is None else out.dtype))
    ot = _type(out, "out")
    if not out.is_contiguous():
        raise ValueError("out: expected a contiguous tensor")
    nb = ctypes.c_int64()
    _r._check(L.recis_embed_grad_workspace(n, num_rows, D, ctypes.byref(nb)), "recis_embed_grad_workspace")
    ws = _scratch(nb.value, dev)
    _r._check(L.recis_embed_grad(_ptr(tokens), n, _ptr(grad_out), gt, grad_stride, num_rows, D, scale, padding,
                                 1 if accumulate else 0, out.data_ptr(), ot, _ptr(ws), nb.value, _raw(dev)),
              "recis_embed_grad")
    return out


# ------------------------------------------------------------------ layer norm
def _norm_params(weight, bias, D):
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is not None and (t.shape != (D,) or not t.is_contiguous()):
            raise ValueError(f"{name}: expected a contiguous [{D}] tensor, got {tuple(t.shape)}")
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise TypeError(f"weight and bias differ in type: {weight.dtype}, {bias.dtype}")
    t = weight if weight is not None else bias
    return 0 if t is None else _type(t, "weight")


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               eps: float = 1e-5, out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
               stream=None):
    """recis_layer_norm over the last dimension: (y, mean, rstd), mean and rstd
    fp32 of x.shape[:-1].  out_dtype: x's by default."""
    xt = _type(x, "x")
    M, D, xs = _rows(x, "x")
    wt = _norm_params(weight, bias, D)
    if _elsewhere(stream, x, weight, bias, out):
        with _on(stream, x):
            return layer_norm(x, weight, bias, eps, out_dtype, out)
    dev = x.device
    y = _out(out, "out", x, None, out_dtype or (x.dtype if out is None else out.dtype))
    yt = _type(y, "out")
    ys = _rows(y, "out", D)[2]
    mean = x.new_empty(x.shape[:-1], dtype=torch.float32)
    rstd = torch.empty_like(mean)
    _r._check(_r.load().recis_layer_norm(_ptr(x), xt, xs, M, D, _ptr(weight), _ptr(bias), wt, eps, _ptr(y), yt, ys,
                                         _ptr(mean), _ptr(rstd), _raw(dev)), "recis_layer_norm")
    return y, mean, rstd


def layer_norm_backward(grad_y: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                        grad_x: Optional[torch.Tensor] = None, stream=None):
    """recis_layer_norm_backward: (grad_x, grad_weight, grad_bias); the last two
    of weight's and bias's type, None where weight or bias is None."""
    xt, yt = _type(x, "x"), _type(grad_y, "grad_y")
    M, D, xs = _rows(x, "x")
    if grad_y.shape != x.shape:
        raise ValueError(f"grad_y: expected {tuple(x.shape)}, got {tuple(grad_y.shape)}")
    gs = _rows(grad_y, "grad_y")[2]
    wt = _norm_params(weight, bias, D)
    for t, name in ((mean, "mean"), (rstd, "rstd")):
        if t.dtype != torch.float32 or t.shape != x.shape[:-1] or not t.is_contiguous():
            raise ValueError(f"{name}: expected contiguous {tuple(x.shape[:-1])} of {torch.float32}")
    if _elsewhere(stream, x, grad_y, mean, rstd, weight, bias, grad_x):
        with _on(stream, x):
            return layer_norm_backward(grad_y, x, mean, rstd, weight, bias, grad_x)
    L, dev = _r.load(), x.device
    gx = _out(grad_x, "grad_x", x, None, x.dtype)
    gxs = _rows(gx, "grad_x", D)[2]
    gw = None if weight is None else torch.empty_like(weight)
    gb = None if bias is None else torch.empty_like(bias)
    nb = ctypes.c_int64()
    _r._check(L.recis_layer_norm_backward_workspace(M, D, ctypes.byref(nb)), "recis_layer_norm_backward_workspace")
    ws = _scratch(nb.value, dev)
    _r._check(L.recis_layer_norm_backward(_ptr(grad_y), yt, gs, _ptr(x), xt, xs, M, D, _ptr(weight), wt, _ptr(mean),
                                          _ptr(rstd), _ptr(gx), gxs, _ptr(gw), _ptr(gb), _ptr(ws), nb.value,
                                          _raw(dev)), "recis_layer_norm_backward")
    return gx, gw, gb


# ------------------------------------------------------------------ attention
_ATTEND_TYPES = {torch.bfloat16: 1, torch.float16: 2}


def _heads(t: torch.Tensor, name: str, dtype, shape=None):
    """(row stride, head stride) of a [rows, heads, D] tensor."""
    if t.dim() != 3 or (shape is not None and t.shape != shape):
        raise ValueError(f"{name}: expected {'[rows, heads, D]' if shape is None else tuple(shape)}, "
                         f"got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    T, H, D = t.shape
    a, b, c = t.stride()
    if c != 1 and D > 1:
        raise ValueError(f"{name}: the elements of a head must be contiguous")
    return (a if T > 1 else H * D), (b if H > 1 else D)


def _written(t: torch.Tensor, name: str, strides):
    """Refuses an output whose rows or heads share memory."""
    T, H, D = t.shape
    a, b = strides
    apart = (T <= 1 or H <= 1 or (b >= D and a >= (H - 1) * b + D) or (a >= D and b >= (T - 1) * a + D))
    if t.numel() and not (apart and (T <= 1 or a >= D) and (H <= 1 or b >= D)):
        raise ValueError(f"{name}: rows or heads share memory")


def _attend_args(q, k, v, q_offsets, k_offsets, max_q, max_k, scale, key_mask):
    dtype = q.dtype
    kind = _type(q, "q", _ATTEND_TYPES)
    qs, qh = _heads(q, "q", dtype)
    ks, kh = _heads(k, "k", dtype)
    vs, vh = _heads(v, "v", dtype, k.shape)
    Tq, Hq, D = q.shape
    Tk, Hkv, Dk = k.shape
    if Dk != D or Hkv == 0 or Hq == 0 or Hq % Hkv:
        raise ValueError(f"k: heads of {tuple(k.shape)} do not fit q's {tuple(q.shape)}")
    n = q_offsets.numel()
    for t, name in ((q_offsets, "q_offsets"), (k_offsets, "k_offsets")):
        if _int64(t, name).dim() != 1 or n < 1 or t.numel() != n:
            raise ValueError(f"{name}: expected [B + 1] offsets, got {tuple(t.shape)}")
    if key_mask is not None and (key_mask.dtype not in (torch.bool, torch.uint8) or key_mask.shape != (Tk,)
                                 or not key_mask.is_contiguous()):
        raise ValueError(f"key_mask: expected a contiguous [{Tk}] bool tensor")
    return AttendArgs(kind, D, Hq, Hkv, n - 1, Tq, Tk, max_q, max_k, float(D) ** -0.5 if scale is None else scale,
                      q_offsets.data_ptr(), k_offsets.data_ptr(), _ptr(key_mask), _ptr(q), _ptr(k), _ptr(v),
                      qs, qh, ks, kh, vs, vh)


def attend(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_offsets: torch.Tensor, k_offsets: torch.Tensor,
           max_q: int, max_k: int, scale: Optional[float] = None, key_mask: Optional[torch.Tensor] = None,
           out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, stream=None):
    """recis_attend: every bag's queries (rows q_offsets[b] .. q_offsets[b+1] of q
    [Tq, Hq, D]) over the bag's keys (rows k_offsets[b] .. of k and v
    [Tk, Hkv, D]); (out [Tq, Hq, D], lse fp32 [Tq, Hq]).  scale: 1/sqrt(D) by
    default; key_mask: bool [Tk], False keys take no part.  Rows of no bag are
    left as they are in `out` and `lse` where given, undefined in new ones."""
    a = _attend_args(q, k, v, q_offsets, k_offsets, max_q, max_k, scale, key_mask)
    if _elsewhere(stream, q, k, v, q_offsets, k_offsets, key_mask, out, lse):
        with _on(stream, q):
            return attend(q, k, v, q_offsets, k_offsets, max_q, max_k, scale, key_mask, out, lse)
    L, dev = _r.load(), q.device
    given = out is not None
    out = _out(out, "out", q, None, q.dtype)
    a.out_stride, a.out_head_stride = _heads(out, "out", q.dtype)
    if given:
        _written(out, "out", (a.out_stride, a.out_head_stride))
    lse = _out(lse, "lse", q, q.shape[:2], torch.float32)
    if not lse.is_contiguous():
        raise ValueError("lse: expected a contiguous tensor")
    a.out, a.lse = _ptr(out), _ptr(lse)
    nb, ref = ctypes.c_int64(), ctypes.byref(a)
    _r._check(L.recis_attend_workspace(ref, 0, ctypes.byref(nb)), "recis_attend_workspace")
    ws = _scratch(nb.value, dev)
    _r._check(L.recis_attend(ref, _ptr(ws), nb.value, _raw(dev)), "recis_attend")
    return out, lse


def attend_backward(grad_out: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                    lse: torch.Tensor, q_offsets: torch.Tensor, k_offsets: torch.Tensor, max_q: int, max_k: int,
                    scale: Optional[float] = None, key_mask: Optional[torch.Tensor] = None,
                    grad_q: Optional[torch.Tensor] = None, grad_k: Optional[torch.Tensor] = None,
                    grad_v: Optional[torch.Tensor] = None, stream=None):
    """recis_attend_backward: (grad_q, grad_k, grad_v) from attend's inputs, its
    out and lse, and out's gradient.  Rows of no bag are left as they are in
    the gradients where given, undefined in new ones."""
    a = _attend_args(q, k, v, q_offsets, k_offsets, max_q, max_k, scale, key_mask)
    dtype = q.dtype
    a.out_stride, a.out_head_stride = _heads(out, "out", dtype, q.shape)
    a.grad_out_stride, a.grad_out_head_stride = _heads(grad_out, "grad_out", dtype, q.shape)
    if lse.dtype != torch.float32 or lse.shape != q.shape[:2] or not lse.is_contiguous():
        raise ValueError(f"lse: expected contiguous {tuple(q.shape[:2])} of {torch.float32}")
    if _elsewhere(stream, q, k, v, out, lse, grad_out, q_offsets, k_offsets, key_mask, grad_q, grad_k, grad_v):
        with _on(stream, q):
            return attend_backward(grad_out, q, k, v, out, lse, q_offsets, k_offsets, max_q, max_k, scale, key_mask,
                                   grad_q, grad_k, grad_v)
    L, dev = _r.load(), q.device
    grads, strides = [], []
    for t, name, like in ((grad_q, "grad_q", q), (grad_k, "grad_k", k), (grad_v, "grad_v", v)):
        g = _out(t, name, like, None, dtype)
        st = _heads(g, name, dtype)
        if t is not None:
            _written(g, name, st)
        grads.append(g)
        strides.append(st)
    a.out, a.lse, a.grad_out = _ptr(out), _ptr(lse), _ptr(grad_out)
    a.grad_q, a.grad_k, a.grad_v = _ptr(grads[0]), _ptr(grads[1]), _ptr(grads[2])
    ((a.grad_q_stride, a.grad_q_head_stride), (a.grad_k_stride, a.grad_k_head_stride),
     (a.grad_v_stride, a.grad_v_head_stride)) = strides
    nb, ref = ctypes.c_int64(), ctypes.byref(a)
    _r._check(L.recis_attend_workspace(ref, 1, ctypes.byref(nb)), "recis_attend_workspace")
    ws = _scratch(nb.value, dev)
    _r._check(L.recis_attend_backward(ref, _ptr(ws), nb.value, _raw(dev)), "recis_attend_backward")
    return tuple(grads)


# ------------------------------------------------------------------ attention pooling of a table's bags
class SequenceAttention:
    """Attention pooling of a table's bags, beside lookup_pooled's SUM and MEAN:
    each bag's rows are the sequence that the bag's candidates attend to.

    The table's rows of D = 2 * kv_heads * head_dim hold a key and a value half.
    A step looks the bags' keys up (Table.lookup_pooled, unpooled rows),
    normalises the rows (layer norm, fp32 rows to `dtype`), looks the
    candidates' tokens up in `query_weight` [V, heads * head_dim], scaled, and
    attends.  backward returns the dense gradients and applies the rows'
    gradients to the table with its optimiser (Table.backward_update)."""

    def __init__(self, table: _r.Table, query_weight: torch.Tensor, heads: int, kv_heads: int,
                 norm_weight: torch.Tensor, norm_bias: torch.Tensor, query_scale: float = 1.0, eps: float = 1e-5,
                 dtype: torch.dtype = torch.bfloat16):
        if table.dim % (2 * kv_heads) or query_weight.dim() != 2 or (
                query_weight.shape[1] != heads * (table.dim // (2 * kv_heads))):
            raise ValueError(f"rows of {table.dim} hold no key and value of {kv_heads} heads that "
                             f"{heads} heads of {tuple(query_weight.shape)} attend to")
        self.table, self.query_weight = table, query_weight
        self.norm_weight, self.norm_bias = norm_weight, norm_bias
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, table.dim // (2 * kv_heads)
        self.query_scale, self.eps, self.dtype = query_scale, eps, dtype
        self._ctx = None

    def _halves(self, x):
        """The key and the value half of rows, as [N, kv_heads, head_dim]."""
        w = self.kv_heads * self.head_dim
        return (x[:, :w].unflatten(1, (self.kv_heads, self.head_dim)),
                x[:, w:].unflatten(1, (self.kv_heads, self.head_dim)))

    def forward(self, batch: _r.Batch, keys: torch.Tensor, bag_offsets: torch.Tensor, tokens: torch.Tensor,
                token_offsets: torch.Tensor, max_tokens: int, max_keys: int,
                key_mask: Optional[torch.Tensor] = None) -> torch.Tensor:
        """keys int64[N] in bags bag_offsets int64[B+1]; tokens int64[T] in bags
        token_offsets int64[B+1]; returns [T, heads, head_dim], zeros for tokens
        of no bag or of a bag that passes max_tokens or max_keys.  keys and
        bag_offsets stay unchanged until backward.  A lookup that the table rejects
        (Table.status_sync) leaves the answers and the dense gradients undefined, and
        the table's rows as they were.  What a forward keeps for its
        backward is let go by the backward, or by the next forward.  Runs on the
        current stream of the tensors' device, the table's."""
        if _elsewhere(None, keys, bag_offsets, tokens, token_offsets, key_mask, self.query_weight, self.norm_weight,
                      self.norm_bias):
            with _on(None, keys):
                return self.forward(batch, keys, bag_offsets, tokens, token_offsets, max_tokens, max_keys, key_mask)
        B = bag_offsets.numel() - 1
        # (a row at least: a lookup without an output array is refused, and bags may all be empty)
        rows = torch.empty((max(keys.numel(), 1), self.table.dim), dtype=torch.float32, device=keys.device)
        self.table.lookup_pooled(batch, keys, bag_offsets, 1, B, unpooled_out=rows)
        rows = rows[:keys.numel()]
        kv, mean, rstd = layer_norm(rows, self.norm_weight, self.norm_bias, self.eps, self.dtype)
        q = embed_lookup(self.query_weight, tokens, self.query_scale, out_dtype=self.dtype)
        q = q.view(-1, self.heads, self.head_dim)
        k, v = self._halves(kv)
        bags = (token_offsets, bag_offsets, max_tokens, max_keys)
        out, lse = attend(q, k, v, *bags, key_mask=key_mask, out=torch.zeros_like(q))
        self._ctx = (batch, rows, mean, rstd, tokens, q, kv, out, lse, bags, key_mask)
        return out

    def backward(self, grad_out: torch.Tensor):
        """(grad of query_weight, of norm_weight, of norm_bias); the table's rows
        are updated.  Keys and tokens of no bag, or of a bag that passes max_keys or
        max_tokens, have gradients of zero."""
        if self._ctx is None:
            raise RuntimeError("backward before forward")
        if _elsewhere(None, grad_out, self._ctx[1]):
            with _on(None, grad_out):
                return self.backward(grad_out)
        batch, rows, mean, rstd, tokens, q, kv, out, lse, bags, key_mask = self._ctx
        k, v = self._halves(kv)
        # attend_backward leaves the rows of no bag, and of a bag it reports, as they
        # were; all rows go on into the sums and the table
        dkv, dq = torch.zeros_like(kv), torch.zeros_like(q)
        dk, dv = self._halves(dkv)
        attend_backward(grad_out, q, k, v, out, lse, *bags, key_mask=key_mask, grad_q=dq, grad_k=dk, grad_v=dv)
        drows, dw, db = layer_norm_backward(dkv, rows, mean, rstd, self.norm_weight, self.norm_bias)
        self.table.backward_update(batch, grad_unpooled=drows)
        dquery = embed_grad(tokens, dq.flatten(1), self.query_weight.shape[0], self.query_scale)
        self._ctx = None
        return dquery, dw, db
