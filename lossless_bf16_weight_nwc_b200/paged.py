"""What a decode layer does between its compressed projections: per-head norms
with the position rotation, a paged key/value cache, and attention over it for
a batch whose sequences may share prefixes.

A layer's step with a fused q/k/v matrix (`CompressedMatrix.compress_fused`):

    y = wqkv.gemv(x)                                   # FP32 [rows, ...]
    q, k, v = (t.unflatten(-1, (-1, dim)) for t in wqkv.split(y))
    q = cache.append(batch, k, v, q=q, freq=freq, q_weight=qn, k_weight=kn)
    o = cache.attend(batch, q)                         # BF16 [rows, heads, dim]
    y = wo.gemv(o.flatten(1))

`AttentionBlock` holds those pieces for one layer.  All of it runs in libnwc's
kernels; lengths and tables stay on the device, so a step can be captured into a
CUDA graph and replayed as they change.  Nothing here has a gradient: inputs
that require one are refused while gradients are recorded, as are those with a
forward-mode tangent.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch
from torch.autograd import forward_ad

from . import _lib

# The calls' structures are packed here and passed as addresses, which takes half as
# long as filling _lib's ctypes structures: for one token a call is bound by the host.
_RAW = ctypes.CDLL(_lib.LIB_PATH)
_P, _I = ctypes.c_void_p, ctypes.c_int32
_RAW.nwc_qk_norm_rope.argtypes = [_P] * 4 + [_I] * 4 + [_P, _I, _P, _P]
_RAW.nwc_kv_append.argtypes = [_P] * 4 + [_I] + [_P] * 4
_RAW.nwc_kv_attention.argtypes = [_P, _P, _P, _I, ctypes.c_float, _P, _P, _P, ctypes.c_uint64, _P]
_check = _lib._check
_Tensor, _grad_enabled, _empty = torch.Tensor, torch.is_grad_enabled, torch.empty_strided
_bfloat16 = torch.bfloat16
_TYPES = {torch.bfloat16: _lib.NWC_TYPE_BF16, torch.float32: _lib.NWC_TYPE_F32}
_HEADS = ctypes.sizeof(_lib.nwc_heads)
_ROPE = ctypes.sizeof(_lib.nwc_rope)
_pack_heads = struct.Struct("@IIPqq").pack
_pack_rope = struct.Struct("@IiiIPPPf0P").pack
assert len(_pack_heads(0, 0, 0, 0, 0)) == _HEADS
assert len(_pack_rope(0, 0, 0, 0, 0, 0, 0, 0)) == _ROPE
_POSITIONS = (torch.int32, torch.int64)
_BF16 = (torch.bfloat16,)
_F64 = (torch.float64,)


def rope_frequencies(rotary_dim: int, theta: float = 10000.0, device="cuda",
                     factor: float = 1.0, low_freq_factor: float = 1.0,
                     high_freq_factor: float = 4.0, original_positions: int = 8192):
    """FP64 [rotary_dim / 2] radians a position, theta^(-2i / rotary_dim).  factor
    > 1 stretches them as Llama-3.1's configuration does: frequencies of fewer
    than low_freq_factor turns over original_positions are divided by factor,
    those of more than high_freq_factor kept, those between interpolated."""
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("rotary_dim: an even number")
    f = theta ** (-torch.arange(0, rotary_dim, 2, dtype=torch.float64) / rotary_dim)
    if factor != 1.0:
        turns = original_positions * f / (2 * math.pi)
        keep = ((turns - low_freq_factor) / (high_freq_factor - low_freq_factor)).clamp(0, 1)
        f = f * (keep + (1 - keep) / factor)
    return f.to(device)


def _no_grad(*tensors) -> None:
    if _grad_enabled():
        for t in tensors:
            if t is not None and isinstance(t, _Tensor) and t.requires_grad:
                raise ValueError("a tensor requires a gradient, which these kernels do not "
                                 "give; call under torch.no_grad()")
    # (The level saves asking every tensor where no dual level is open.)
    if getattr(forward_ad, "_current_level", 0) >= 0:
        for t in tensors:
            if isinstance(t, _Tensor) and forward_ad.unpack_dual(t).tangent is not None:
                raise ValueError("a tensor has a tangent, a forward-mode gradient that these "
                                 "kernels do not carry on; unpack it first")


def _heads(t, what: str, shape, device, dtypes=_TYPES, wide: bool = False,
           output: bool = False) -> bytes:
    """The C view of a tensor [tokens, heads, dim] with any strides but a
    contiguous last dimension; wide: moved 16 bytes at a time; output: no two
    elements at one place."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{what}: expected a torch.Tensor, got {type(t).__name__}")
    dtype = t.dtype
    if dtype not in dtypes:
        raise TypeError(f"{what}: dtype {dtype}, expected one of {[str(d) for d in dtypes]}")
    if t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    ts, hs, es = t.stride()
    if es != 1:
        raise ValueError(f"{what}: the last dimension must be contiguous")
    if t.device != device:
        raise ValueError(f"{what}: on {t.device}, expected {device}")
    tokens, heads, dim = shape
    if tokens < 2:
        ts = 0
    if heads < 2:
        hs = 0
    at = t.data_ptr()
    if wide and tokens and (at % 16 or ts % 8 or hs % 8):
        raise ValueError(f"{what}: needs 16-byte alignment and strides of multiples of 8 elements")
    if output and tokens and not (
            (heads < 2 or hs >= dim) and (tokens < 2 or ts >= dim) and
            (heads < 2 or tokens < 2 or ts >= (heads - 1) * hs + dim or
             hs >= (tokens - 1) * ts + dim)):
        raise ValueError(f"{what}: its elements overlap")
    return _pack_heads(_HEADS, _TYPES[dtype], at, ts, hs)


def _meet(a, b) -> bool:
    """Whether two tensors [tokens, heads, dim] hold a byte in common; told apart where
    their strides are the same (views of one tensor), else taken to be so."""
    steps = []
    for d in (0, 1):   # (step in bytes, the most that b is steps behind a, and before it)
        n, m = a.shape[d], b.shape[d]
        s, t = a.stride(d) * a.element_size(), b.stride(d) * b.element_size()
        s, t = (t if n < 2 else s), (s if m < 2 else t)
        if s != t:
            return True
        if s and (n > 1 or m > 1):
            steps.append((s, n - 1, m - 1))
    steps.sort(reverse=True)
    wide, width = a.shape[2] * a.element_size(), b.shape[2] * b.element_size()

    def any_at(apart, k):   # b's first byte lies `apart` behind a's
        if k == len(steps):
            return -width < apart < wide
        # The steps k + 1, ... change `apart` by -down to up.
        down = sum(s * n for s, n, _ in steps[k + 1:])
        up = sum(s * m for s, _, m in steps[k + 1:])
        s, n, m = steps[k]
        first = max(-n, -((apart + up + width - 1) // s))
        last = min(m, (down + wide - 1 - apart) // s)
        return any(any_at(apart + i * s, k + 1) for i in range(first, last + 1))

    return any_at(b.data_ptr() - a.data_ptr(), 0)


def _bytes(t):
    """A tensor's first byte and the one behind its last."""
    at, last = t.data_ptr(), 0
    for n, s in zip(t.shape, t.stride()):
        if n == 0:
            return at, at
        last += (n - 1) * s
    return at, at + (last + 1) * t.element_size()


def _apart(out, what: str, source, *others) -> None:
    """Refuses an output in memory of another tensor of its call, whose kernels read
    while they write; `source` (an input of its shape) may be the output itself, but
    not in a second part of the call."""
    at, end = _bytes(out)
    for i, t in enumerate((source, *others)):
        if t is None:
            continue
        first, behind = _bytes(t)
        if behind <= at or end <= first or first == behind or at == end:
            continue
        if (i == 0 and first == at and t.dtype == out.dtype and
                all(n < 2 or s == o for n, s, o in zip(t.shape, t.stride(), out.stride()))):
            continue
        if t.dim() != 3 or _meet(out, t):
            raise ValueError(f"{what}: overlaps another tensor of the call")


def _new(device, shape):
    """A new BF16 tensor of a shape [tokens, heads, dim], and its C view."""
    _, heads, dim = shape
    row = heads * dim
    t = _empty(shape, (row, dim, 1), dtype=_bfloat16, device=device)
    return t, _pack_heads(_HEADS, 0, t.data_ptr(), row, dim)


def _vector(t, what: str, device, n: int, dtypes) -> int:
    """The address of a contiguous vector of n elements."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{what}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype not in dtypes:
        raise TypeError(f"{what}: dtype {t.dtype}, expected one of {[str(d) for d in dtypes]}")
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{what}: expected {n} contiguous elements, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{what}: on {t.device}, expected {device}")
    return t.data_ptr()


def _rope(dim: int, device, freq, q_weight, k_weight, eps: float, interleaved: bool):
    if not 0 <= eps < math.inf:
        raise ValueError("eps: a finite number, not negative")
    n, d_freq, d_q, d_k, kind = 0, 0, 0, 0, 0
    if freq is not None:
        n = freq.numel() if isinstance(freq, torch.Tensor) else 0
        d_freq = _vector(freq, "freq", device, n, _F64)
        if 2 * n > dim or n % 4:
            raise ValueError(f"freq: {n} elements; a multiple of 4 up to {dim // 2}")
    if q_weight is not None:
        d_q = _vector(q_weight, "q_weight", device, dim, _TYPES)
        kind = _TYPES[q_weight.dtype]
    if k_weight is not None:
        if q_weight is not None and k_weight.dtype != q_weight.dtype:
            raise TypeError("q_weight and k_weight: expected one dtype")
        d_k = _vector(k_weight, "k_weight", device, dim, _TYPES)
        kind = _TYPES[k_weight.dtype]
    return _pack_rope(_ROPE, 2 * n, interleaved, kind, d_freq, d_q, d_k, eps)


class _On:
    """Makes a call's device current and, when a stream is given, that stream
    current too: what the call allocates then belongs to the stream it runs on.
    Entering gives the stream's handle."""

    def __init__(self, device, stream):
        if stream is None:
            self.context = torch.cuda.device(device)
        else:
            if not isinstance(stream, torch.cuda.Stream):
                raw = int(getattr(stream, "cuda_stream", stream))
                stream = (torch.cuda.ExternalStream(raw, device=device) if raw
                          else torch.cuda.default_stream(device))
            if stream.device != device:
                raise ValueError(f"stream: on {stream.device}, expected {device}")
            self.context = torch.cuda.stream(stream)

    def __enter__(self):
        self.context.__enter__()
        return torch.cuda.current_stream().cuda_stream

    def __exit__(self, *args):
        return self.context.__exit__(*args)


def _raw_stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# The same without building a torch.cuda.Stream (3 us less a call), and the current
# device without asking whether CUDA has been initialised.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _on(device, stream, call):
    """call(raw stream) where it should run."""
    if stream is None and _current_device() == device.index:
        return call(_raw_stream(device.index))
    with _On(device, stream) as raw:
        return call(raw)


def _cuda(t, what: str):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: expected a torch.Tensor, got {type(t).__name__}")
    if not t.is_cuda:
        raise ValueError(f"{what}: on {t.device}, expected a CUDA device")
    return t.device


def qk_norm_rope(q, k, positions, freq=None, q_weight=None, k_weight=None, eps: float = 1e-6,
                 interleaved: bool = False, out=None, stream=None):
    """(q_out, k_out): each head of q [tokens, heads, dim] and k [tokens,
    kv_heads, dim] divided by its root mean square and times its weight (where
    one is given), then rotated by positions [tokens] x freq (FP64, from
    rope_frequencies; None: no rotation) in pairs (i, i + rotary / 2), or
    (2i, 2i + 1) when interleaved.  q and k are FP32 or BF16 with any strides but
    a contiguous last dimension (views of a GEMV's result); either may be None.
    The results are BF16, or what `out` (a pair of tensors) holds: q and k
    themselves, or memory of no other tensor of the call."""
    first = q if q is not None else k
    device = _cuda(first, "q" if q is not None else "k")
    _no_grad(q, k, freq, q_weight, k_weight, *(out or ()))
    if first.dim() != 3:
        raise ValueError("q, k: expected [tokens, heads, dim]")
    tokens, heads, dim = first.shape
    if not 8 <= dim <= 256 or dim % 8:
        raise ValueError(f"dim {dim}: a multiple of 8 from 8 to 256")
    qh = None if q is None else _heads(q, "q", (tokens, heads, dim), device)
    kh, kv_heads = None, heads
    if k is not None:
        if not isinstance(k, torch.Tensor) or k.dim() != 3:
            raise ValueError("k: expected a tensor [tokens, heads, dim]")
        kv_heads = k.shape[1]
        kh = _heads(k, "k", (tokens, kv_heads, dim), device, (first.dtype,))
    rope = _rope(dim, device, freq, q_weight, k_weight, eps, interleaved)
    at = _vector(positions, "positions", device, tokens, _POSITIONS)

    def call(raw):
        qo = ko = qoh = koh = None
        if out is None:
            if q is not None:
                qo, qoh = _new(device, (tokens, heads, dim))
            if k is not None:
                ko, koh = _new(device, (tokens, kv_heads, dim))
        else:
            qo, ko = out
            if (qo is None) != (q is None) or (ko is None) != (k is None):
                raise ValueError("out: a pair of tensors for q and k, None where the input is "
                                 "None")
            if q is not None:
                qoh = _heads(qo, "out[0]", (tokens, heads, dim), device, output=True)
            if k is not None:
                koh = _heads(ko, "out[1]", (tokens, kv_heads, dim), device,
                             _TYPES if q is None else (qo.dtype,), output=True)
            read = (positions, freq, q_weight, k_weight)
            if q is not None:
                _apart(qo, "out[0]", q, k, ko, *read)
            if k is not None:
                _apart(ko, "out[1]", k, q, *read)
        if tokens:
            _check(_RAW.nwc_qk_norm_rope(qh, kh, qoh, koh, tokens, heads, kv_heads, dim, at,
                                         positions.dtype == torch.int64, rope, raw),
                   "nwc_qk_norm_rope")
        return qo, ko

    return _on(device, stream, call)


class PagedBatch:
    """The sequences of a call and where their tokens are.

    block_table  int32 [sequences, width]: sequence b's own pages, in order.
    seq_lens     int32 [sequences]: own tokens, a call's new ones among them.
    q_lens       int32 [sequences] or None: how many of a sequence's rows are
                 new tokens, from its first row; the others are padding.  New
                 tokens that seq_lens does not count (the first, where it counts
                 fewer) have no place: they are not appended, their q still turns
                 at its position (the prefix's length plus an index below zero)
                 and sees the prefix alone.
    prefix_table int32 [groups, width], prefix_lens int32 [groups], group_start
                 int32 [groups + 1]: sequences group_start[g] up to
                 group_start[g + 1] share prefix g, which comes before their own
                 tokens; all three or none, no more groups than sequences (groups
                 may be empty).

    All on one CUDA device; their contents are read when a kernel runs, so they
    may be changed in place between calls.  Entries behind a sequence's last page
    are not read."""

    def __init__(self, block_table, seq_lens, q_lens=None, prefix_table=None, prefix_lens=None,
                 group_start=None):
        self.device = _cuda(block_table, "block_table")
        self._keep = (block_table, seq_lens, q_lens, prefix_table, prefix_lens, group_start)
        i32 = (torch.int32,)
        table = self._table(block_table, "block_table")
        self.sequences = block_table.shape[0]
        lens = _vector(seq_lens, "seq_lens", self.device, self.sequences, i32)
        fresh = None if q_lens is None else _vector(q_lens, "q_lens", self.device,
                                                    self.sequences, i32)
        if len({x is None for x in (prefix_table, prefix_lens, group_start)}) != 1:
            raise ValueError("prefix_table, prefix_lens, group_start: all three or none")
        self.groups = 0
        far = (0, None, None, 0, 0, None)
        if prefix_table is not None and prefix_table.shape[0]:
            shared = self._table(prefix_table, "prefix_table")
            self.groups = prefix_table.shape[0]
            if self.groups > self.sequences:
                raise ValueError(f"{self.groups} groups of {self.sequences} sequences")
            far = (self.groups,
                   _vector(group_start, "group_start", self.device, self.groups + 1, i32),
                   *shared,
                   _vector(prefix_lens, "prefix_lens", self.device, self.groups, i32))
        self._fields = (*table, lens, fresh, *far)
        self._views, self._structs = {}, []

    def _table(self, t, what: str):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.dim() != 2:
            raise TypeError(f"{what}: expected an int32 tensor [rows, width]")
        if t.device != self.device:
            raise ValueError(f"{what}: on {t.device}, expected {self.device}")
        if t.stride(1) != 1 and t.shape[1] > 1:
            raise ValueError(f"{what}: its rows must be contiguous")
        return t.data_ptr(), t.stride(0) if t.shape[0] > 1 else 0, t.shape[1]

    def _view(self, rows: int):
        """The address of the C view for calls of `rows` rows in all."""
        view = self._views.get(rows)
        if view is None:
            chunk = rows // self.sequences if self.sequences else 1
            if chunk < 1 or (chunk * self.sequences != rows):
                raise ValueError(f"{rows} rows for {self.sequences} sequences: the same number, "
                                 "at least one, for each")
            if rows > 1 << 24:
                raise ValueError(f"{rows} rows; a call takes up to 2^24")
            fields = _lib.nwc_kv_batch(ctypes.sizeof(_lib.nwc_kv_batch), self.sequences, chunk,
                                       *self._fields)
            self._structs.append(fields)
            view = self._views[rows] = ctypes.addressof(fields)
        return view


class PagedKV:
    """A paged key/value cache over the caller's pages: k_pages and v_pages BF16
    [pages, page_size, kv_heads, dim] on one CUDA device, the last dimension
    contiguous, other strides multiples of 8 elements, 16-byte aligned (a
    permuted view gives pages that keep each head's tokens together).
    page_size: a power of two, 8 or more.

    Calls run on the device's current torch stream, or the stream given; append
    and attend on the same pages must be ordered by the caller."""

    def __init__(self, k_pages, v_pages):
        self.device = _cuda(k_pages, "k_pages")
        for t, what in ((k_pages, "k_pages"), (v_pages, "v_pages")):
            if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or t.dim() != 4:
                raise TypeError(f"{what}: expected a BF16 tensor [pages, page_size, kv_heads, dim]")
            if t.device != self.device or t.shape != k_pages.shape:
                raise ValueError(f"{what}: {tuple(t.shape)} on {t.device}, expected "
                                 f"{tuple(k_pages.shape)} on {self.device}")
        _no_grad(k_pages, v_pages)
        self.k_pages, self.v_pages = k_pages, v_pages
        self.pages, self.page_size, self.kv_heads, self.dim = k_pages.shape
        if self.page_size < 8 or self.page_size & (self.page_size - 1):
            raise ValueError(f"page_size {self.page_size}: a power of two, 8 or more")
        if not 8 <= self.dim <= 256 or self.dim % 8:
            raise ValueError(f"dim {self.dim}: a multiple of 8 from 8 to 256")
        if self.pages < 1 or self.kv_heads < 1:
            raise ValueError("k_pages: no pages")
        strides = []
        for t, what in ((k_pages, "k_pages"), (v_pages, "v_pages")):
            st = [s if n > 1 else 8 for s, n in zip(t.stride(), t.shape)]
            if t.stride(3) != 1 or any(s % 8 or s < 8 for s in st[:3]) or t.data_ptr() % 16:
                raise ValueError(f"{what}: needs a contiguous last dimension, other strides of "
                                 "multiples of 8 elements, and 16-byte alignment")
            strides += st[:3]
        with torch.cuda.device(self.device):
            self._error = torch.zeros(1, dtype=torch.int32, device=self.device)
            torch.cuda.current_stream().synchronize()  # zero before any stream's kernel
        self._view = _lib.nwc_kv_cache(ctypes.sizeof(_lib.nwc_kv_cache), self.page_size,
                                       self.kv_heads, self.dim, self.pages, k_pages.data_ptr(),
                                       v_pages.data_ptr(), *strides, self._error.data_ptr())
        self._at = ctypes.addressof(self._view)
        self._workspace = {}

    def device_error(self, stream=None) -> tuple[int, int]:
        """(status, raw word) of this cache's device error word (read and cleared):
        bit 1 a bounded wait gave up, bit 4 a table or length named a page that is
        not there."""
        with torch.cuda.device(self.device):
            return _lib.nwc_kv_get_error(self._view, stream)

    def _rows(self, batch, t, what: str):
        if not isinstance(batch, PagedBatch):
            raise TypeError(f"batch: expected a PagedBatch, got {type(batch).__name__}")
        if batch.device != self.device:
            raise ValueError(f"batch: on {batch.device}, expected {self.device}")
        if not isinstance(t, torch.Tensor) or t.dim() != 3:
            raise ValueError(f"{what}: expected a tensor [rows, heads, dim]")
        return t.shape[0], batch._view(t.shape[0])

    def append(self, batch: PagedBatch, k, v, q=None, freq=None, q_weight=None, k_weight=None,
               eps: float = 1e-6, interleaved: bool = False, q_out=None, stream=None):
        """Appends the new tokens' k (normed and rotated as in qk_norm_rope, at the
        position of its token: the prefix's length plus its own index) and v, both
        [rows, kv_heads, dim], to their sequences' pages, and returns q [rows,
        heads, dim], normed and rotated likewise, as BF16 (None without q).  Inputs
        FP32 or BF16, one type, with any strides but a contiguous last dimension.
        seq_lens counts the new tokens already.  Padding rows are not appended,
        their q is zero.  q_out: q itself, or memory of no other tensor of the call
        or the cache; k and v may lie in pages, but not where the call appends."""
        rows, view = self._rows(batch, k, "k")
        _no_grad(q, k, v, freq, q_weight, k_weight, q_out, self.k_pages, self.v_pages)
        device = self.device
        shape = (rows, self.kv_heads, self.dim)
        kh = _heads(k, "k", shape, device)
        same = (k.dtype,)
        vh = _heads(v, "v", shape, device, same)
        heads, qh = 1, None
        if q is not None:
            if not isinstance(q, torch.Tensor) or q.dim() != 3:
                raise ValueError("q: expected a tensor [rows, heads, dim]")
            heads = q.shape[1]
            shape = (rows, heads, self.dim)
            qh = _heads(q, "q", shape, device, same)
        elif q_out is not None:
            raise ValueError("q_out: given without q")
        rope = _rope(self.dim, device, freq, q_weight, k_weight, eps, interleaved)

        def call(raw, q_out=q_out, qoh=None):
            if q_out is not None:
                qoh = _heads(q_out, "q_out", shape, device, _BF16, output=True)
                _apart(q_out, "q_out", q, k, v, freq, q_weight, k_weight, self.k_pages,
                       self.v_pages, *batch._keep)
            elif q is not None:
                q_out, qoh = _new(device, shape)
            if rows:
                _check(_RAW.nwc_kv_append(self._at, view, qh, qoh, heads, kh, vh, rope, raw),
                       "nwc_kv_append")
            return q_out

        return _on(device, stream, call)

    def attend(self, batch: PagedBatch, q, scale: float | None = None, out=None,
               return_lse: bool = False, stream=None):
        """softmax(scale q K^T) V for q BF16 [rows, heads, dim] (heads a multiple of
        kv_heads; dim 64 or 128; scale None: 1 / sqrt(dim)): each row sees its
        prefix and its sequence's own tokens up to itself.  BF16 of q's shape;
        with return_lse also FP32 [rows, heads], the logarithm of the sum of
        exponentials.  A row that sees nothing, and a padding row, is zero (-inf).
        out: q itself, or memory of no other tensor of the call or the cache."""
        rows, view = self._rows(batch, q, "q")
        _no_grad(q, out, self.k_pages, self.v_pages)
        if self.dim not in (64, 128):
            raise ValueError(f"dim {self.dim}: attention takes heads of 64 or 128")
        heads = q.shape[1]
        if heads < 1 or heads % self.kv_heads:
            raise ValueError(f"q: {heads} heads, expected a multiple of {self.kv_heads}")
        shape = (rows, heads, self.dim)
        qh = _heads(q, "q", shape, self.device, _BF16, wide=True)
        if scale is None:
            scale = self.dim ** -0.5

        def call(raw, out=out):
            if out is None:
                out, oh = _new(self.device, shape)
            else:
                oh = _heads(out, "out", shape, self.device, _BF16, wide=True, output=True)
                _apart(out, "out", q, self.k_pages, self.v_pages, *batch._keep)
            lse = torch.empty((rows, heads), dtype=torch.float32,
                              device=self.device) if return_lse else None
            if rows:
                key = (rows, batch.sequences, batch.groups, heads)
                need = self._workspace.get(key)
                if need is None:
                    need = _lib.nwc_kv_attention_workspace(
                        self._view, _lib.nwc_kv_batch.from_address(view), heads)
                    self._workspace[key] = need
                # From torch's allocator on the call's stream: calls on different
                # streams, and captured graphs, each have their own.
                ws = torch.empty(need, dtype=torch.uint8, device=self.device)
                _check(_RAW.nwc_kv_attention(self._at, view, qh, heads, scale, oh,
                                             None if lse is None else lse.data_ptr(),
                                             ws.data_ptr(), need, raw), "nwc_kv_attention")
            return (out, lse) if return_lse else out

        return _on(self.device, stream, call)


class AttentionBlock:
    """One layer's attention over compressed projections: wqkv, a fused matrix of
    the q, k and v rows (`CompressedMatrix.compress_fused([wq, wk, wv])`), and wo.

    step(x, batch) appends x's tokens to the layer's cache and returns the output
    projection FP32 [rows, wo.rows]; q_weight and k_weight are the per-head norms
    of models that have them."""

    def __init__(self, wqkv, wo, cache: PagedKV, freq, q_weight=None, k_weight=None,
                 eps: float = 1e-6, interleaved: bool = False, scale: float | None = None):
        b = wqkv.row_splits
        width = cache.kv_heads * cache.dim
        if len(b) != 4 or b[2] - b[1] != width or b[3] - b[2] != width or b[1] % cache.dim:
            raise ValueError(f"wqkv: row splits {b} do not fit {cache.kv_heads} key heads of "
                             f"{cache.dim}")
        if wo.cols != b[1]:
            raise ValueError(f"wo: {wo.cols} columns, expected {b[1]}")
        # What attend would refuse is refused here: a step would have appended by then.
        heads = b[1] // cache.dim
        if heads < 1 or heads % cache.kv_heads:
            raise ValueError(f"wqkv: {heads} query heads, expected a multiple of {cache.kv_heads}")
        if cache.dim not in (64, 128):
            raise ValueError(f"dim {cache.dim}: attention takes heads of 64 or 128")
        if scale is not None and not abs(scale) * 1.4426950408889634 < 2.0 ** 128:
            raise ValueError("scale: a finite number, also divided by ln 2 in FP32")
        for m, what in ((wqkv, "wqkv"), (wo, "wo")):
            if m.image.device != cache.device:
                raise ValueError(f"{what}: on {m.image.device}, expected {cache.device}")
        _rope(cache.dim, cache.device, freq, q_weight, k_weight, eps, interleaved)
        self.wqkv, self.wo, self.cache, self.freq = wqkv, wo, cache, freq
        self.q_weight, self.k_weight, self.eps = q_weight, k_weight, eps
        self.interleaved, self.scale = interleaved, scale

    def step(self, x, batch: PagedBatch):
        """x BF16 [rows, wqkv.cols], 1 to 64 rows, a sequence's rows together."""
        _no_grad(x)
        dim = self.cache.dim
        q, k, v = (t.unflatten(-1, (-1, dim)) for t in self.wqkv.split(self.wqkv.gemv(x)))
        q = self.cache.append(batch, k, v, q=q, freq=self.freq, q_weight=self.q_weight,
                              k_weight=self.k_weight, eps=self.eps,
                              interleaved=self.interleaved)
        return self.wo.gemv(self.cache.attend(batch, q, scale=self.scale).flatten(1))
