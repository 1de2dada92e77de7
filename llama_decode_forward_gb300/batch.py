"""Batched decoding over CUDA tensors: the operators llm_kv_append,
llm_attend_batch, llm_kv_read (on pages in float16 or of 4-bit values),
llm_pages_update, llm_pages_compact, llm_logits_adjust and llm_logprobs of
include/llm.h.

Each class checks its tensors once, keeps them (and the C arguments made of
them) and enqueues one call of its operator whenever it is called, on the
current stream or the one given: a decoding loop writes each step's values into
the same tensors, or captures the calls into a CUDA graph.
"""
from __future__ import annotations

import ctypes
import operator

import torch

from . import binding as _b

_DTYPES = {torch.float32: _b.LLM_F32, torch.float16: _b.LLM_F16}


def _stream(stream) -> int:
    return torch.cuda.current_stream().cuda_stream if stream is None else stream


# The current device and its current stream without a Stream object (they are asked
# at every call); None where PyTorch has no such functions.
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
if _current_device is None or _current_stream is None:
    _current_device = torch.cuda.current_device
    _current_stream = lambda index: torch.cuda.current_stream(index).cuda_stream  # noqa: E731


def _torch_stream(raw: int, device):
    """The torch stream of a CUDA stream (0 and 1: the legacy default stream)."""
    return torch.cuda.default_stream(device) if raw in (None, 0, 1) else torch.cuda.ExternalStream(raw, device=device)


def _run(rc: int) -> None:
    if rc != _b.LLM_OK:
        raise _b.LlmError(rc, _b._lib.llm_last_error(None).decode())


def _tensor(name, t, dtypes, shape, device, strided=False):
    """Refuses a tensor of another type, shape, device or memory order: row
    major without gaps, or with strided=True free in its first stride."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes:
        raise TypeError(f"{name} must be a tensor of {' or '.join(str(d) for d in dtypes)}")
    if t.device.type != "cuda" or (device is not None and t.device != device):
        raise ValueError(f"{name} is on {t.device}, not on {device or 'a CUDA device'}")
    if len(t.shape) != len(shape) or any(w is not None and w != n for n, w in zip(t.shape, shape)):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    inner = t[0] if strided and t.shape[0] else t
    if not inner.is_contiguous():
        raise ValueError(f"{name} is not contiguous{' within a row' if strided else ''}")
    return t


def _int32(**sizes) -> None:
    """Refuses a size that a C int32 does not hold (ctypes would cut it off)."""
    for name, n in sizes.items():
        if not -2 ** 31 <= operator.index(n) < 2 ** 31:
            raise ValueError(f"{name} {n} is not a 32-bit integer")


def _capturing() -> bool:
    return torch.cuda.is_current_stream_capturing()


class _Owner:
    """An object with tensors of its own (own, allocated on the current stream) that its
    user may hand to any stream.  (A capture in which a stream first uses them must begin
    after the work of the stream that they were made on, as that of torch.cuda.graph
    does.)"""

    def _owns(self, own, device) -> None:
        self._own, self._index = own, device.index
        self._streams = {_current_stream(device.index)}    # the streams that own's memory waits for when it is given back
        self._free = None                                  # and what others wait for: earlier tensors there, own's fill
        if own and not _capturing():
            self._free = torch.cuda.Event()
            self._free.record(torch.cuda.current_stream(device))

    def _use_on(self, stream: int) -> None:
        if stream in self._streams:
            return
        self._streams.add(stream)
        if not self._own:
            return
        s = _torch_stream(stream, self._own[0].device)
        with torch.cuda.stream(s):
            if self._free is not None and not _capturing():
                s.wait_event(self._free)
        for t in self._own:
            t.record_stream(s)


class PagedBatch(_Owner):
    """n_seqs sequences of n_new new tokens each behind a shared prefix of
    prefix_len rows (llm_pages).  k_pages, v_pages: float16 [n_pages,
    page_size, n_kv_heads, head_dim]; page_table int32 [n_seqs, max_pages];
    lens int32 [n_seqs], the rows behind the prefix, the new ones among them.
    ``err`` (int32, one value) collects the errors seen on the device
    (LLM_PAGES_*); errors() reads it."""

    def __init__(self, k_pages, v_pages, page_table, lens, n_new: int = 1, prefix_len: int = 0, err=None):
        _int32(n_new=n_new, prefix_len=prefix_len)
        _tensor("k_pages", k_pages, (torch.float16,), (None,) * 4, None)
        self._set(k_pages, v_pages, page_table, lens, *k_pages.shape[1:], n_new, prefix_len, err)

    def _set(self, k_pages, v_pages, page_table, lens, page_size, n_kv, hd, n_new, prefix_len, err) -> None:
        dev = k_pages.device
        _tensor("v_pages", v_pages, (k_pages.dtype,), tuple(k_pages.shape), dev)
        _tensor("lens", lens, (torch.int32,), (None,), dev)
        _tensor("page_table", page_table, (torch.int32,), (lens.shape[0], None), dev)
        made = err is None
        if made:
            err = torch.zeros(1, dtype=torch.int32, device=dev)
        _tensor("err", err, (torch.int32,), (1,), dev)
        self._owns((err,) if made else (), dev)
        self.k_pages, self.v_pages, self.page_table, self.lens, self.err = k_pages, v_pages, page_table, lens, err
        self.device = dev
        n_pages = k_pages.shape[0]
        _int32(n_pages=n_pages, page_size=page_size, sequences=lens.shape[0], max_pages=page_table.shape[1])
        self.rows = lens.shape[0] * n_new
        self.struct = _b.llm_pages(n_seqs=lens.shape[0], n_new=n_new, prefix_len=prefix_len, page_size=page_size,
                                   n_pages=n_pages, max_pages=page_table.shape[1], n_kv_heads=n_kv, head_dim=hd,
                                   k_pages=k_pages.data_ptr(), v_pages=v_pages.data_ptr(),
                                   page_table=page_table.data_ptr(), lens=lens.data_ptr(), err=err.data_ptr())

    def errors(self) -> int:
        """The LLM_PAGES_* bits seen so far (waits for the device)."""
        torch.cuda.synchronize(self.device)
        return int(self.err.item())


class PagedBatchQ4(PagedBatch):
    """The same over pages of 4-bit values (include/llm.h): k_pages, v_pages uint8
    [n_pages, bytes of a page], as q4_pages() makes them."""

    def __init__(self, k_pages, v_pages, page_table, lens, page_size: int, n_kv_heads: int, head_dim: int, n_new: int = 1,
                 prefix_len: int = 0, err=None):
        _int32(n_new=n_new, prefix_len=prefix_len)
        _tensor("k_pages", k_pages, (torch.uint8,), (None, _q4_page_bytes(page_size, n_kv_heads, head_dim)), None)
        self._set(k_pages, v_pages, page_table, lens, page_size, n_kv_heads, head_dim, n_new, prefix_len, err)


def _q4_page_bytes(page_size: int, n_kv_heads: int, head_dim: int) -> int:
    _int32(page_size=page_size, n_kv_heads=n_kv_heads, head_dim=head_dim)
    n = _b._lib.llm_q4_page_bytes(page_size, n_kv_heads, head_dim)
    if n < 0:
        _run(int(n))
    return int(n)


def q4_pages(n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, n_layers: int | None = None, device="cuda") -> torch.Tensor:
    """Pages of 4-bit values, all zero: uint8 [n_pages, bytes of a page], with n_layers
    [n_layers, n_pages, bytes of a page]."""
    shape = (n_pages, _q4_page_bytes(page_size, n_kv_heads, head_dim))
    return torch.zeros(shape if n_layers is None else (n_layers, *shape), dtype=torch.uint8, device=device)


class _Op(_Owner):
    """One operator with its arguments; calling it enqueues one run.  The operator must
    live as long as a graph that captured its runs.  A stream given by number must live
    as long as the operator."""

    def _made(self, fn, pages, kept, structs, own, device) -> None:
        self._owns(own, device)
        if pages is not None:
            pages._use_on(_current_stream(device.index))
        self._fn, self._pages, self._kept = fn, pages, (kept, structs)
        self._args = tuple(ctypes.addressof(x) for x in structs)

    def __call__(self, stream=None) -> None:
        index = self._index
        if _current_device() != index:
            raise ValueError(f"the operator's tensors are on cuda:{index}, the current device is another")
        if stream is None:
            stream = _current_stream(index)
        if stream not in self._streams:
            if self._pages is not None:
                self._pages._use_on(stream)
            self._use_on(stream)
        rc = self._fn(*self._args, stream)
        if rc:
            _run(rc)


class KvAppend(_Op):
    """llm_kv_append: rotates q [rows, n_heads, head_dim] into q_out and k
    [rows, n_kv_heads, head_dim] on its way into the pages, which take v too.
    q, k, v: float32 or float16, free in the row stride (parts of one fused
    projection); q None: no queries.  q_out: float32 or float16, q itself for a
    rotation in place.  cos_sin: float32 [positions, rope_dims / 2, 2] from
    rope_table() or the caller's own."""

    def __init__(self, pages: PagedBatch, q, k, v, cos_sin, q_out=None, rope_neox: bool = False):
        p, dev = pages.struct, pages.device
        kv = (pages.rows, p.n_kv_heads, p.head_dim)
        _tensor("k", k, _DTYPES, kv, dev, strided=True)
        _tensor("v", v, (k.dtype,), kv, dev, strided=True)
        _tensor("cos_sin", cos_sin, (torch.float32,), (None, None, 2), dev)
        _int32(positions=cos_sin.shape[0], rope_dims=2 * cos_sin.shape[1])
        a = _b.llm_append(n_heads=0, rope_dims=2 * cos_sin.shape[1], rope_neox=int(rope_neox),
                          table_rows=cos_sin.shape[0], dtype=_DTYPES[k.dtype], q_out_dtype=_b.LLM_F32,
                          k=k.data_ptr(), v=v.data_ptr(), k_stride=k.stride(0), v_stride=v.stride(0),
                          cos_sin=cos_sin.data_ptr())
        if q is not None:
            _tensor("q", q, (k.dtype,), (pages.rows, None, p.head_dim), dev, strided=True)
            _tensor("q_out", q_out, _DTYPES, tuple(q.shape), dev, strided=True)
            a.n_heads, a.q, a.q_stride = q.shape[1], q.data_ptr(), q.stride(0)
            a.q_out, a.q_out_stride, a.q_out_dtype = q_out.data_ptr(), q_out.stride(0), _DTYPES[q_out.dtype]
        fn = _b._lib.llm_kv_append_q4 if isinstance(pages, PagedBatchQ4) else _b._lib.llm_kv_append
        self._made(fn, pages, (q, k, v, cos_sin, q_out), (p, a), (), dev)


class KvRead(_Op):
    """llm_kv_read: the new rows' k and v into k_out, v_out [rows, n_kv_heads,
    head_dim] (float32 or float16, free in the row stride)."""

    def __init__(self, pages: PagedBatch, k_out, v_out):
        p, dev = pages.struct, pages.device
        kv = (pages.rows, p.n_kv_heads, p.head_dim)
        _tensor("k_out", k_out, _DTYPES, kv, dev, strided=True)
        _tensor("v_out", v_out, (k_out.dtype,), kv, dev, strided=True)
        a = _b.llm_read(dtype=_DTYPES[k_out.dtype], k_out=k_out.data_ptr(), v_out=v_out.data_ptr(), k_stride=k_out.stride(0),
                        v_stride=v_out.stride(0))
        fn = _b._lib.llm_kv_read_q4 if isinstance(pages, PagedBatchQ4) else _b._lib.llm_kv_read
        self._made(fn, pages, (k_out, v_out), (p, a), (), dev)


class AttendBatch(_Op):
    """llm_attend_batch: out = attention of q [rows, n_heads, head_dim] over
    the shared prefix_k, prefix_v (float16 [at least prefix_len, n_kv_heads,
    head_dim], free in the row stride) and the sequences' pages.  q, out:
    float32 or float16, free in the row stride.  The operator owns its
    workspace, so runs of one object must not overlap in time: give each stream
    (and each captured graph that may run beside another) its own."""

    def __init__(self, pages: PagedBatch, q, out, prefix_k=None, prefix_v=None, scale: float = 0.0):
        p, dev = pages.struct, pages.device
        _tensor("q", q, _DTYPES, (pages.rows, None, p.head_dim), dev, strided=True)
        _tensor("out", out, _DTYPES, tuple(q.shape), dev, strided=True)
        a = _b.llm_attend(n_heads=q.shape[1], q_dtype=_DTYPES[q.dtype], out_dtype=_DTYPES[out.dtype], scale=scale,
                          q=q.data_ptr(), q_stride=q.stride(0), out=out.data_ptr(), out_stride=out.stride(0))
        if p.prefix_len > 0:
            for name, t in (("prefix_k", prefix_k), ("prefix_v", prefix_v)):
                _tensor(name, t, (torch.float16,), (None, p.n_kv_heads, p.head_dim), dev, strided=True)
                if t.shape[0] < p.prefix_len:
                    raise ValueError(f"{name} holds {t.shape[0]} rows, the prefix has {p.prefix_len}")
            if prefix_k.stride(0) != prefix_v.stride(0):
                raise ValueError("prefix_k and prefix_v have different row strides")
            a.prefix_k, a.prefix_v, a.prefix_stride = prefix_k.data_ptr(), prefix_v.data_ptr(), prefix_k.stride(0)
        q4 = isinstance(pages, PagedBatchQ4)
        n = (_b._lib.llm_attend_batch_q4_workspace if q4 else _b._lib.llm_attend_batch_workspace)(ctypes.byref(p), ctypes.byref(a))
        if n < 0:
            _run(int(n))
        self.workspace = torch.empty(max(int(n), 1), dtype=torch.uint8, device=dev)
        a.workspace, a.workspace_bytes = self.workspace.data_ptr(), int(n)
        self._made(_b._lib.llm_attend_batch_q4 if q4 else _b._lib.llm_attend_batch, pages, (q, out, prefix_k, prefix_v), (p, a), (self.workspace,), dev)


class PagePool(_Owner):
    """Sequences and the pages that they hold (llm_pool), for PagesUpdate and
    PagesCompact.  k_pages, v_pages: float16 [n_pages, page_size, n_kv_heads, head_dim],
    or uint8 [n_pages, bytes of a page] (then page_size is wanted), each also with the
    layers before that, free in the layers' stride; None: tables only.  page_table
    int32 [n_seqs, max_pages], lens int32 [n_seqs], refs int32 [n_pages]; ``err``
    collects errors as in PagedBatch, whose page_table, lens and err these may be."""

    def __init__(self, k_pages, v_pages, page_table, lens, refs, page_size: int | None = None, err=None):
        _tensor("refs", refs, (torch.int32,), (None,), None)
        dev, n_pages = refs.device, refs.shape[0]
        _tensor("lens", lens, (torch.int32,), (None,), dev)
        _tensor("page_table", page_table, (torch.int32,), (lens.shape[0], None), dev)
        made = err is None
        if made:
            err = torch.zeros(1, dtype=torch.int32, device=dev)
        _tensor("err", err, (torch.int32,), (1,), dev)
        s = _b.llm_pool(n_seqs=lens.shape[0], n_pages=n_pages, max_pages=page_table.shape[1], page_table=page_table.data_ptr(),
                        lens=lens.data_ptr(), refs=refs.data_ptr(), err=err.data_ptr())
        if k_pages is not None:
            page = 3 if isinstance(k_pages, torch.Tensor) and k_pages.dtype == torch.float16 else 1
            layers = isinstance(k_pages, torch.Tensor) and k_pages.dim() == page + 2
            shape = ((None,) if layers else ()) + (n_pages,) + (None,) * page
            _tensor("k_pages", k_pages, (torch.float16, torch.uint8), shape, dev, strided=layers)
            _tensor("v_pages", v_pages, (k_pages.dtype,), tuple(k_pages.shape), dev, strided=layers)
            if layers and k_pages.stride(0) != v_pages.stride(0):
                raise ValueError("k_pages and v_pages have different layer strides")
            size = k_pages.element_size()
            one = k_pages.shape[1 + layers:].numel() * size
            if page == 3:
                if page_size not in (None, k_pages.shape[1 + layers]):
                    raise ValueError(f"page_size {page_size}: the pages have {k_pages.shape[1 + layers]} rows")
                page_size = k_pages.shape[1 + layers]
                s.row_bytes = one // max(page_size, 1)
            s.n_layers = k_pages.shape[0] if layers else 1
            s.k_pages, s.v_pages, s.page_bytes = k_pages.data_ptr(), v_pages.data_ptr(), one
            s.layer_stride = k_pages.stride(0) * size if layers else n_pages * one
        if page_size is None:
            raise ValueError("page_size is wanted for pages of bytes, and without pages")
        _int32(n_seqs=s.n_seqs, page_size=page_size, pages=n_pages, max_pages=page_table.shape[1], layers=s.n_layers)
        s.page_size = page_size
        self._owns((err,) if made else (), dev)
        self.k_pages, self.v_pages, self.page_table, self.lens, self.refs, self.err = k_pages, v_pages, page_table, lens, refs, err
        self.device, self.struct = dev, s

    def errors(self) -> int:
        """The LLM_PAGES_* bits seen so far (waits for the device)."""
        torch.cuda.synchronize(self.device)
        return int(self.err.item())


class PagesUpdate(_Op):
    """llm_pages_update: sequence s goes on from parents[s] (int32 [n_seqs]; None: itself)
    and has rows[s] rows then (int32 [n_seqs]; None: as many as its parent).  The
    operator owns its workspace, as AttendBatch does."""

    def __init__(self, pool: PagePool, parents=None, rows=None):
        p, dev = pool.struct, pool.device
        for name, t in (("parents", parents), ("rows", rows)):
            if t is not None:
                _tensor(name, t, (torch.int32,), (p.n_seqs,), dev)
        n = _b._lib.llm_pages_update_workspace(ctypes.byref(p))
        if n < 0:
            _run(int(n))
        self.workspace = torch.empty(max(int(n), 1), dtype=torch.uint8, device=dev)
        self._made(_b._lib.llm_pages_update, pool, (parents, rows), (p,), (self.workspace,), dev)
        self._args += tuple(t.data_ptr() if t is not None else None for t in (parents, rows)) + (self.workspace.data_ptr(), int(n))


class PagesCompact(_Op):
    """llm_pages_compact: the pages in use to the front of the pool.  table_out and
    refs_out (None: the pool's own tensors, in place) receive the new tables; moved int32
    [n_pages] and n_live int32 [1] (None: made here) each page's new number and how
    many are in use."""

    def __init__(self, pool: PagePool, table_out=None, refs_out=None, moved=None, n_live=None):
        p, dev = pool.struct, pool.device
        own = []
        table_out = pool.page_table if table_out is None else table_out
        refs_out = pool.refs if refs_out is None else refs_out
        if moved is None:
            moved = torch.empty_like(pool.refs)
            own.append(moved)
        if n_live is None:
            n_live = torch.empty(1, dtype=torch.int32, device=dev)
            own.append(n_live)
        for name, t, shape in (("table_out", table_out, tuple(pool.page_table.shape)), ("refs_out", refs_out, (p.n_pages,)),
                               ("moved", moved, (p.n_pages,)), ("n_live", n_live, (1,))):
            _tensor(name, t, (torch.int32,), shape, dev)
        n = _b._lib.llm_pages_compact_workspace(ctypes.byref(p))
        if n < 0:
            _run(int(n))
        self.workspace = torch.empty(max(int(n), 1), dtype=torch.uint8, device=dev)
        self.table_out, self.refs_out, self.moved, self.n_live = table_out, refs_out, moved, n_live
        self._made(_b._lib.llm_pages_compact, pool, (table_out, refs_out, moved, n_live), (p,), (self.workspace, *own), dev)
        self._args += tuple(t.data_ptr() for t in (table_out, refs_out, moved, n_live, self.workspace)) + (int(n),)


class AdjustLogits(_Op):
    """llm_logits_adjust: penalties for repeated tokens, biases and masks on logits
    [rows, vocab] (float32 or float16, free in the row stride) into out (likewise; None:
    logits itself).  history int32 [rows, max_history] with history_lens int32 [rows]
    and, float32 [rows] or None each, repetition, frequency and presence; window: how many
    of the last tokens count (0: all).  bias_ids int32 and bias float32 [rows, n_bias].
    masks int32 [n_masks, at least vocab / 32] (bit 0: banned), mask_of int32 [rows] the
    mask of each row (None: its own)."""

    def __init__(self, logits, out=None, history=None, history_lens=None, window: int = 0, repetition=None, frequency=None,
                 presence=None, bias_ids=None, bias=None, masks=None, mask_of=None):
        _int32(window=window)
        _tensor("logits", logits, _DTYPES, (None, None), None, strided=True)
        dev, (n, vocab) = logits.device, logits.shape
        out = logits if out is None else out
        _tensor("out", out, _DTYPES, (n, vocab), dev, strided=True)
        _int32(rows=n, vocab=vocab)
        a = _b.llm_adjust(n_rows=n, vocab=vocab, dtype=_DTYPES[logits.dtype], out_dtype=_DTYPES[out.dtype], logits=logits.data_ptr(),
                          stride=logits.stride(0), out=out.data_ptr(), out_stride=out.stride(0), window=window)
        if history is None and any(t is not None for t in (history_lens, repetition, frequency, presence)):
            raise ValueError("penalties without a history")
        if history is not None:
            _tensor("history", history, (torch.int32,), (n, None), dev, strided=True)
            _tensor("history_lens", history_lens, (torch.int32,), (n,), dev)
            _int32(max_history=history.shape[1])
            a.history, a.history_stride, a.max_history = history.data_ptr(), history.stride(0), history.shape[1]
            a.history_lens = history_lens.data_ptr()
            for name, t in (("repetition", repetition), ("frequency", frequency), ("presence", presence)):
                if t is not None:
                    _tensor(name, t, (torch.float32,), (n,), dev)
                    setattr(a, name, t.data_ptr())
        if (bias_ids is None) != (bias is None):
            raise ValueError("bias_ids and bias belong together")
        if bias_ids is not None:
            _tensor("bias_ids", bias_ids, (torch.int32,), (n, None), dev)
            _tensor("bias", bias, (torch.float32,), tuple(bias_ids.shape), dev)
            _int32(n_bias=bias_ids.shape[1])
            a.bias_ids, a.bias, a.n_bias = bias_ids.data_ptr(), bias.data_ptr(), bias_ids.shape[1]
        if masks is None and mask_of is not None:
            raise ValueError("mask_of without masks")
        if masks is not None:
            _tensor("masks", masks, (torch.int32,), (None, None), dev, strided=True)
            if masks.shape[1] < -(-vocab // 32):
                raise ValueError(f"masks of {masks.shape[1]} words, {-(-vocab // 32)} are wanted")
            if mask_of is None and masks.shape[0] < n:
                raise ValueError(f"{masks.shape[0]} masks for {n} rows")
            _int32(n_masks=masks.shape[0])
            a.masks, a.n_masks, a.mask_stride = masks.data_ptr(), masks.shape[0], masks.stride(0)
            if mask_of is not None:
                _tensor("mask_of", mask_of, (torch.int32,), (n,), dev)
                a.mask_of = mask_of.data_ptr()
        self.out = out
        self._made(_b._lib.llm_logits_adjust, None,
                   (logits, out, history, history_lens, repetition, frequency, presence, bias_ids, bias, masks, mask_of), (a,), (), dev)


class LogProbs(_Op):
    """llm_logprobs of logits [rows, vocab] (float32 or float16, free in the
    row stride): the log probability of each token of targets (int32 [rows,
    n_targets], -1: none; None: no targets), the entropy and the ``top`` most
    likely tokens of each row, in the tensors logprob, entropy, top_id and
    top_logprob."""

    def __init__(self, logits, targets=None, top: int = 0):
        _int32(top=top)
        _tensor("logits", logits, _DTYPES, (None, None), None, strided=True)
        n, dev = logits.shape[0], logits.device
        if targets is not None:
            _tensor("targets", targets, (torch.int32,), (n, None), dev)
        n_targets = 0 if targets is None else targets.shape[1]
        _int32(rows=n, vocab=logits.shape[1], n_targets=n_targets)
        self.logprob = torch.empty(n, n_targets, dtype=torch.float32, device=dev)
        self.entropy = torch.empty(n, dtype=torch.float32, device=dev)
        self.top_id = torch.empty(n, max(top, 0), dtype=torch.int32, device=dev)
        self.top_logprob = torch.empty(n, max(top, 0), dtype=torch.float32, device=dev)
        a = _b.llm_logprobs_args(n_rows=n, vocab=logits.shape[1], dtype=_DTYPES[logits.dtype], n_targets=n_targets,
                                 top=top, logits=logits.data_ptr(), stride=logits.stride(0),
                                 targets=targets.data_ptr() if n_targets else None, logprob=self.logprob.data_ptr(),
                                 entropy=self.entropy.data_ptr(), top_id=self.top_id.data_ptr(),
                                 top_logprob=self.top_logprob.data_ptr())
        self._made(_b._lib.llm_logprobs, None, (logits, targets), (a,),
                   (self.logprob, self.entropy, self.top_id, self.top_logprob), dev)


class BatchDecoder:
    """Steps of n_seqs continuations of the prompt in rows 0 .. prefix_len - 1 of a
    decoder's cache (llm_decode_batch).  tokens int32 [n_seqs, n_new], lens int32
    [n_seqs] (the rows behind the prompt, this step's among them) and page_table
    int32 [n_seqs, max_pages] are this object's tensors, to be written before each
    step; logits float32 [n_seqs, n_new, vocab] is the step's result.  ``pages``
    holds every layer's K and V pages; page_table starts with each sequence's own
    pages in a row.  q4: pages of 4-bit values (llm_decode_batch_q4).  step() enqueues on the decoder's stream; where that is not the
    current one, it runs behind what the current stream has been given (the tensors'
    new values) and before what it is given next."""

    def __init__(self, decoder, n_seqs: int, max_len: int, prefix_len: int, n_new: int = 1, page_size: int = 16, q4: bool = False):
        _int32(n_seqs=n_seqs, max_len=max_len, prefix_len=prefix_len, n_new=n_new, page_size=page_size)
        if page_size < 1:
            raise ValueError(f"page_size {page_size} is not positive")
        c = _b.llm_get_config(decoder.h)
        dev = torch.device("cuda", torch.cuda.current_device())
        max_pages = -(-max_len // page_size)
        n_pages = n_seqs * max_pages
        _int32(n_pages=n_pages)
        self.decoder, self.q4 = decoder, bool(q4)
        self._device, self._stream = dev, _torch_stream(decoder.stream, dev)
        # the tensors are the decoder's stream's: filled there, and their memory, when it is
        # given back, goes to later work of that stream only
        with torch.cuda.stream(self._stream):
            n_bytes = max(1, _b.llm_batch_pages_bytes(decoder.h, n_pages, page_size, q4))
            self.pages = torch.zeros(n_bytes if q4 else n_bytes // 2, dtype=torch.uint8 if q4 else torch.float16, device=dev)
            self.page_table = torch.arange(n_pages, dtype=torch.int32, device=dev).view(n_seqs, max_pages)
            self.lens = torch.zeros(n_seqs, dtype=torch.int32, device=dev)
            self.tokens = torch.zeros(n_seqs, n_new, dtype=torch.int32, device=dev)
            self.logits = torch.empty(n_seqs, n_new, c.vocab, dtype=torch.float32, device=dev)
            self.err = torch.zeros(1, dtype=torch.int32, device=dev)
        self._users = {self._stream.cuda_stream}           # the streams that the tensors' memory waits for
        self._use_on(torch.cuda.current_stream(dev))
        self.struct = _b.llm_batch(n_seqs=n_seqs, n_new=n_new, prefix_len=prefix_len, page_size=page_size,
                                   n_pages=n_pages, max_pages=max_pages, pages=self.pages.data_ptr(),
                                   page_table=self.page_table.data_ptr(), lens=self.lens.data_ptr(),
                                   tokens=self.tokens.data_ptr(), logits=self.logits.data_ptr(), err=self.err.data_ptr())

    def pool(self, refs, err=None) -> "PagePool":
        """The decoder's pages as a pool, with refs int32 [n_pages] the pages' holders: what the
        sequences hold is then up to PagesUpdate, which page_table and lens are written by."""
        if refs.shape[0] != self.struct.n_pages:
            raise ValueError(f"{refs.shape[0]} counts of holders for {self.struct.n_pages} pages")
        c, p = _b.llm_get_config(self.decoder.h), self.struct
        page = (_q4_page_bytes(p.page_size, c.n_kv_heads, c.head_dim),) if self.q4 else (p.page_size, c.n_kv_heads, c.head_dim)
        shape = torch.Size((c.n_layers, 2, p.n_pages, *page))
        kv = self.pages[:shape.numel()].view(shape)
        return PagePool(kv[:, 0], kv[:, 1], self.page_table, self.lens, refs, page_size=p.page_size, err=err)

    def _use_on(self, stream) -> None:
        """What `stream` is given from now on may use the tensors."""
        stream.wait_stream(self._stream)
        if stream.cuda_stream not in self._users:
            self._users.add(stream.cuda_stream)
            for t in (self.pages, self.page_table, self.lens, self.tokens, self.logits, self.err):
                t.record_stream(stream)

    def step(self) -> None:
        if _current_stream(self._device.index) == self._stream.cuda_stream:
            _b.llm_decode_batch(self.decoder.h, self.struct, self.q4)
            return
        current = torch.cuda.current_stream(self._device)
        self._stream.wait_stream(current)
        try:
            _b.llm_decode_batch(self.decoder.h, self.struct, self.q4)
        finally:
            self._use_on(current)

    def errors(self) -> int:
        """The LLM_PAGES_* bits seen so far (waits for the device)."""
        torch.cuda.synchronize(self._device)
        return int(self.err.item())


def rope_table(n_pos: int, rope_dims: int, rope_base: float, rope_freqs=None, pos0: int = 0, device="cuda",
               stream=None) -> torch.Tensor:
    """llm_rope_table: float32 [n_pos, rope_dims / 2, 2] of the decode step's
    angles at positions pos0 .. pos0 + n_pos - 1."""
    _int32(n_pos=n_pos, rope_dims=rope_dims, pos0=pos0)
    out = torch.empty(n_pos, rope_dims // 2, 2, dtype=torch.float32, device=device)
    if out.device.index != _current_device():
        raise ValueError(f"the table is on {out.device}, the current device is another")
    if rope_freqs is not None:
        _tensor("rope_freqs", rope_freqs, (torch.float32,), (rope_dims // 2,), out.device)
    if stream is not None and stream != _current_stream(out.device.index):
        other = _torch_stream(stream, out.device)
        other.wait_stream(torch.cuda.current_stream(out.device))
        out.record_stream(other)
    _run(_b._lib.llm_rope_table(out.data_ptr(), pos0, n_pos, rope_dims, rope_base,
                                rope_freqs.data_ptr() if rope_freqs is not None else None, _stream(stream)))
    return out
