"""The stand-alone operators around the decode: attention of one new token over a
cache, the pages of a paged cache, and log probabilities of given tokens.

Argument marshalling only, as in engine.py: every step runs in libxlpk.so's
kernels (include/xlpk.h has the definitions).  Calls are asynchronous on the
device's current stream, or on `stream`; tensors are used on the device they are
on, whichever is current.  What a call allocates (results, workspaces) comes from
torch's allocator on that stream, one for each call, so calls on several streams
and captured CUDA graphs do not share any.  Wrong dtypes, shapes and devices
raise ValueError, refused calls XlpkError; what only the device can see goes to
a status word.  No gradients are recorded.

The smallest calls take a few microseconds on the GPU, so the host side is kept
short: messages are only put together for a call that fails, arguments are
packed in one go, and nothing is asked of the library twice.
"""
from __future__ import annotations

import ctypes as C
import struct
from operator import index
from typing import NamedTuple, Optional

import torch

from . import _abi
from .engine import XlpkError, _check, get_lib

_IO = {torch.float32: _abi.XLPK_DTYPE_FP32, torch.bfloat16: _abi.XLPK_DTYPE_BF16}
_KV = {torch.bfloat16: _abi.XLPK_DTYPE_BF16, torch.uint8: _abi.XLPK_DTYPE_FP8_E4M3,
       torch.float8_e4m3fn: _abi.XLPK_DTYPE_FP8_E4M3}
_I32 = (torch.int32,)
_ATTENTION = struct.Struct("10P15q11i3f")    # xlpk_attention_args
_POOL = struct.Struct("6P7i4x")              # xlpk_page_pool
_F = {}                                      # the library's functions


def _fn(name: str):
    f = _F.get(name)
    if f is None:
        f = _F[name] = getattr(get_lib(), name)
    return f


def _refuse(what: str):
    raise ValueError(what)


def _tensor(t, name: str, dim: int, dtypes, device: int) -> None:
    """`t` is a `dim`-d CUDA tensor of one of `dtypes`, on GPU `device` (< 0: any)."""
    if isinstance(t, torch.Tensor) and t.dtype in dtypes and t.dim() == dim:
        at = t.get_device()
        if at >= 0 and (at == device or device < 0):
            return
    have = f"{t.dim()}-d {t.dtype} on {t.device}" if isinstance(t, torch.Tensor) else type(t).__name__
    where = "a GPU" if device < 0 else f"cuda:{device}"
    _refuse(f"{name} is {have}, want {dim}-d {' or '.join(str(d) for d in dtypes)} on {where}")


def _int32(v, name: str) -> int:
    try:
        n = index(v)
    except TypeError:
        _refuse(f"{name} = {v!r} is not an integer")
    if not -(1 << 31) <= n < 1 << 31:
        _refuse(f"{name} = {n} does not fit an int32")
    return n


def _distinct(t) -> bool:
    """No two elements share memory (sufficient: every stride steps over all inner ones)."""
    reach = 0
    for s, n in sorted((s, n) for s, n in zip(t.stride(), t.shape) if n > 1):
        if s <= reach:
            return False
        reach += s * (n - 1)
    return True


# empty_strided(size, stride, dtype) on the current device, where torch has it without the
# parsing of keyword arguments (0.7 us against 1.9 for new_empty; a call makes two to five)
_guards = getattr(getattr(torch._C, "_dynamo", None), "guards", None)
_strided = getattr(_guards, "_empty_strided_cuda", None) or (
    lambda size, stride, dtype: torch.empty_strided(size, stride, dtype=dtype, device="cuda"))


def _contiguous(size):
    """Strides of a contiguous tensor of a tuple's size."""
    stride, n = [1] * len(size), 1
    for i in range(len(size) - 1, -1, -1):
        stride[i] = n
        n *= size[i] or 1
    return tuple(stride)


def _on(device: int, stream, tensors, launch):
    """launch(handle) on the stream: its allocations belong to that stream, and so, for
    an explicit one, do the tensors it uses, until that use is over."""
    if stream is None:
        if torch._C._cuda_getDevice() == device:
            return launch(torch._C._cuda_getCurrentRawStream(device))
        with torch.cuda.device(device):
            return launch(torch._C._cuda_getCurrentRawStream(device))
    if stream.device.index != device:
        _refuse(f"stream is on {stream.device}, the tensors on cuda:{device}")
    with torch.cuda.stream(stream):
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
        return launch(stream.cuda_stream)


# ---- attention

_WORKSPACE = {}    # (wide group, head_dim) -> bytes


def decode_attention(q, k_cache, v_cache, seq_lens, page_table=None, *, k_new=None, v_new=None,
                     scale: Optional[float] = None, window: int = 0, sinks: int = 0, k_scale: float = 1.0,
                     v_scale: float = 1.0, out=None, return_lse: bool = False, status=None, stream=None):
    """xlpk_decode_attention: softmax(scale * q . K^T) V of one new token per sequence.

    `q` [B][n_q][d], bf16 or fp32 (d 64 or 128); `k_cache`, `v_cache` one layer of
    the decode's cache, bf16 or e4m3 codes (uint8 or float8_e4m3fn; value = code *
    k_scale, v_scale): paged [n_pages][n_kv][page_size][d] with `page_table` int32
    [B][pages per sequence], or contiguous [B][n_kv][capacity][d].  `seq_lens`
    int32 [B]: positions in the cache, the new one included.  `k_new`, `v_new`
    [B][n_kv][d] (q's dtype) are stored first as the row of position seq_lens - 1.
    `window` > 0 hides positions before seq_lens - window except the first `sinks`.
    `scale` defaults to 1/sqrt(d).  Returns out [B][n_q][d] of q's dtype, with
    `return_lse` also the fp32 [B][n_q] log of the softmax's denominator.  Any
    order of the tensors is taken whose rows of d are contiguous and whose strides
    are multiples of 16 bytes.  `status`, one int32 on the device, is set where a
    visible position names a page outside the pool or a length does not fit
    (that sequence's output is NaN).
    """
    _tensor(q, "q", 3, _IO, -1)
    dev = q.get_device()
    _tensor(k_cache, "k_cache", 4, _KV, dev)
    _tensor(v_cache, "v_cache", 4, (k_cache.dtype,), dev)
    _tensor(seq_lens, "seq_lens", 1, _I32, dev)
    B, H, D = q.shape
    n_pages, KH, P, d = k_cache.shape
    if v_cache.shape != k_cache.shape or d != D or D == 0:
        _refuse(f"caches of {tuple(k_cache.shape)} and {tuple(v_cache.shape)} for head_dim {D}")
    if seq_lens.shape[0] != B or (B > 1 and seq_lens.stride(0) != 1):
        _refuse("seq_lens must be a contiguous [B]")
    qs, ks, vs = q.stride(), k_cache.stride(), v_cache.stride()
    if qs[2] != 1 or ks[3] != 1 or vs[3] != 1:
        _refuse("rows of head_dim must be contiguous")
    # nothing steps along a dimension of one element: its stride is not looked at
    one_b, one_h, one_kh, one_p, one_pos = B < 2, H < 2, KH < 2, n_pages < 2, P < 2
    if page_table is None:
        if n_pages != B:
            _refuse(f"a contiguous cache of {n_pages} sequences for {B} queries")
        table_at, cols, table_step = 0, 1, 0
    else:
        _tensor(page_table, "page_table", 2, _I32, dev)
        rows, cols = page_table.shape
        if rows != B or (cols > 1 and page_table.stride(1) != 1):
            _refuse("page_table must be [B][pages] with contiguous rows")
        table_at, table_step = page_table.data_ptr(), 0 if one_b else page_table.stride(0)
    kn = vn = nk0 = nk1 = nv0 = nv1 = 0
    if k_new is not None or v_new is not None:
        for t, name in ((k_new, "k_new"), (v_new, "v_new")):
            _tensor(t, name, 3, (q.dtype,), dev)
            if t.shape != (B, KH, D) or t.stride(2) != 1:
                _refuse(f"{name} must be [B][n_kv][d] with contiguous rows")
        if not (k_cache.is_contiguous() or _distinct(k_cache)) or not (v_cache.is_contiguous() or _distinct(v_cache)):
            _refuse("a cache that is written must not overlap itself")
        kn, vn = k_new.data_ptr(), v_new.data_ptr()
        (nk0, nk1, _), (nv0, nv1, _) = k_new.stride(), v_new.stride()
    if out is not None:
        _tensor(out, "out", 3, (q.dtype,), dev)
        if out.shape != q.shape or out.stride(2) != 1 or not _distinct(out):
            _refuse("out must be [B][n_q][d] with rows of its own")
    if status is not None:
        _tensor(status, "status", 1, _I32, dev)
        if status.shape[0] < 1:
            _refuse("status must hold one int32")
    key = (KH > 0 and H > 8 * KH, D)

    def launch(handle):
        o = _strided((B, H, D), (H * D, D, 1), q.dtype) if out is None else out
        os = o.stride()
        lse = _strided((B, H), (H, 1), torch.float32) if return_lse else None
        try:
            args = _ATTENTION.pack(
                q.data_ptr(), kn, vn, k_cache.data_ptr(), v_cache.data_ptr(), table_at, seq_lens.data_ptr(), o.data_ptr(),
                0 if lse is None else lse.data_ptr(), 0 if status is None else status.data_ptr(),
                0 if one_b else qs[0], 0 if one_h else qs[1],
                0 if one_b else nk0, 0 if one_kh else nk1, 0 if one_b else nv0, 0 if one_kh else nv1,
                0 if one_b else os[0], 0 if one_h else os[1],
                0 if one_p else ks[0], 0 if one_kh else ks[1], 0 if one_pos else ks[2],
                0 if one_p else vs[0], 0 if one_kh else vs[1], 0 if one_pos else vs[2], table_step,
                B, H, KH, D, n_pages, P, cols, _IO[q.dtype], _KV[k_cache.dtype], window, sinks,
                D ** -0.5 if scale is None else scale, k_scale, v_scale)
        except (struct.error, OverflowError, TypeError) as e:
            raise ValueError(f"window, sinks, scale, k_scale or v_scale: {e}") from None
        need = _WORKSPACE.get(key)
        if need is None:
            need = _fn("xlpk_decode_attention_workspace")(args)
            if need:
                _WORKSPACE[key] = need
        ws = _strided((need or 16,), (1,), torch.uint8)
        st = _fn("xlpk_decode_attention")(args, ws.data_ptr(), need, handle)
        if st:
            _check(st, "xlpk_decode_attention")
        return (o, lse) if return_lse else o

    return _on(dev, stream, (q, k_cache, v_cache, seq_lens, page_table, k_new, v_new, out, status), launch)


# ---- pages

class PagePool:
    """The pages of a paged cache and who holds them (xlpk_page_pool).

    `k`, `v` [L][n_pages][n_kv][page_size][d] as the engine's pools; `page_table`
    int32 [rows][cols] (-1: no page), `seq_lens` int32 [rows], `refs` int32
    [n_pages] (None: counted from the table; the caller may add references of its
    own).  All stay the caller's and are updated in place; the attributes of these
    names may be assigned other tensors, which later calls then use.  Calls are
    asynchronous; one that cannot be done changes nothing and sets `status`
    (int32 [1]), which stops later calls until `check()` has reported it.  Calls on
    several streams are the caller's to put in order, as with any tensor.
    """

    def __init__(self, k, v, page_table, seq_lens, refs=None, status=None):
        if refs is None:
            _tensor(k, "k", 5, _KV, -1)
            _tensor(page_table, "page_table", 2, _I32, k.get_device())
            held, n_pages = page_table.reshape(-1), k.shape[1]
            held = held[(held >= 0) & (held < n_pages)]
            refs = torch.bincount(held, minlength=n_pages).to(torch.int32)
        if status is None:
            _tensor(k, "k", 5, _KV, -1)
            status = torch.zeros(1, dtype=torch.int32, device=k.device)
        self._streams = set()     # handles of the streams of the calls so far, for check()
        self._bind(k, v, page_table, seq_lens, refs, status)

    def _bind(self, k, v, page_table, seq_lens, refs, status) -> None:
        """Takes the six tensors, all of them or (ValueError) none."""
        _tensor(k, "k", 5, _KV, -1)
        dev = k.get_device()
        _tensor(v, "v", 5, (k.dtype,), dev)
        _tensor(page_table, "page_table", 2, _I32, dev)
        _tensor(seq_lens, "seq_lens", 1, _I32, dev)
        _tensor(refs, "refs", 1, _I32, dev)
        _tensor(status, "status", 1, _I32, dev)
        L, n_pages, KH, P, D = k.shape
        rows, cols = page_table.shape
        if v.shape != k.shape:
            _refuse(f"pools of {tuple(k.shape)} and {tuple(v.shape)}")
        if seq_lens.shape[0] != rows or refs.shape[0] != n_pages or status.shape[0] < 1:
            _refuse("seq_lens must have the table's rows, refs the pool's pages")
        if not (k.is_contiguous() and v.is_contiguous() and page_table.is_contiguous() and seq_lens.is_contiguous()
                and refs.is_contiguous()):
            _refuse("pool tensors must be contiguous")
        held = (k, v, page_table, seq_lens, refs, status)
        at = [t.data_ptr() for t in held]
        try:
            c = _POOL.pack(*at, L, n_pages, KH, P, D * k.element_size(), rows, cols)
        except struct.error as e:
            raise ValueError(f"a size does not fit an int32: {e}") from None
        self._held, self._at, self._c, self._device, self._rows_n, self._pages_n = held, at, c, dev, rows, n_pages

    # The tensors may be assigned, and are checked again then (`pool.seq_lens += 1` assigns too).
    k, v, page_table, seq_lens, refs, status = (
        property(lambda self, i=i: self._held[i],
                 lambda self, t, i=i: self._bind(*self._held[:i], t, *self._held[i + 1:])) for i in range(6))

    @property
    def device(self):
        return self.k.device

    def _call(self, name: str, stream, *args, row=None, row_name: str = "", workspace: bool = False) -> None:
        """`row`: the call's first argument, an int32 tensor of one entry a row."""
        if [t.data_ptr() for t in self._held] != self._at:   # one was given other memory (t.data = ..., resize_)
            self._bind(*self._held)
        if row_name:
            _tensor(row, row_name, 1, _I32, self._device)
            if row.shape[0] != self._rows_n or not row.is_contiguous():
                _refuse(f"{row_name} must be a contiguous [rows]")
            args = (row.data_ptr(), *args)

        def launch(handle):
            self._streams.add(handle)
            if workspace:
                n = _fn("xlpk_pages_workspace")(self._c)
                ws = _strided((n or 16,), (1,), torch.uint8)
                st = _fn(name)(self._c, *args, ws.data_ptr(), n, handle)
            else:
                st = _fn(name)(self._c, *args, handle)
            if st:
                _check(st, name)
        _on(self._device, stream, () if stream is None else (*self._held, row), launch)

    def fork(self, parents, stream=None) -> None:
        """xlpk_pages_fork: row r becomes what row parents[r] was (-1: empty); `parents` int32 [rows]."""
        self._call("xlpk_pages_fork", stream, row=parents, row_name="parents", workspace=True)

    def reserve(self, want, stream=None) -> None:
        """xlpk_pages_reserve: pages so that row r can hold want[r] positions; `want` int32 [rows].
        Pages that a row shares with others are not copied first."""
        self._call("xlpk_pages_reserve", stream, row=want, row_name="want")

    def trim(self, window: int, sinks: int = 0, stream=None) -> None:
        """xlpk_pages_trim: give back the pages a sliding window has passed (decode_attention's;
        Engine's decode has none and stops at a page that is gone)."""
        self._call("xlpk_pages_trim", stream, _int32(window, "window"), _int32(sinks, "sinks"))

    def compact(self, stream=None):
        """xlpk_pages_compact: move the live pages to the lowest numbers; returns the new
        number of every page, int32 [n_pages] (-1: free)."""
        remap = _on(self._device, stream, (), lambda _: _strided((self._pages_n,), (1,), torch.int32))
        self._call("xlpk_pages_compact", stream, remap.data_ptr(), workspace=True)
        return remap

    def copy(self, src, dst, stream=None) -> None:
        """xlpk_pages_copy: page src[i] to page dst[i] in every layer (host integers)."""
        src, dst = [_int32(p, "a page") for p in src], [_int32(p, "a page") for p in dst]
        n = len(src)
        if len(dst) != n:
            _refuse("src and dst of different lengths")
        self._call("xlpk_pages_copy", stream, (C.c_int32 * n)(*src), (C.c_int32 * n)(*dst), n)

    def check(self) -> None:
        """Waits for the calls so far, on whatever streams they were made; raises what stopped one
        of them, and lets the pool go on.  (The streams have to exist still.  Replays of a captured
        graph are calls of the stream that it was replayed on, which the caller has to wait for.)"""
        with torch.cuda.device(self._device):
            here = torch.cuda.current_stream()
            for handle in self._streams - {here.cuda_stream}:
                there = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
                with torch.cuda.stream(there):
                    recording = torch.cuda.is_current_stream_capturing()   # what it records has not run
                if not recording:
                    here.wait_stream(there)
                    self._streams.discard(handle)
            st = int(self.status[0])
            if st != _abi.XLPK_OK:
                self.status[:1] = 0
                here.synchronize()     # before any stream's next call
                raise XlpkError(st, "page pool", detail="the call that met it, and those after it, changed nothing")


# ---- log probabilities

class TokenLogprobs(NamedTuple):
    logprob: torch.Tensor                   # fp32, the tokens' shape
    entropy: torch.Tensor                   # fp32, of each row's distribution, in nats
    rank: torch.Tensor                      # int32, tokens that come before this one (0: the most probable)
    top_ids: Optional[torch.Tensor]         # int32 [..., top_k]
    top_logprobs: Optional[torch.Tensor]    # fp32 [..., top_k]


def token_logprobs(logits, tokens, top_k: int = 0, stream=None) -> TokenLogprobs:
    """xlpk_token_logprobs: log probabilities of `tokens` under `logits`.

    `logits` [..., vocab] fp32 or bf16, as a decode writes them ([steps][B][vocab]),
    rows at any stride; `tokens` int32 of the leading shape.  top_k <= 64
    alternatives, best first, ties by the lower id.  Masked logits are -inf, or finite
    and far below the others.
    """
    if not isinstance(logits, torch.Tensor) or logits.dim() < 1 or logits.dtype not in _IO or not logits.is_cuda:
        _refuse("logits must be an fp32 or bf16 CUDA tensor [..., vocab]")
    dev, vocab, dims = logits.get_device(), logits.shape[-1], logits.dim()
    _tensor(tokens, "tokens", dims - 1, _I32, dev)
    if tokens.shape != logits.shape[:-1] or not tokens.is_contiguous():
        _refuse("tokens must be contiguous, one for each row of logits")
    if vocab == 0 or (vocab > 1 and logits.stride(-1) != 1):
        _refuse("rows of logits must be contiguous")
    rows, top_k = tokens.numel(), _int32(top_k, "top_k")
    x = logits
    if dims != 2:
        try:
            x = logits.view(rows, vocab)
        except RuntimeError:
            _refuse("the leading dimensions of logits must step evenly")
    f32, i32 = torch.float32, torch.int32

    def launch(handle):
        shape = tuple(tokens.shape)
        stride = _contiguous(shape)
        logprob, entropy, rank = _strided(shape, stride, f32), _strided(shape, stride, f32), _strided(shape, stride, i32)
        top_ids = top = None
        ids_at = top_at = 0
        if top_k > 0:
            shape, stride = (*shape, top_k), (*[n * top_k for n in stride], 1)
            top_ids, top = _strided(shape, stride, i32), _strided(shape, stride, f32)
            ids_at, top_at = top_ids.data_ptr(), top.data_ptr()
        st = _fn("xlpk_token_logprobs")(
            x.data_ptr(), _IO[x.dtype], rows, vocab, x.stride(0) if rows > 1 else 0, tokens.data_ptr(), top_k,
            logprob.data_ptr(), entropy.data_ptr(), rank.data_ptr(), ids_at, top_at, handle)
        if st:
            _check(st, "xlpk_token_logprobs")
        return TokenLogprobs(logprob, entropy, rank, top_ids, top)

    return _on(dev, stream, (logits, tokens), launch)
