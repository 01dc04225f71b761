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
"""
from __future__ import annotations

import contextlib
import ctypes as C
import math
from typing import NamedTuple, Optional

import torch

from . import _abi
from .engine import XlpkError, _check, _ptr, lib

_IO = {torch.float32: _abi.XLPK_DTYPE_FP32, torch.bfloat16: _abi.XLPK_DTYPE_BF16}
_KV = {torch.bfloat16: _abi.XLPK_DTYPE_BF16, torch.uint8: _abi.XLPK_DTYPE_FP8_E4M3,
       torch.float8_e4m3fn: _abi.XLPK_DTYPE_FP8_E4M3}


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _tensor(t, name: str, dim: int, dtypes, device) -> None:
    _need(isinstance(t, torch.Tensor) and t.is_cuda, f"{name} must be a CUDA tensor")
    _need(device is None or t.device == device, f"{name} is on {t.device}, not on {device}")
    _need(t.dim() == dim and t.dtype in dtypes, f"{name}: {t.dim()}-d {t.dtype}, want {dim}-d {' or '.join(map(str, dtypes))}")


def _steps(t):
    """Strides of all but the last dimension (0 where there is nothing to step to)."""
    return [s if n > 1 else 0 for n, s in zip(t.shape[:-1], t.stride()[:-1])]


def _distinct(t) -> bool:
    """No two elements share memory (sufficient: every stride steps over all inner ones)."""
    reach = 0
    for s, n in sorted((s, n) for s, n in zip(t.stride(), t.shape) if n > 1):
        if s <= reach:
            return False
        reach += s * (n - 1)
    return True


@contextlib.contextmanager
def _on(device, stream, tensors=()):
    """The stream handle to launch on; allocations inside belong to that stream."""
    if stream is None:
        with torch.cuda.device(device):
            yield torch.cuda.current_stream(device).cuda_stream or None
        return
    _need(stream.device == device, f"stream is on {stream.device}, the tensors on {device}")
    with torch.cuda.stream(stream):
        for t in tensors:
            if t is not None:
                t.record_stream(stream)   # their memory is not reused before this use of it
        yield stream.cuda_stream or None


# ---- attention

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
    _tensor(q, "q", 3, _IO, None)
    dev = q.device
    B, H, D = q.shape
    _tensor(k_cache, "k_cache", 4, _KV, dev)
    _tensor(v_cache, "v_cache", 4, (k_cache.dtype,), dev)
    n_pages, KH, P, dc = k_cache.shape
    _need(v_cache.shape == k_cache.shape and dc == D, f"caches of {tuple(k_cache.shape)} and {tuple(v_cache.shape)} for head_dim {D}")
    _tensor(seq_lens, "seq_lens", 1, (torch.int32,), dev)
    _need(seq_lens.shape[0] == B and (B < 2 or seq_lens.stride(0) == 1), "seq_lens must be a contiguous [B]")
    _need(D > 0 and all(t.stride(-1) == 1 for t in (q, k_cache, v_cache)), "rows of head_dim must be contiguous")
    a = _abi.xlpk_attention_args()
    if page_table is not None:
        _tensor(page_table, "page_table", 2, (torch.int32,), dev)
        _need(page_table.shape[0] == B and (page_table.shape[1] < 2 or page_table.stride(1) == 1),
              "page_table must be [B][pages] with contiguous rows")
        a.page_table_dev, a.table_cols = _ptr(page_table), page_table.shape[1]
        a.table_stride = page_table.stride(0) if B > 1 else 0
    else:
        _need(n_pages == B, f"a contiguous cache of {n_pages} sequences for {B} queries")
        a.table_cols = 1
    _need((k_new is None) == (v_new is None), "k_new and v_new come together")
    if k_new is not None:
        for t, name in ((k_new, "k_new"), (v_new, "v_new")):
            _tensor(t, name, 3, (q.dtype,), dev)
            _need(t.shape == (B, KH, D) and t.stride(-1) == 1, f"{name} must be [B][n_kv][d] with contiguous rows")
        _need(_distinct(k_cache) and _distinct(v_cache), "a cache that is written must not overlap itself")
        a.k_new_dev, a.v_new_dev = _ptr(k_new), _ptr(v_new)
        a.new_k_seq_stride, a.new_k_head_stride = _steps(k_new)
        a.new_v_seq_stride, a.new_v_head_stride = _steps(v_new)
    if out is not None:
        _tensor(out, "out", 3, (q.dtype,), dev)
        _need(out.shape == q.shape and out.stride(-1) == 1 and _distinct(out), "out must be [B][n_q][d] with rows of its own")
    if status is not None:
        _tensor(status, "status", 1, (torch.int32,), dev)
        _need(status.shape[0] >= 1, "status must hold one int32")
    a.q_dev, a.k_dev, a.v_dev, a.seq_lens_dev, a.status_dev = (_ptr(t) for t in (q, k_cache, v_cache, seq_lens, status))
    a.q_seq_stride, a.q_head_stride = _steps(q)
    a.k_page_stride, a.k_head_stride, a.k_pos_stride = _steps(k_cache)
    a.v_page_stride, a.v_head_stride, a.v_pos_stride = _steps(v_cache)
    a.n_seqs, a.n_q_heads, a.n_kv_heads, a.head_dim, a.n_pages, a.page_size = B, H, KH, D, n_pages, P
    a.io_dtype, a.kv_dtype = _IO[q.dtype], _KV[k_cache.dtype]
    a.window, a.sinks, a.k_scale, a.v_scale = int(window), int(sinks), float(k_scale), float(v_scale)
    a.scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    with _on(dev, stream, (q, k_cache, v_cache, seq_lens, page_table, k_new, v_new, out, status)) as handle:
        if out is None:
            out = torch.empty((B, H, D), dtype=q.dtype, device=dev)
        a.out_dev = _ptr(out)
        a.out_seq_stride, a.out_head_stride = _steps(out)
        lse = torch.empty((B, H), dtype=torch.float32, device=dev) if return_lse else None
        a.lse_dev = _ptr(lse)
        n = lib.xlpk_decode_attention_workspace(C.byref(a))
        ws = torch.empty(max(n, 16), dtype=torch.uint8, device=dev)
        _check(lib.xlpk_decode_attention(C.byref(a), _ptr(ws), ws.numel(), handle), "xlpk_decode_attention")
    return (out, lse) if return_lse else out


# ---- pages

class PagePool:
    """The pages of a paged cache and who holds them (xlpk_page_pool).

    `k`, `v` [L][n_pages][n_kv][page_size][d] as the engine's pools; `page_table`
    int32 [rows][cols] (-1: no page), `seq_lens` int32 [rows], `refs` int32
    [n_pages] (None: counted from the table; the caller may add references of its
    own).  All stay the caller's and are updated in place.  Calls are
    asynchronous; one that cannot be done changes nothing and sets `status`
    (int32 [1]), which stops later calls until `check()` has reported it.
    """

    def __init__(self, k, v, page_table, seq_lens, refs=None, status=None):
        _tensor(k, "k", 5, _KV, None)
        dev = self.device = k.device
        _tensor(v, "v", 5, (k.dtype,), dev)
        _tensor(page_table, "page_table", 2, (torch.int32,), dev)
        _tensor(seq_lens, "seq_lens", 1, (torch.int32,), dev)
        L, n_pages, KH, P, D = k.shape
        if refs is None:
            held = page_table.reshape(-1)
            held = held[(held >= 0) & (held < n_pages)]
            refs = torch.bincount(held, minlength=n_pages).to(torch.int32)
        if status is None:
            status = torch.zeros(1, dtype=torch.int32, device=dev)
        _tensor(refs, "refs", 1, (torch.int32,), dev)
        _tensor(status, "status", 1, (torch.int32,), dev)
        rows, cols = page_table.shape
        _need(v.shape == k.shape, f"pools of {tuple(k.shape)} and {tuple(v.shape)}")
        _need(seq_lens.shape[0] == rows and refs.shape[0] == n_pages and status.shape[0] >= 1,
              "seq_lens must have the table's rows, refs the pool's pages")
        _need(all(t.is_contiguous() for t in (k, v, page_table, seq_lens, refs)), "pool tensors must be contiguous")
        self.k, self.v, self.page_table, self.seq_lens, self.refs, self.status = k, v, page_table, seq_lens, refs, status
        self._c = _abi.xlpk_page_pool(_ptr(k), _ptr(v), _ptr(page_table), _ptr(seq_lens), _ptr(refs), _ptr(status),
                                      L, n_pages, KH, P, D * k.element_size(), rows, cols)

    def _call(self, name, stream, *args, workspace: bool = False, uses=()):
        with _on(self.device, stream, (self.k, self.v, self.page_table, self.seq_lens, self.refs, self.status, *uses)) as handle:
            if workspace:
                n = lib.xlpk_pages_workspace(C.byref(self._c))
                ws = torch.empty(max(n, 16), dtype=torch.uint8, device=self.device)
                args = (*args, _ptr(ws), ws.numel())
            _check(getattr(lib, name)(C.byref(self._c), *args, handle), name)

    def _rows(self, t, name: str):
        _tensor(t, name, 1, (torch.int32,), self.device)
        _need(t.shape[0] == self.page_table.shape[0] and t.is_contiguous(), f"{name} must be a contiguous [rows]")
        return _ptr(t)

    def fork(self, parents, stream=None) -> None:
        """xlpk_pages_fork: row r becomes what row parents[r] was (-1: empty); `parents` int32 [rows]."""
        self._call("xlpk_pages_fork", stream, self._rows(parents, "parents"), workspace=True, uses=(parents,))

    def reserve(self, want, stream=None) -> None:
        """xlpk_pages_reserve: pages so that row r can hold want[r] positions; `want` int32 [rows]."""
        self._call("xlpk_pages_reserve", stream, self._rows(want, "want"), uses=(want,))

    def trim(self, window: int, sinks: int = 0, stream=None) -> None:
        """xlpk_pages_trim: give back the pages a sliding window has passed."""
        self._call("xlpk_pages_trim", stream, int(window), int(sinks))

    def compact(self, stream=None):
        """xlpk_pages_compact: move the live pages to the lowest numbers; returns the new
        number of every page, int32 [n_pages] (-1: free)."""
        with _on(self.device, stream):
            remap = torch.empty(self.refs.shape[0], dtype=torch.int32, device=self.device)
        self._call("xlpk_pages_compact", stream, _ptr(remap), workspace=True)
        return remap

    def copy(self, src, dst, stream=None) -> None:
        """xlpk_pages_copy: page src[i] to page dst[i] in every layer (host integers)."""
        src, dst = [int(p) for p in src], [int(p) for p in dst]
        _need(len(src) == len(dst), "src and dst of different lengths")
        n = len(src)
        self._call("xlpk_pages_copy", stream, (C.c_int32 * n)(*src), (C.c_int32 * n)(*dst), n)

    def check(self) -> None:
        """Waits for the calls so far; raises what stopped one of them, and lets the pool go on."""
        st = int(self.status[0])
        if st != _abi.XLPK_OK:
            self.status[:1] = 0
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
    alternatives, best first, ties by the lower id.  Masked logits are -inf.
    """
    _need(isinstance(logits, torch.Tensor) and logits.is_cuda and logits.dim() >= 1 and logits.dtype in _IO,
          "logits must be an fp32 or bf16 CUDA tensor [..., vocab]")
    dev, vocab = logits.device, logits.shape[-1]
    _tensor(tokens, "tokens", logits.dim() - 1, (torch.int32,), dev)
    _need(tokens.shape == logits.shape[:-1] and tokens.is_contiguous(), "tokens must be contiguous, one for each row of logits")
    _need(vocab > 0 and (vocab == 1 or logits.stride(-1) == 1), "rows of logits must be contiguous")
    rows = tokens.numel()
    try:
        x = logits if logits.dim() == 2 else logits.view(rows, vocab)
    except RuntimeError:
        raise ValueError("the leading dimensions of logits must step evenly") from None
    shape = tuple(tokens.shape)
    with _on(dev, stream, (logits, tokens)) as handle:
        f32, i32 = dict(dtype=torch.float32, device=dev), dict(dtype=torch.int32, device=dev)
        logprob, entropy, rank = torch.empty(shape, **f32), torch.empty(shape, **f32), torch.empty(shape, **i32)
        top_ids = torch.empty((*shape, top_k), **i32) if top_k > 0 else None
        top = torch.empty((*shape, top_k), **f32) if top_k > 0 else None
        _check(lib.xlpk_token_logprobs(_ptr(x), _IO[x.dtype], rows, vocab, x.stride(0) if rows > 1 else 0, _ptr(tokens),
                                       int(top_k), _ptr(logprob), _ptr(entropy), _ptr(rank), _ptr(top_ids), _ptr(top),
                                       handle), "xlpk_token_logprobs")
    return TokenLogprobs(logprob, entropy, rank, top_ids, top)
