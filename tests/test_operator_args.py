"""Refusals of the stand-alone operators: bad arguments are turned down on the host,
with a reason, before anything reaches a GPU.  CPU only (device pointers are
made-up addresses that no call gets as far as using)."""
import ctypes as C
import os
import subprocess

import pytest
import torch

from persistent_decode_b200 import _abi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20      # a 16-byte aligned stand-in for a device address
INVALID, UNSUPPORTED = _abi.XLPK_ERR_INVALID_ARG, _abi.XLPK_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    from persistent_decode_b200.build import build
    build()
    return _abi.load()


def _attn(**kw):
    a = _abi.xlpk_attention_args(
        q_dev=P, k_dev=P, v_dev=P, page_table_dev=P, seq_lens_dev=P, out_dev=P, q_seq_stride=4 * 64, q_head_stride=64,
        out_seq_stride=4 * 64, out_head_stride=64, k_page_stride=2 * 16 * 64, k_head_stride=16 * 64, k_pos_stride=64,
        v_page_stride=2 * 16 * 64, v_head_stride=16 * 64, v_pos_stride=64, table_stride=8, n_seqs=2, n_q_heads=4,
        n_kv_heads=2, head_dim=64, n_pages=16, page_size=16, table_cols=8, io_dtype=_abi.XLPK_DTYPE_BF16,
        kv_dtype=_abi.XLPK_DTYPE_BF16, scale=0.125, k_scale=1.0, v_scale=1.0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("bad", [
    dict(n_seqs=-1), dict(n_q_heads=0), dict(n_kv_heads=3), dict(page_size=0), dict(n_pages=-1), dict(window=-1),
    dict(sinks=-2), dict(table_cols=-1), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")),
    dict(scale=-1.0), dict(io_dtype=_abi.XLPK_DTYPE_FP8_E4M3), dict(kv_dtype=_abi.XLPK_DTYPE_FP32),
    dict(kv_dtype=_abi.XLPK_DTYPE_FP8_E4M3, k_scale=0.3), dict(kv_dtype=_abi.XLPK_DTYPE_FP8_E4M3, v_scale=2.0 ** 25),
    dict(q_dev=0), dict(q_dev=P + 8), dict(out_dev=P + 4), dict(k_dev=0), dict(v_dev=P + 2), dict(seq_lens_dev=0),
    dict(seq_lens_dev=P + 2), dict(k_new_dev=P), dict(v_new_dev=P), dict(k_pos_stride=65), dict(v_head_stride=4),
    dict(q_head_stride=66), dict(out_seq_stride=1), dict(k_page_stride=-2 * 16 * 64), dict(q_seq_stride=-256),
    dict(table_stride=-8), dict(page_table_dev=0), dict(page_table_dev=0, table_cols=1)],
    ids=lambda d: ",".join(f"{k}={v}" for k, v in d.items()))
def test_attention_refuses_invalid(lib, bad):
    a = _attn(**bad)
    assert lib.xlpk_decode_attention(C.byref(a), P, 1 << 30, None) == INVALID
    assert lib.xlpk_last_cuda_error().startswith(b"xlpk_decode_attention:")


@pytest.mark.parametrize("bad", [dict(head_dim=96), dict(head_dim=256), dict(n_q_heads=34, n_kv_heads=2),
                                 dict(table_cols=1 << 20, page_size=1 << 12),
                                 dict(table_cols=1, page_size=(1 << 31) - 1),
                                 dict(n_seqs=1 << 20, n_q_heads=64, n_kv_heads=64, table_cols=1 << 16)])
def test_attention_refuses_unsupported(lib, bad):
    a = _attn(**bad)
    assert lib.xlpk_decode_attention(C.byref(a), P, 1 << 30, None) == UNSUPPORTED


def test_attention_refuses_heads_past_32_bits(lib):
    # n_q_heads * head_dim is counted in 32 bits where a sequence without positions is written
    a = _attn(n_seqs=1, n_q_heads=1 << 25, n_kv_heads=1 << 25, table_cols=1)
    assert lib.xlpk_decode_attention(C.byref(a), P, 1 << 30, None) == UNSUPPORTED
    assert b"heads" in lib.xlpk_last_cuda_error()


def test_attention_refuses_a_scale_that_overflows(lib):
    for scale in (2.0 ** 127, 3e38):     # times log2(e) it has no place in fp32
        assert lib.xlpk_decode_attention(C.byref(_attn(scale=scale)), P, 1 << 30, None) == INVALID
        assert b"scale" in lib.xlpk_last_cuda_error()


def test_attention_workspace(lib):
    a = _attn()
    n = lib.xlpk_decode_attention_workspace(C.byref(a))
    assert 0 < n < 1 << 27
    assert lib.xlpk_decode_attention_workspace(C.byref(_attn(n_q_heads=0))) == 0
    assert lib.xlpk_decode_attention_workspace(None) == 0
    for ws, size in ((0, n), (P + 8, n), (P, n - 1), (P, 0)):
        assert lib.xlpk_decode_attention(C.byref(a), ws, size, None) == INVALID
        assert b"workspace" in lib.xlpk_last_cuda_error()
    assert lib.xlpk_decode_attention(None, P, n, None) == INVALID


def _pool(**kw):
    p = _abi.xlpk_page_pool(P, P, P, P, P, P, 2, 16, 2, 16, 128, 4, 8)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def _page_calls(lib, p, ws=P, size=1 << 20):
    one = (C.c_int32 * 1)(1)
    two = (C.c_int32 * 1)(2)
    ref = C.byref(p) if p is not None else None
    return {"fork": lambda: lib.xlpk_pages_fork(ref, P, ws, size, None),
            "compact": lambda: lib.xlpk_pages_compact(ref, P, ws, size, None),
            "reserve": lambda: lib.xlpk_pages_reserve(ref, P, None),
            "trim": lambda: lib.xlpk_pages_trim(ref, 8, 0, None),
            "copy": lambda: lib.xlpk_pages_copy(ref, one, two, 1, None)}


@pytest.mark.parametrize("bad", [
    dict(n_layers=0), dict(n_pages=0), dict(n_kv_heads=-1), dict(page_size=0), dict(rows=0), dict(cols=0),
    dict(row_bytes=0), dict(row_bytes=24), dict(k_dev=0), dict(v_dev=P + 8), dict(page_table_dev=0),
    dict(seq_lens_dev=P + 1), dict(refs_dev=0), dict(status_dev=0)], ids=str)
def test_pages_refuse_a_bad_pool(lib, bad):
    for name, call in _page_calls(lib, _pool(**bad)).items():
        assert call() == INVALID, name
    for name, call in _page_calls(lib, None).items():
        assert call() == INVALID, name


def test_pages_refuse_large_tables(lib):
    for big in (dict(rows=1025), dict(cols=1 << 20, page_size=1 << 12)):
        for name, call in _page_calls(lib, _pool(**big)).items():
            assert call() == UNSUPPORTED, name


def test_pages_refuse_counts_near_2_31(lib):
    # loops over pages and columns step 1024 at a time, in 32 bits
    for big in (dict(n_pages=(1 << 30) + 1), dict(n_pages=(1 << 31) - 1), dict(cols=(1 << 30) + 1, page_size=1),
                dict(cols=(1 << 31) - 1, page_size=1)):
        for name, call in _page_calls(lib, _pool(**big), size=1 << 40).items():
            assert call() == UNSUPPORTED, (name, big)


def test_pages_refuse_bad_arguments(lib):
    p = _pool()
    n = lib.xlpk_pages_workspace(C.byref(p))
    assert n > 0 and lib.xlpk_pages_workspace(None) == 0
    for ws, size in ((0, n), (P + 4, n), (P, n - 1)):
        calls = _page_calls(lib, p, ws, size)
        assert calls["fork"]() == INVALID and calls["compact"]() == INVALID
    assert lib.xlpk_pages_fork(C.byref(p), 0, P, n, None) == INVALID
    assert lib.xlpk_pages_reserve(C.byref(p), P + 2, None) == INVALID
    assert lib.xlpk_pages_trim(C.byref(p), -1, 0, None) == INVALID
    assert lib.xlpk_pages_trim(C.byref(p), 4, -1, None) == INVALID
    assert lib.xlpk_pages_compact(C.byref(p), P + 1, P, n, None) == INVALID

    def copy(src, dst):
        k = len(src)
        return lib.xlpk_pages_copy(C.byref(p), (C.c_int32 * k)(*src), (C.c_int32 * k)(*dst), k, None)

    # outside the pool; a destination twice; a page both source and destination, in either order
    for src, dst in (([16], [1]), ([1], [-1]), ([1, 2], [3, 3]), ([1, 2], [2, 3]), ([2, 1], [3, 2]), ([4], [4])):
        assert copy(src, dst) == INVALID, (src, dst)
    assert lib.xlpk_pages_copy(C.byref(p), None, None, 1, None) == INVALID
    assert lib.xlpk_pages_copy(C.byref(p), None, None, -1, None) == INVALID


def test_logprobs_refuse_bad_arguments(lib):
    def call(x=P, dtype=_abi.XLPK_DTYPE_FP32, rows=2, vocab=100, stride=100, tok=P, k=5, lp=P, ent=P, rank=P, ids=P, top=P):
        return lib.xlpk_token_logprobs(x, dtype, rows, vocab, stride, tok, k, lp, ent, rank, ids, top, None)

    for bad in (dict(dtype=1), dict(dtype=9), dict(rows=-1), dict(vocab=0), dict(stride=-100), dict(k=-1), dict(k=101),
                dict(x=0), dict(x=P + 2), dict(x=P + 1, dtype=0), dict(tok=0), dict(tok=P + 2), dict(lp=0), dict(ent=P + 2),
                dict(rank=P + 1), dict(ids=0), dict(top=0), dict(top=P + 3)):
        assert call(**bad) == INVALID, bad
        assert lib.xlpk_last_cuda_error().startswith(b"xlpk_token_logprobs:"), bad
    assert call(k=65) == UNSUPPORTED
    assert call(rows=1 << 31) == UNSUPPORTED
    assert call(vocab=(1 << 30) + 1, stride=(1 << 30) + 1) == UNSUPPORTED


def test_struct_layout_matches_header(tmp_path):
    structs = [_abi.xlpk_attention_args, _abi.xlpk_page_pool]
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "xlpk.h"', 'int main(void) {']
    for st in structs:
        lines.append(f'  printf("%zu\\n", sizeof({st.__name__}));')
        lines += [f'  printf("%zu\\n", offsetof({st.__name__}, {f}));' for f, _ in st._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    want = []
    for st in structs:
        want += [C.sizeof(st)] + [getattr(st, f).offset for f, _ in st._fields_]
    assert got == want


def test_python_refuses_what_is_not_on_a_gpu():
    from persistent_decode_b200 import PagePool, decode_attention, token_logprobs
    with pytest.raises(ValueError):
        decode_attention(torch.zeros(1, 4, 64), torch.zeros(1, 2, 8, 64), torch.zeros(1, 2, 8, 64),
                         torch.ones(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        token_logprobs(torch.zeros(2, 100), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        PagePool(torch.zeros(1, 4, 2, 8, 64), torch.zeros(1, 4, 2, 8, 64), torch.zeros(1, 4, dtype=torch.int32),
                 torch.zeros(1, dtype=torch.int32))


def test_integers_are_not_rounded():
    # a window, an alternative count or a page of 2.5 is refused, not taken for 2
    from persistent_decode_b200.ops import _int32
    import numpy as np
    assert [_int32(v, "x") for v in (3, -1, True, np.int64(7), torch.tensor(5))] == [3, -1, 1, 7, 5]
    for bad in (2.5, 2.0, float("nan"), "3", None, torch.tensor(2.0), 1 << 31, -(1 << 31) - 1):
        with pytest.raises(ValueError):
            _int32(bad, "x")


def test_an_error_does_not_quote_another_calls_refusal(lib):
    from persistent_decode_b200 import XlpkError
    assert lib.xlpk_token_logprobs(P, _abi.XLPK_DTYPE_FP32, 1, 100, 100, P, 65, P, None, None, P, P, None) == UNSUPPORTED
    assert "top_k over 64" in str(XlpkError(UNSUPPORTED, "xlpk_token_logprobs"))
    assert str(XlpkError(_abi.XLPK_ERR_KV_FULL, "xlpk_decode")) == "xlpk_decode: XLPK_ERR_KV_FULL"
    assert _page_calls(lib, _pool(rows=1025))["fork"]() == UNSUPPORTED
    assert "1024 rows" in str(XlpkError(UNSUPPORTED, "xlpk_pages_fork"))      # (its text begins "xlpk_pages:")
    assert "1024 rows" not in str(XlpkError(INVALID, "xlpk_create"))
