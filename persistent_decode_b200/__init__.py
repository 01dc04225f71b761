"""Persistent single-kernel small-batch decode for B200 (sm_100a).

The compute path is the C-ABI library libxlpk.so (include/xlpk.h); this
package only marshals arguments to it.  The library is loaded on first use
and its absence raises ImportError: there is no CPU fallback.  The stand-alone
operators around the decode (decode_attention, PagePool, token_logprobs) are in
ops.py.
"""
from ._abi import LIB_PATH, load  # noqa: F401
from .engine import Engine, XlpkError, get_lib, lib, tc_gemm_tile  # noqa: F401


def __getattr__(name):
    # ops.py needs torch, the modules above do not
    if name in ("decode_attention", "PagePool", "token_logprobs", "TokenLogprobs"):
        from . import ops
        return globals().setdefault(name, getattr(ops, name))
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
