"""Calls of the stand-alone operators that must be refused or taken for what
they say, checked on the host (no GPU needed: nothing here reaches a kernel)."""
import ctypes

import pytest

from tests.test_ops_refusals import P, _args, _desc, river  # noqa: F401

torch = pytest.importorskip("torch")


def _shared(river, **kw):
    a, d = _args(kw), _desc(river, **kw)
    return river._lib.rl_shared_prefix_attention(ctypes.byref(d), P(a["q"]), P(a["pk"]), P(a["pv"]), a["prefix"],
                                                 (ctypes.c_int64 * 4)(*a["ps"]), P(a["k"]), P(a["v"]), P(a["kv_len"]),
                                                 P(a["out"]), P(a["lse"]), P(a["ws"]), 1 << 40, None, None)


@pytest.mark.parametrize("ps", [(1024, 0, 1024, 64), (1024, 64, 1024, 0), (0, 0, 0, 0)])
def test_prefix_token_stride_zero_is_refused(river, ps):
    """Rows 64 elements apart would be read behind a buffer of one row."""
    assert _shared(river, ps=ps) == river.RL_ERR_UNSUPPORTED
    assert "token strides" in river.rl_last_error()
