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


def derivatives_refused(river, call, ops, which, plain):
    """Each operand of `which` in turn with a gradient, with a tangent, and
    plain beside an open dual level (`plain(call)`: what holds then)."""
    import torch.autograd.forward_ad as fw
    for i in which:
        x = ops[i]

        def given(y):
            return lambda: call(*ops[:i], y, *ops[i + 1:])

        def refused(y):
            with pytest.raises(river.RiverError) as e:
                given(y)()
            assert e.value.status == river.RL_ERR_UNSUPPORTED, e.value
        refused(x.clone().requires_grad_())
        with fw.dual_level():
            refused(fw.make_dual(x, torch.ones_like(x)))
            with torch.no_grad():  # (which does not stop forward mode)
                refused(fw.make_dual(x, torch.ones_like(x)))
            plain(given(x))


def forms(river, device):
    """The Python forms as functions of their floating-point operands."""
    n = torch.ones(1, dtype=torch.int32, device=device)

    def zeros(*shape):
        return torch.zeros(shape, dtype=torch.bfloat16, device=device)
    return [(river.token_logprobs, [zeros(2, 10)]),
            (lambda q, k, v: river.window_attention(q, k, v, n, 4), [zeros(1, 1, 4, 64), zeros(1, 2, 8, 64), zeros(1, 2, 8, 64)]),
            (lambda q, pk, pv, k, v: river.shared_prefix_attention(q, pk, pv, k, v, n),
             [zeros(1, 4, 64), zeros(2, 8, 64), zeros(2, 8, 64), zeros(1, 2, 8, 64), zeros(1, 2, 8, 64)])]


def test_operands_with_derivatives_are_refused(river):
    """A tangent (forward mode) is no more dropped in silence than a gradient."""
    def plain(call):
        with pytest.raises(river.RiverError) as e:
            call()
        assert e.value.status == river.RL_ERR_INVALID_ARG  # (host tensors)
    for call, ops in forms(river, "cpu"):
        derivatives_refused(river, call, ops, [0], plain)


class Recorder:
    """Stands in for the library: every call's 32-bit arguments as C sees them."""

    def __init__(self, lib):
        self.lib, self.seen = lib, []

    def __getattr__(self, name):
        real = getattr(self.lib, name)

        def call(*args):
            self.seen.append([t(a).value if t is ctypes.c_int32 else None for t, a in zip(real.argtypes, args)])
            return 0
        return call


def test_windows_and_prefixes_beyond_32_bits(river, monkeypatch):
    """2^32 + 5 is no window of 5, and -2^31 - 1 none at all."""
    rec = Recorder(river._lib)
    monkeypatch.setattr(river, "_lib", rec)
    kv = object.__new__(river.KVCache)
    kv.handle = None
    big = 2**31 - 1
    for n, c in ((0, 0), (5, 5), (big, big), (2**32, big), (2**32 + 5, big), (-1, -1), (-2**31 - 1, -1), (-2**32 + 5, -1)):
        kv.set_window(n, n)
        assert rec.seen.pop()[1:] == [c, c]
        kv.share_prefix(n)
        assert rec.seen.pop()[1:] == [c]
        river.rl_window_attention(_desc(river), None, None, None, None, None, n, n, None, None, stream=Stream)
        assert rec.seen.pop()[6:8] == [c, c]


class Stream:
    cuda_stream = None


def test_sizes_beyond_32_bits_are_refused(river, monkeypatch):
    """A size is never taken for its low 32 bits (2^32 + 2 rows for two)."""
    n = 2**32 + 2

    def refused(call, *args, **kw):
        with pytest.raises(river.RiverError) as e:
            call(*args, **kw)
        assert e.value.status == river.RL_ERR_UNSUPPORTED, e.value
    for shape in ((n, 1), (1, n)):  # (meta tensors: sizes without memory)
        refused(river.token_logprobs, torch.empty(shape, dtype=torch.bfloat16, device="meta"))
    q, k = torch.zeros((1, 1, 4, 64), dtype=torch.bfloat16), torch.zeros((1, 2, 8, 64), dtype=torch.bfloat16)
    for bad in (k[:, :, :1].expand(1, 2, n, 64), k[:, :1].expand(1, n, 8, 64)):
        refused(river._attn_desc, "x", q, bad, bad, q, None)
    river._attn_desc("x", q, k, k, q, None)
    # behind the check of devices, which these host tensors pass by
    monkeypatch.setattr(river, "_operands", lambda name, tensors: 0)
    refused(river.shared_prefix_attention, q[0], k[0, :, :1].expand(2, n, 64), k[0, :, :1].expand(2, n, 64), k, k,
            torch.ones(1, dtype=torch.int32))


def test_a_scale_that_rounds_to_zero_is_not_the_default(river):
    q, k = torch.zeros((1, 1, 4, 64), dtype=torch.bfloat16), torch.zeros((1, 2, 8, 64), dtype=torch.bfloat16)
    for scale in (1e-50, 2.0**-150, 0.0, -1.0, float("nan")):
        with pytest.raises(river.RiverError) as e:
            river._attn_desc("x", q, k, k, q, scale)
        assert e.value.status == river.RL_ERR_INVALID_ARG
    assert river._attn_desc("x", q, k, k, q, None).scale == 0.0  # (0 asks for the default)
    assert river._attn_desc("x", q, k, k, q, 2.0**-149).scale == 2.0**-149


def test_prefill_score_refuses_tokens_it_cannot_read(river):
    """Before the library sees an address (no model is needed for that)."""
    t = torch.zeros((2, 6), dtype=torch.int32)
    for bad in (t[0], t.long(), t.t(), t[:, ::2], t):  # (the last: host memory)
        with pytest.raises(river.RiverError) as e:
            river.prefill_score(None, None, bad, None)
        assert e.value.status == river.RL_ERR_INVALID_ARG


def test_a_buffer_that_requires_a_gradient_is_refused(river):
    t = torch.zeros(3).requires_grad_()
    with pytest.raises(river.RiverError) as e:
        river._buffer({"lse": t}, "lse", (3,), t, torch.float32, None, "x")
    assert e.value.status == river.RL_ERR_UNSUPPORTED
    with torch.no_grad():
        assert river._buffer({"lse": t}, "lse", (3,), t, torch.float32, None, "x") is t
