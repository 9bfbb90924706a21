"""What the stand-alone operators refuse, checked on the host before anything
is enqueued (no GPU needed: every call here must be refused)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def river():
    import __graft_entry__
    __graft_entry__.build()
    import early_exit_decoding_gb300 as r
    return r


P = ctypes.c_void_p
A = 0x10000  # an aligned address that no refused call reads


def _logprobs(river, **kw):
    a = dict(logits=A, dtype=0, rows=2, vocab=100, stride=100, tokens=A, n_tok=1, top_k=2, lse=A, ent=A, lp=A,
             ids=A, tlp=A, err=None)
    a.update(kw)
    return river._lib.rl_token_logprobs(P(a["logits"]), a["dtype"], a["rows"], a["vocab"], a["stride"], P(a["tokens"]),
                                        a["n_tok"], a["top_k"], P(a["lse"]), P(a["ent"]), P(a["lp"]), P(a["ids"]),
                                        P(a["tlp"]), P(a["err"]), None)


@pytest.mark.parametrize("kw", [dict(logits=None), dict(dtype=3), dict(dtype=-1), dict(rows=0), dict(vocab=0), dict(stride=99),
                                dict(n_tok=-1), dict(n_tok=257), dict(tokens=None), dict(lp=None), dict(top_k=-1),
                                dict(top_k=33), dict(vocab=1, top_k=2), dict(ids=None), dict(tlp=None), dict(logits=A + 2)])
def test_logprobs_refuses(river, kw):
    assert _logprobs(river, **kw) == river.RL_ERR_INVALID_ARG
    assert "rl_token_logprobs" in river.rl_last_error()


def _desc(river, **kw):
    a = dict(kv_dtype=river.RL_DT_BF16, q_dtype=river.RL_DT_BF16, batch=2, q_len=1, n_q_heads=4, n_kv_heads=2, head_dim=64,
             kv_capacity=32, scale=0.0, q_stride=(256, 256, 64), out_stride=(256, 256, 64), k_stride=(4096, 2048, 64),
             v_stride=(4096, 2048, 64))
    a.update({k: v for k, v in kw.items() if k in a})
    d = river.rl_attn_desc()
    for k, v in a.items():
        if k.endswith("_stride"):
            getattr(d, k)[:] = list(v)
        else:
            setattr(d, k, v)
    return d


SHARED = [
    (dict(kv_dtype=0), "UNSUPPORTED"), (dict(q_dtype=2), "UNSUPPORTED"), (dict(batch=0), "INVALID_ARG"),
    (dict(q_len=0), "INVALID_ARG"), (dict(n_kv_heads=0), "INVALID_ARG"), (dict(kv_capacity=0), "INVALID_ARG"),
    (dict(head_dim=96), "UNSUPPORTED"), (dict(n_kv_heads=3), "UNSUPPORTED"), (dict(scale=-1.0), "INVALID_ARG"),
    (dict(scale=float("nan")), "INVALID_ARG"), (dict(q_stride=(256, 256, 60)), "UNSUPPORTED"),
    (dict(out_stride=(-256, 256, 64)), "UNSUPPORTED"), (dict(k_stride=(4096, 2048, 68)), "UNSUPPORTED"),
    (dict(v_stride=(1 << 39, 2048, 64)), "UNSUPPORTED"), (dict(k_stride=(4096, 2048, 0)), "UNSUPPORTED"),
    (dict(batch=1 << 20, q_len=1 << 12), "UNSUPPORTED"),
    (dict(kv_capacity=(1 << 30) + 1), "UNSUPPORTED"), (dict(out_stride=(0, 256, 64)), "INVALID_ARG"),
    (dict(out_stride=(256, 256, 0)), "INVALID_ARG"), (dict(out_stride=(128, 256, 64)), "INVALID_ARG"),
    (dict(out_stride=(64, 256, 64)), "INVALID_ARG"),
    (dict(q=None), "INVALID_ARG"), (dict(k=None), "INVALID_ARG"), (dict(v=None), "INVALID_ARG"),
    (dict(kv_len=None), "INVALID_ARG"), (dict(out=None), "INVALID_ARG"), (dict(q=A + 8), "UNSUPPORTED"),
    (dict(k=A + 2), "UNSUPPORTED"), (dict(out=A + 4 * 4096 + 8), "UNSUPPORTED"), (dict(out=A), "INVALID_ARG"),
]


def _args(kw):
    a = dict(q=A, k=A + 4096, v=A + 8192, kv_len=A + 12288, q_len=None, window=8, sinks=2, out=A + 16384, lse=None, pk=A + 20480,
             pv=A + 24576, prefix=16, ps=(1024, 64, 1024, 64), ws=A + 28672, ws_bytes=None)
    a.update({k: v for k, v in kw.items() if k in a})
    return a


@pytest.mark.parametrize("kw,status", SHARED + [(dict(window=0), "INVALID_ARG"), (dict(sinks=-1), "INVALID_ARG")])
def test_window_attention_refuses(river, kw, status):
    a, d = _args(kw), _desc(river, **kw)
    st = river._lib.rl_window_attention(ctypes.byref(d), P(a["q"]), P(a["k"]), P(a["v"]), P(a["kv_len"]), P(a["q_len"]),
                                        a["window"], a["sinks"], P(a["out"]), P(a["lse"]), None, None)
    assert st == getattr(river, "RL_ERR_" + status), river.rl_last_error()


@pytest.mark.parametrize("kw,status", [x for x in SHARED if "q_len" not in x[0]] + [
    (dict(q_len=2, out_stride=(512, 256, 64)), "UNSUPPORTED"), (dict(prefix=-1), "INVALID_ARG"), (dict(prefix=(1 << 30) + 1), "UNSUPPORTED"), (dict(pk=None), "INVALID_ARG"), (dict(pv=A + 24576 + 8), "UNSUPPORTED"),
    (dict(ps=(1024, 65, 1024, 64)), "UNSUPPORTED"), (dict(ws=None), "INVALID_ARG"), (dict(ws_bytes=16), "INVALID_ARG"),
    (dict(ws=A + 28672 + 4), "UNSUPPORTED")])
def test_shared_prefix_attention_refuses(river, kw, status):
    a, d = _args(kw), _desc(river, **kw)
    n = ctypes.c_uint64(1 << 40)
    if a["ws_bytes"] is None:
        river._lib.rl_shared_prefix_workspace(ctypes.byref(d), max(0, a["prefix"]), ctypes.byref(n))
    else:
        n.value = a["ws_bytes"]
    st = river._lib.rl_shared_prefix_attention(ctypes.byref(d), P(a["q"]), P(a["pk"]), P(a["pv"]), a["prefix"],
                                               (ctypes.c_int64 * 4)(*a["ps"]), P(a["k"]), P(a["v"]), P(a["kv_len"]), P(a["out"]),
                                               P(a["lse"]), P(a["ws"]), n, None, None)
    assert st == getattr(river, "RL_ERR_" + status), river.rl_last_error()


def test_null_descriptor(river):
    assert river._lib.rl_window_attention(None, P(A), P(A), P(A), P(A), None, 1, 0, P(A), None, None, None) == river.RL_ERR_INVALID_ARG
    n = ctypes.c_uint64()
    assert river._lib.rl_shared_prefix_workspace(None, 1, ctypes.byref(n)) == river.RL_ERR_INVALID_ARG


def test_python_forms_refuse_host_tensors_and_bad_shapes(river):
    """Host tensors never reach the library."""
    x = torch.zeros((2, 10))
    with pytest.raises(river.RiverError) as e:
        river.token_logprobs(x)
    assert e.value.status == river.RL_ERR_INVALID_ARG
    with pytest.raises(river.RiverError):
        river.token_logprobs(torch.zeros((2, 10), dtype=torch.float64))
    with pytest.raises(river.RiverError):
        river.token_logprobs(torch.zeros((10, 2)).t())
    q = torch.zeros((1, 1, 4, 64), dtype=torch.bfloat16)
    k = torch.zeros((1, 2, 8, 64), dtype=torch.bfloat16)
    with pytest.raises(river.RiverError):
        river.window_attention(q, k, k, torch.ones(1, dtype=torch.int32), 4)
    with pytest.raises(river.RiverError):
        river.shared_prefix_attention(q[0], k[0], k[0], k, k, torch.ones(1, dtype=torch.int32))
