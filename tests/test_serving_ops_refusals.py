"""What the packed and paged operators and sampling refuse, checked on the host
before anything is enqueued (no GPU needed: every call here must be refused)."""
import ctypes

import pytest

from tests.test_ops_refusals import A, P, river  # noqa: F401

torch = pytest.importorskip("torch")


def _packed(river, **kw):
    a = dict(dtype=river.RL_DT_BF16, batch=2, rows=8, max_rows=0, n_q_heads=4, n_kv_heads=2, head_dim=64, scale=0.0,
             q_stride=(256, 64), k_stride=(128, 64), v_stride=(128, 64), out_stride=(256, 64))
    a.update({k: v for k, v in kw.items() if k in a})
    d = river.rl_packed_desc()
    for k, v in a.items():
        if k.endswith("_stride"):
            getattr(d, k)[:] = list(v)
        else:
            setattr(d, k, v)
    return d


def _cache(river, **kw):
    a = dict(n_pages=4, page=16, k_codes=A, k_scale=A + 4096, v_codes=A + 8192, v_scale=A + 12288, code_stride=(1024, 1024),
             scale_stride=(64, 64), d_table=A + 16384, table_stride=3, table_width=3)
    a.update({k: v for k, v in kw.items() if k in a})
    c = river.rl_kv4()
    for k, v in a.items():
        if k.endswith("_stride") and k != "table_stride":
            getattr(c, k)[:] = list(v)
        else:
            setattr(c, k, v)
    return c


def _call(river, name, **kw):
    a = dict(q=A + 20480, k=A + 24576, v=A + 28672, out=A + 32768, start=A + 36864, kv_len=A + 40960, rope=A + 45056, rope_len=9, ro=A + 49152,
             cache=True, desc=True, ws=A + 53248, ws_bytes=1 << 40)
    a.update({k: v for k, v in kw.items() if k in a})
    d, c = _packed(river, **kw), _cache(river, **kw)
    pd, pc = (ctypes.byref(d) if a["desc"] else None), (ctypes.byref(c) if a["cache"] else None)
    if name == "packed":
        return river._lib.rl_packed_attention(pd, P(a["q"]), P(a["k"]), P(a["v"]), P(a["start"]), P(a["out"]), None, None, None)
    if name == "append":
        return river._lib.rl_kv4_append(pc, pd, P(a["start"]), P(a["kv_len"]), P(a["q"]), P(a["k"]), P(a["v"]), P(a["rope"]), a["rope_len"],
                                        P(a["out"]), None, None)
    if name == "read":
        return river._lib.rl_kv4_read(pc, pd, P(a["start"]), P(a["kv_len"]), P(a["k"]), P(a["v"]), None, None)
    return river._lib.rl_kv4_attention(pc, pd, P(a["start"]), P(a["kv_len"]), P(a["q"]), P(a["out"]), None,
                                       P(a["ws"]), a["ws_bytes"], None, None)


ALL = ("packed", "append", "read", "attention")
DESC = [(dict(desc=False), "INVALID_ARG"), (dict(dtype=0), "UNSUPPORTED"), (dict(dtype=3), "UNSUPPORTED"), (dict(batch=0), "INVALID_ARG"),
        (dict(rows=0), "INVALID_ARG"), (dict(max_rows=-1), "INVALID_ARG"), (dict(n_q_heads=0), "INVALID_ARG"), (dict(n_kv_heads=0), "INVALID_ARG"),
        (dict(n_kv_heads=3), "UNSUPPORTED"), (dict(head_dim=96), "UNSUPPORTED"), (dict(scale=-1.0), "INVALID_ARG"),
        (dict(scale=float("nan")), "INVALID_ARG"), (dict(batch=(1 << 16) + 1), "UNSUPPORTED"), (dict(n_kv_heads=2048, n_q_heads=2048), "UNSUPPORTED"), (dict(rows=(1 << 27) + 1), "UNSUPPORTED"),
        (dict(rows=1 << 27, n_q_heads=32), "UNSUPPORTED")]


@pytest.mark.parametrize("name", ALL)
@pytest.mark.parametrize("kw,status", DESC)
def test_descriptor(river, name, kw, status):
    assert _call(river, name, **kw) == getattr(river, "RL_ERR_" + status), river.rl_last_error()


CACHE = [(dict(cache=False), "INVALID_ARG"), (dict(n_pages=0), "INVALID_ARG"), (dict(table_width=0), "INVALID_ARG"), (dict(page=0), "UNSUPPORTED"),
         (dict(page=8), "UNSUPPORTED"), (dict(page=48), "UNSUPPORTED"), (dict(page=512), "UNSUPPORTED"), (dict(table_width=1 << 27, table_stride=1 << 27), "UNSUPPORTED"),
         (dict(k_codes=None), "INVALID_ARG"), (dict(v_scale=None), "INVALID_ARG"), (dict(d_table=None), "INVALID_ARG"), (dict(k_scale=A + 4), "UNSUPPORTED"),
         (dict(v_codes=A + 8), "UNSUPPORTED"), (dict(d_table=A + 2), "UNSUPPORTED"), (dict(table_stride=2), "INVALID_ARG"),
         (dict(table_stride=-3), "INVALID_ARG"), (dict(code_stride=(1023, 1024)), "UNSUPPORTED"), (dict(code_stride=(1024, 512)), "INVALID_ARG"),
         (dict(scale_stride=(60, 64)), "UNSUPPORTED"), (dict(scale_stride=(64, 56)), "INVALID_ARG"), (dict(code_stride=(-1024, 1024)), "INVALID_ARG"),
         (dict(kv_len=None), "INVALID_ARG"), (dict(start=None), "INVALID_ARG")]


@pytest.mark.parametrize("name", ALL[1:])
@pytest.mark.parametrize("kw,status", CACHE)
def test_cache(river, name, kw, status):
    assert _call(river, name, **kw) == getattr(river, "RL_ERR_" + status), river.rl_last_error()


@pytest.mark.parametrize("name,kw,status", [
    ("packed", dict(q=None), "INVALID_ARG"), ("packed", dict(k=None), "INVALID_ARG"), ("packed", dict(v=None), "INVALID_ARG"),
    ("packed", dict(start=None), "INVALID_ARG"), ("packed", dict(out=None), "INVALID_ARG"), ("packed", dict(q=A + 8), "UNSUPPORTED"),
    ("packed", dict(out=A + 20480), "INVALID_ARG"), ("packed", dict(k_stride=(0, 64)), "UNSUPPORTED"), ("packed", dict(q_stride=(260, 64)), "UNSUPPORTED"),
    ("packed", dict(out_stride=(128, 64)), "INVALID_ARG"), ("packed", dict(out_stride=(256, 32)), "INVALID_ARG"),
    ("packed", dict(v_stride=(1 << 39, 64)), "UNSUPPORTED"), ("packed", dict(k_stride=(-128, 64)), "UNSUPPORTED"),
    ("append", dict(k=None), "INVALID_ARG"), ("append", dict(v=None), "INVALID_ARG"), ("append", dict(out=None), "INVALID_ARG"),
    ("append", dict(rope_len=0), "INVALID_ARG"), ("append", dict(rope=A + 8), "UNSUPPORTED"), ("append", dict(k=A + 2), "UNSUPPORTED"),
    ("append", dict(out=A + 24576), "INVALID_ARG"), ("append", dict(out=A + 20480, out_stride=(512, 64)), "INVALID_ARG"),
    ("read", dict(k=None), "INVALID_ARG"), ("read", dict(v=A + 24576), "INVALID_ARG"), ("read", dict(k_stride=(64, 64)), "INVALID_ARG"),
    ("read", dict(v=A + 4), "UNSUPPORTED"),
    ("attention", dict(q=None), "INVALID_ARG"), ("attention", dict(out=None), "INVALID_ARG"), ("attention", dict(out=A + 20480), "INVALID_ARG"),
    ("attention", dict(ws=None), "INVALID_ARG"), ("attention", dict(ws_bytes=1000), "INVALID_ARG"), ("attention", dict(ws=A + 8), "UNSUPPORTED"),
    ("attention", dict(q=A + 8), "UNSUPPORTED"), ("attention", dict(out_stride=(0, 64)), "INVALID_ARG")])
def test_operands(river, name, kw, status):
    assert _call(river, name, **kw) == getattr(river, "RL_ERR_" + status), river.rl_last_error()


def test_attention_beyond_any_grid(river):
    kw = dict(rows=1 << 20, n_pages=1, page=256, table_width=1 << 22, table_stride=1 << 22)
    assert _call(river, "attention", **kw) == river.RL_ERR_UNSUPPORTED and b"2^38" in river._lib.rl_last_error()


def _sample(river, **kw):
    a = dict(logits=A, dtype=0, rows=2, vocab=100, stride=100, u=A, set=True, token=A)
    a.update({k: v for k, v in kw.items() if k in a})
    s = river.rl_sampling(kw.get("temperature", 1.0), kw.get("top_k", 0), kw.get("top_p", 1.0), kw.get("min_p", 0.0))
    return river._lib.rl_sample(P(a["logits"]), a["dtype"], a["rows"], a["vocab"], a["stride"], P(a["u"]), ctypes.byref(s) if a["set"] else None,
                                P(a["token"]), None, None)


@pytest.mark.parametrize("key", ["d_temperature", "d_top_k", "d_top_p", "d_min_p", "u", "logits"])
@pytest.mark.parametrize("out", ["token", "logprob"])
def test_sample_outputs_in_inputs_places(river, key, out):
    at = dict(logits=A, u=A + 4096, token=A + 8192, logprob=A + 12288)
    s = river.rl_sampling(1.0, 0, 1.0, 0.0)
    if key in at:
        at[out] = at[key]
    else:
        setattr(s, key, at[out])
    assert river._lib.rl_sample(P(at["logits"]), 0, 2, 100, 100, P(at["u"]), ctypes.byref(s), P(at["token"]), P(at["logprob"]),
                                None) == river.RL_ERR_INVALID_ARG and b"overlaps" in river._lib.rl_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), "INVALID_ARG"), (dict(u=None), "INVALID_ARG"), (dict(set=False), "INVALID_ARG"), (dict(token=None), "INVALID_ARG"),
    (dict(dtype=3), "INVALID_ARG"), (dict(rows=0), "INVALID_ARG"), (dict(vocab=0), "INVALID_ARG"), (dict(stride=99), "INVALID_ARG"),
    (dict(logits=A + 2), "INVALID_ARG"), (dict(vocab=(1 << 19) + 1, stride=1 << 20), "UNSUPPORTED"), (dict(temperature=-0.5), "INVALID_ARG"),
    (dict(temperature=float("nan")), "INVALID_ARG"), (dict(temperature=float("inf")), "INVALID_ARG"), (dict(top_k=-1), "INVALID_ARG"),
    (dict(top_p=-0.1), "INVALID_ARG"), (dict(top_p=float("nan")), "INVALID_ARG"), (dict(min_p=-1.0), "INVALID_ARG"), (dict(min_p=float("inf")), "INVALID_ARG")])
def test_sample(river, kw, status):
    assert _sample(river, **kw) == getattr(river, "RL_ERR_" + status)
    assert "rl_sample" in river.rl_last_error()


def _tensors(river):
    bf, i32 = torch.bfloat16, torch.int32
    return dict(cache=river.KV4Cache.alloc(4, 2, 64, page=16, device="cpu"), table=torch.zeros((2, 3), dtype=i32), n=torch.ones(2, dtype=i32),
                start=torch.tensor([0, 3, 5], dtype=i32), q=torch.zeros((5, 4, 64), dtype=bf), k=torch.zeros((5, 2, 64), dtype=bf))


def test_python_forms_refuse_host_tensors(river):
    t = _tensors(river)
    for call in (lambda: river.packed_attention(t["q"], t["k"], t["k"], t["start"]),
                 lambda: river.kv4_append(t["cache"], t["table"], t["n"], t["k"], t["k"], q=t["q"], start=t["start"]),
                 lambda: river.kv4_read(t["cache"], t["table"], t["n"], start=t["start"], rows=5),
                 lambda: river.kv4_attention(t["q"], t["cache"], t["table"], t["n"], start=t["start"]),
                 lambda: river.sample(torch.zeros((2, 9)), torch.zeros(2))):
        with pytest.raises(river.RiverError) as e:
            call()
        assert e.value.status == river.RL_ERR_INVALID_ARG and "CUDA" in str(e.value)


def test_python_forms_refuse_what_does_not_fit(river, monkeypatch):
    """Shapes, types and layouts, behind the check of devices (which these host tensors pass by)."""
    monkeypatch.setattr(river, "_operands", lambda name, tensors: -1)
    monkeypatch.setattr(river, "_run", lambda *a: pytest.fail("reached the library"))
    t = _tensors(river)
    q, k, c, tab, n, st = (t[x] for x in ("q", "k", "cache", "table", "n", "start"))
    half = river.KV4Cache(*(x.half() if x.dtype == torch.bfloat16 else x for x in c))
    bad = [lambda: river.packed_attention(q, k, k[:, :1], st), lambda: river.packed_attention(q, k, k.half(), st), lambda: river.packed_attention(q.float(), k, k, st),
           lambda: river.packed_attention(q, k, k, st.long()), lambda: river.packed_attention(q[0], k, k, st), lambda: river.packed_attention(q, k, k, st, scale=-1.0),
           lambda: river.packed_attention(q, k, k, st, scale=1e-60), lambda: river.packed_attention(q[:0], k[:0], k[:0], st),
           lambda: river.packed_attention(q, k.transpose(1, 2), k, st),
           lambda: river.kv4_append(half, tab, n, k, k, start=st), lambda: river.kv4_append(c, tab.long(), n, k, k, start=st), lambda: river.kv4_append(c, tab[:1], n, k, k, start=st),
           lambda: river.kv4_append(c, tab, n, k, k), lambda: river.kv4_append(c, tab, n, k, k[:4], start=st), lambda: river.kv4_append(c, tab, n, k, k, q=q[:4], start=st),
           lambda: river.kv4_append(c, tab, n, k, k, start=st, rope=torch.zeros((9, 32))), lambda: river.kv4_append(c, tab, n, k, k, start=st, rope=torch.zeros((9, 64, 2))),
           lambda: river.kv4_append(c, tab, n, k, k, start=st, rope=torch.zeros((9, 32, 2), dtype=torch.float64)), lambda: river.kv4_append(c, tab, n.long(), k, k, start=st),
           lambda: river.kv4_append(c, tab, n, k, k, q=q, start=st, out={"q": q[:4]}), lambda: river.kv4_append(c, tab, n, k, k, start=st, err=n),
           lambda: river.kv4_read(c, tab, n, start=st), lambda: river.kv4_read(c, tab, n, start=st[:2], rows=5), lambda: river.kv4_read(c, tab, n, start=st, rows=0),
           lambda: river.kv4_read(c, tab, n, start=st, rows=5, out={"k": k[:4]}), lambda: river.kv4_read(c, tab, n, start=st, rows=5, out={"k": k.half()}),
           lambda: river.kv4_read((c[0][:, :, ::2], c[1][:, :, ::2], c[2][:, :, ::2], c[3][:, :, ::2]), tab, n, start=st, rows=5),
           lambda: river.kv4_attention(q.half(), c, tab, n, start=st), lambda: river.kv4_attention(q, c, tab, n), lambda: river.kv4_attention(q[..., :32], c, tab, n, start=st),
           lambda: river.kv4_attention(q, (c[0], c[1], c[2][:3], c[3]), tab, n, start=st), lambda: river.kv4_attention(q, c, tab.t(), n, start=st),
           lambda: river.kv4_attention(q, c, tab, n, start=st, out={"lse": torch.zeros(3)}),
           lambda: river.sample(torch.zeros((2, 9)), torch.zeros(3)), lambda: river.sample(torch.zeros((9, 2)).t(), torch.zeros(2)),
           lambda: river.sample(torch.zeros((2, 9), dtype=torch.float64), torch.zeros(2)), lambda: river.sample(torch.zeros((2, 9)), torch.zeros(2), top_k=torch.zeros(2))]
    for i, f in enumerate(bad):
        with pytest.raises(river.RiverError) as e:
            f()
        assert e.value.status in (river.RL_ERR_INVALID_ARG, river.RL_ERR_UNSUPPORTED), i


def test_sizes_beyond_32_bits(river, monkeypatch):
    """A size is never taken for its low 32 bits."""
    monkeypatch.setattr(river, "_operands", lambda name, tensors: -1)
    t, n = _tensors(river), 2**32 + 2
    q = t["q"][:1].expand(n, 4, 64)
    k = t["k"][:1].expand(n, 2, 64)
    for call in (lambda: river.packed_attention(q, k, k, t["start"], out={"out": q}), lambda: river.kv4_attention(q, t["cache"], t["table"], t["n"], start=t["start"], out={"out": q}),
                 lambda: river.kv4_append(t["cache"], t["table"], t["n"], k, k, start=t["start"]),
                 lambda: river.kv4_read(t["cache"], t["table"], t["n"], start=t["start"], rows=n),
                 lambda: river.sample(torch.empty((n, 1), device="meta"), t["n"])):
        with pytest.raises(river.RiverError):
            call()


def test_rope_table_is_the_model_rotation(river):
    import numpy as np
    from oracle.model import rope
    x = np.random.default_rng(1).standard_normal((1, 7, 2, 64)).astype(np.float32)
    tab = river.rope_table(7, 64, 10000.0, device="cpu").numpy()
    a, b = x[..., :32], x[..., 32:]
    c, s = tab[None, :, None, :, 0], tab[None, :, None, :, 1]
    want = rope(x, np.arange(7), 10000.0)
    assert np.abs(np.concatenate([a * c - b * s, b * c + a * s], -1) - want).max() < 1e-5


@pytest.mark.parametrize("bad", [0.5, 2.25, float("nan"), float("inf"), "3"])
def test_fractions_for_whole_numbers(river, monkeypatch, bad):
    """A count is never cut to the whole number below it (top_k 0.5 would keep every id); whole floats are counts."""
    monkeypatch.setattr(river, "_operands", lambda name, tensors: -1)
    monkeypatch.setattr(river, "_run", lambda *a: pytest.fail("reached the library"))
    t = _tensors(river)
    q, k, c, tab, n, st = (t[x] for x in ("q", "k", "cache", "table", "n", "start"))
    for call in (lambda: river.sample(torch.zeros((2, 9)), torch.zeros(2), top_k=bad), lambda: river.kv4_read(c, tab, n, start=st, rows=bad),
                 lambda: river.packed_attention(q, k, k, st, max_rows=bad), lambda: river.kv4_attention(q, c, tab, n, start=st, max_rows=bad)):
        with pytest.raises(river.RiverError) as e:
            call()
        assert e.value.status == river.RL_ERR_INVALID_ARG and "whole" in str(e.value)
    seen = []
    monkeypatch.setattr(river, "_run", lambda dev, stream, fn, *a: seen.append(a))
    river.sample(torch.zeros((2, 9)), torch.zeros(2), top_k=7.0)
    assert seen[0][6].top_k == 7


@pytest.mark.parametrize("out", ["token", "logprob"])
@pytest.mark.parametrize("key,by", [("d_temperature", 4), ("d_top_k", -4), ("d_top_p", 8), ("d_min_p", -8), ("u", 8), ("u", -8), ("logits", -8), ("logits", 396),
                                    ("logits", 480), ("logits", 872), ("other", 4), ("other", 0), ("other", -8)])
def test_sample_outputs_that_overlap_in_part(river, key, by, out):
    """Three rows: an output that starts `by` bytes from an input, or from the other output (rows of logits are 400 bytes, 480 apart)."""
    at = dict(logits=A, u=A + 4096, token=A + 8192, logprob=A + 12288)
    s = river.rl_sampling(1.0, 0, 1.0, 0.0)
    if key == "other":
        at[out] = at["logprob" if out == "token" else "token"] + by
    elif key in at:
        at[out] = at[key] + by
    else:
        setattr(s, key, at[out] - by)
    assert river._lib.rl_sample(P(at["logits"]), 0, 3, 100, 120, P(at["u"]), ctypes.byref(s), P(at["token"]), P(at["logprob"]),
                                None) == river.RL_ERR_INVALID_ARG and b"overlap" in river._lib.rl_last_error()
