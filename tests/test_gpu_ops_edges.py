"""The operators and the model's paths over them where calls meet: other
streams at work, buffers a caller brings, failures half way."""
import numpy as np
import pytest

import synth
from tests.harness import build_pair
from tests.test_ops_edges import derivatives_refused, forms

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TINY = synth.TINY


@pytest.fixture(scope="module")
def river():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import __graft_entry__
    __graft_entry__.build()
    import early_exit_decoding_gb300 as r
    yield r
    r.rl_debug_fail_allocations(-1)


@pytest.fixture(scope="module")
def stream(river):
    return torch.cuda.Stream()


@pytest.fixture(scope="module")
def tiny(river, stream):
    with torch.cuda.stream(stream):
        m = build_pair(TINY, seed=0, gains="random", stream=stream)[0]
    stream.synchronize()
    return m


def busy_default_stream():
    """Queues about half a second of work on the default stream; an event behind it."""
    done = torch.cuda.Event()
    with torch.cuda.stream(torch.cuda.default_stream()):
        torch.cuda._sleep(1_000_000_000)
        done.record()
    return done


def test_share_prefix_beside_a_busy_default_stream(river, stream, tiny):
    """The workspace a shared prefix takes is never touched from a stream that
    the steps do not wait for: steps on another stream give the same values
    while the default stream works, and when its work ends."""
    B, T = 5, 37
    toks = torch.from_numpy(synth.gen_tokens(TINY.vocab, (1, T), seed=1)).cuda()
    tok = torch.from_numpy(synth.gen_tokens(TINY.vocab, (B,), seed=2)).cuda()
    sched = torch.tensor([TINY.n_layers], dtype=torch.int32, device="cuda")
    pol = river.Policy.forced(sched)

    def run(busy):
        kv = tiny.kv_cache_alloc(B, T + 4)
        with torch.cuda.stream(stream):
            river.prefill(tiny, kv, toks, pol, stream=stream)
            kv.sync(stream)
            done = busy_default_stream() if busy else None
            kv.share_prefix()
            outs, more = [], True
            while more and len(outs) < 20000:
                more = done is not None and not done.query()
                kv.set_position(T, 0, stream)
                outs.append(river.decode_step(tiny, kv, tok, pol, stream=stream)["logits"])
                if len(outs) % 64 == 0:
                    stream.synchronize()
            kv.sync(stream)
        torch.cuda.synchronize()
        return outs

    want = run(False)[0]
    for got in run(True):
        assert torch.equal(got, want)


def rnd(*shape, seed, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, device="cuda", generator=g).to(dtype)


def given_up(river, call):
    """``call(err)`` with waits that give up at once, between two ordinary
    calls that must agree: the outputs of the second one's kind."""
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = call(err)
    torch.cuda.synchronize()
    assert int(err) == 0
    river.rl_debug_limit_waits(0)
    try:
        got = call(err)
        torch.cuda.synchronize()
    finally:
        river.rl_debug_limit_waits(-1)
    assert int(err) == river.RL_DEVERR_TIMEOUT
    err.zero_()
    again = call(err)
    torch.cuda.synchronize()
    assert int(err) == 0
    for n in want:
        assert torch.equal(want[n], again[n]), n
    return got


# (sequences, query rows, heads, KV heads, head_dim, keys, window): one key tile (every copy
# is issued before any wait) and many; one CTA a row tile and a cluster
WAITS = [(2, 40, 8, 2, 64, 100, 50), (2, 40, 8, 2, 128, 100, 100), (40, 300, 8, 4, 128, 1500, 900), (1, 40, 8, 1, 64, 4000, 4000)]


@pytest.mark.parametrize("B,T,Hq,Hkv,D,n,window", WAITS)
def test_rows_whose_waits_give_up(river, B, T, Hq, Hkv, D, n, window):
    q, k, v = rnd(B, T, Hq, D, seed=1), rnd(B, Hkv, n, D, seed=2), rnd(B, Hkv, n, D, seed=3)
    kv_len = torch.full((B,), n, dtype=torch.int32, device="cuda")
    got = given_up(river, lambda err: river.window_attention(q, k, v, kv_len, window, err=err))
    assert torch.isnan(got["out"]).all() and torch.isnan(got["lse"]).all()


@pytest.mark.parametrize("B,prefix", [(3, 100), (40, 3000), (160, 700)])
def test_prefix_whose_waits_give_up(river, B, prefix):
    q, pk, pv = rnd(B, 8, 128, seed=1), rnd(4, prefix, 128, seed=2), rnd(4, prefix, 128, seed=3)
    k, v = rnd(B, 4, 24, 128, seed=4), rnd(B, 4, 24, 128, seed=5)
    kv_len = torch.arange(B, dtype=torch.int32, device="cuda") % 25
    got = given_up(river, lambda err: river.shared_prefix_attention(q, pk, pv, k, v, kv_len, err=err))
    assert torch.isnan(got["out"]).all() and torch.isnan(got["lse"]).all()


def test_scores_that_fail_leave_the_prompt(river, stream, tiny):
    """A failure behind the prompt's own pass: position, slots and prefix are
    those of a plain prefill, and decoding goes on from there."""
    kv = tiny.kv_cache_alloc(3, 32)
    pol = river.Policy.forced(torch.tensor([TINY.n_layers], dtype=torch.int32, device="cuda"))
    first = torch.from_numpy(synth.gen_tokens(TINY.vocab, (1, 9), seed=1)).cuda()
    toks = torch.from_numpy(synth.gen_tokens(TINY.vocab, (3, 5), seed=2)).cuda()
    tok = torch.from_numpy(synth.gen_tokens(TINY.vocab, (3,), seed=3)).cuda()
    with torch.cuda.stream(stream):
        river.prefill(tiny, kv, toks, pol, stream=stream)
        want = [river.decode_step(tiny, kv, tok, pol, stream=stream)["logits"] for _ in range(3)]
        river.prefill(tiny, kv, first, pol, stream=stream)
        kv.share_prefix()
        river.rl_debug_fail_allocations(2)  # both workspaces are there, the scores are not
        try:
            with pytest.raises(river.RiverError) as e:
                river.prefill_score(tiny, kv, toks, pol, stream=stream)
        finally:
            river.rl_debug_fail_allocations(-1)
        assert e.value.status == river.RL_ERR_OOM and "injected" in str(e.value)
        assert kv.position() == (5, 0)
        got = [river.decode_step(tiny, kv, tok, pol, stream=stream)["logits"] for _ in range(3)]
        kv.sync(stream)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        kv.set_position(0, 0, stream)  # no prefix any more


def test_operands_with_derivatives_are_refused(river):
    for call, ops in forms(river, "cuda"):
        derivatives_refused(river, call, ops, range(len(ops)), lambda given: given())


def test_windows_beyond_32_bits(river):
    q, k = rnd(1, 1, 4, 64, seed=1), rnd(1, 2, 40, 64, seed=2)
    n = torch.full((1,), 40, dtype=torch.int32, device="cuda")
    want = river.window_attention(q, k, k, n, 40)
    for window in (2**31, 2**32 + 5):
        got = river.window_attention(q, k, k, n, window, 0)
        assert torch.equal(got["out"], want["out"])
        got = river.window_attention(q, k, k, n, 3, window)
        assert torch.equal(got["out"], want["out"])
    for window, sinks in ((0, 0), (-2**31 - 1, 0), (-2**32 + 5, 0), (5, -2**32 + 1), (5, -1)):
        with pytest.raises(river.RiverError) as e:
            river.window_attention(q, k, k, n, window, sinks)
        assert e.value.status == river.RL_ERR_INVALID_ARG


def test_outputs_are_taken_on_the_stream_that_writes_them(river, stream, tiny):
    """Memory that was freed under work still queued on the current stream is
    not written by another one."""
    B, T, V, L = 3, 6, TINY.vocab, TINY.n_layers
    pol = river.Policy.forced(torch.tensor([L], dtype=torch.int32, device="cuda"))
    toks = torch.from_numpy(synth.gen_tokens(V, (B, T), seed=2)).cuda()
    tok = torch.from_numpy(synth.gen_tokens(V, (B,), seed=3)).cuda()
    kv = tiny.kv_cache_alloc(B, 32)
    rows = torch.randn((B, V), device="cuda")
    torch.cuda.synchronize()
    calls = [lambda: river.prefill(tiny, kv, toks, pol, stream=stream),
             lambda: river.decode_step(tiny, kv, tok, pol, stream=stream),
             lambda: river.prefill_score(tiny, kv, toks, pol, top_k=3, stream=stream),
             lambda: river.token_logprobs(rows, tok, top_k=3, stream=stream)]
    want = [{n: t.clone() for n, t in call().items() if stream.synchronize() is None} for call in calls]
    torch.cuda.synchronize()
    sizes = {tuple(t.shape): t.dtype for w in want for t in w.values()}
    torch.cuda._sleep(1_000_000_000)  # the current stream stays behind; what it frees is written late
    late = [torch.empty(s, dtype=d, device="cuda").fill_(77) for s, d in sizes.items() for _ in range(4)]
    del late
    got = [call() for call in calls]
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for n in w:
            assert torch.equal(w[n], g[n]), n


def test_prefill_score_refuses_buffers_that_do_not_fit(river, stream, tiny):
    """A buffer of another shape, type or place is refused, not written past its end."""
    B, T, k = 2, 6, 3
    kv = tiny.kv_cache_alloc(B, 16)
    pol = river.Policy.forced(torch.tensor([TINY.n_layers], dtype=torch.int32, device="cuda"))
    toks = torch.from_numpy(synth.gen_tokens(TINY.vocab, (B, T), seed=2)).cuda()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        good = river.prefill_score(tiny, kv, toks, pol, top_k=k, stream=stream)
        again = river.prefill_score(tiny, kv, toks, pol, top_k=k, out=good, stream=stream)
        kv.sync(stream)
    for n, t in good.items():
        assert again[n] is t
        wrong = [t[:1] if t.shape[0] > 1 else t[:0], t.cpu(), t.to(torch.float16), torch.stack([t, t], -1)[..., 0]]
        for bad in (x for i, x in enumerate(wrong) if i < 3 or not x.is_contiguous()):
            with pytest.raises(river.RiverError) as e:
                river.prefill_score(tiny, kv, toks, pol, top_k=k, out={n: bad}, stream=stream)
            assert e.value.status == river.RL_ERR_INVALID_ARG, n
    with pytest.raises(river.RiverError) as e:
        river.prefill_score(tiny, kv, toks, pol, top_k=k + 1, out=good, stream=stream)
    assert e.value.status == river.RL_ERR_INVALID_ARG


def test_out_buffers_with_a_gradient_are_refused(river):
    """A buffer that requires one would be written behind autograd's back."""
    q, k = rnd(1, 1, 4, 64, seed=1), rnd(1, 2, 40, 64, seed=2)
    n = torch.full((1,), 40, dtype=torch.int32, device="cuda")
    x, pre = torch.randn((1, 9), device="cuda"), k[0]
    for call in (lambda **kw: river.token_logprobs(x, **kw), lambda **kw: river.window_attention(q, k, k, n, 4, **kw),
                 lambda **kw: river.shared_prefix_attention(q[0], pre, pre, k, k, n, **kw)):
        for key, t in call().items():
            bad = t.clone().requires_grad_()
            with pytest.raises(river.RiverError) as e:
                call(out={key: bad})
            assert e.value.status == river.RL_ERR_UNSUPPORTED
            with torch.no_grad():
                assert call(out={key: bad})[key] is bad
