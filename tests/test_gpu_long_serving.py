"""The model's own paths over the stand-alone operators, against the oracle: a
cache with a sliding window, one prompt shared by many continuations, a scored
prefill, and a run of them together.  Tolerances of the other parity tests
(tests/harness.py); log-probabilities move by at most twice the logits'."""
import numpy as np
import pytest

import synth
from oracle.model import KVState, Policy as OPolicy
from tests.harness import LOGIT_TOL, build_pair, check_step

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TINY = synth.TINY
# one layer of the larger head layouts with a small vocabulary
HD64 = synth.scaled(synth.LLAMA_1B, n_layers=1, d_model=512, ffn_dim=512, vocab=2048, name="hd64")
HD128 = synth.scaled(synth.LLAMA_8B, n_layers=1, d_model=512, ffn_dim=512, vocab=2048, name="hd128")


@pytest.fixture(scope="module")
def river():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import __graft_entry__
    __graft_entry__.build()
    import early_exit_decoding_gb300 as r
    return r


@pytest.fixture(scope="module")
def stream(river):
    return torch.cuda.Stream()


_PAIRS = {}


def pair(shape, stream):
    if shape.name not in _PAIRS:
        with torch.cuda.stream(stream):
            _PAIRS[shape.name] = build_pair(shape, seed=0, gains="random", stream=stream)[:2]
        stream.synchronize()
    return _PAIRS[shape.name]


def steps(river, m, om, kv, st, stream, n, B, tok, exits, label):
    """n decode steps on both sides from token ids tok [B], forced exits in turn."""
    for i in range(n):
        e = exits[i % len(exits)]
        sched = torch.tensor([e], dtype=torch.int32, device="cuda")
        with torch.cuda.stream(stream):
            out = river.decode_step(m, kv, torch.from_numpy(tok.copy()).cuda(), river.Policy.forced(sched), stream=stream)
            kv.sync(stream)
        ref = om.decode_step(tok, st, OPolicy.forced(e))
        check_step(out, ref, None, B, f"{label}, step {i}")
        assert int(out["exit_layer"].item()) == e
        tok = ref.logits.argmax(-1).astype(np.int32)
    return tok


@pytest.mark.parametrize("shape,B,T,window,sinks", [
    (TINY, 1, 40, 24, 3), (TINY, 2, 20, 24, 0), (TINY, 16, 33, 16, 1), (TINY, 3, 40, 1, 0), (HD64, 2, 150, 100, 4),
    (HD128, 1, 300, 130, 20), (HD128, 17, 20, 24, 2)])
def test_sliding_window(river, stream, shape, B, T, window, sinks):
    m, om = pair(shape, stream)
    kv = m.kv_cache_alloc(B, T + 16)
    kv.set_window(window, sinks)
    st = KVState(shape, B, T + 16)
    st.window, st.sinks = window, sinks
    toks = synth.gen_tokens(shape.vocab, (B, T), seed=1)
    with torch.cuda.stream(stream):
        out = river.prefill(m, kv, torch.from_numpy(toks).cuda(), river.Policy.tau_(1.01), stream=stream)
        kv.sync(stream)
    ref = om.prefill(toks, st, OPolicy.tau_(1.01))
    check_step(out, ref, None, B, "windowed prefill")
    L = shape.n_layers
    steps(river, m, om, kv, st, stream, 10, B, ref.logits.argmax(-1).astype(np.int32), [L, max(0, L - 2), 0], "windowed")
    # which path: any while every key is in sight, the generic one past the window
    assert kv.decode_path(B) == river.RL_PATH_GENERIC
    kv.set_decode_path(river.RL_PATH_STEP)
    assert kv.decode_path(B) == -1
    kv.set_decode_path(river.RL_PATH_AUTO)
    kv.set_window(0)
    assert kv.decode_path(B) == (river.RL_PATH_STEP if B <= 8 else river.RL_PATH_GENERIC)


@pytest.mark.parametrize("shape,B,T", [(TINY, 1, 37), (TINY, 5, 1), (TINY, 20, 150), (HD64, 6, 301), (HD128, 40, 129)])
def test_shared_prefix(river, stream, shape, B, T):
    m, om = pair(shape, stream)
    cap = T + 12
    kv = m.kv_cache_alloc(B, cap)
    one = KVState(shape, 1, cap)
    toks = synth.gen_tokens(shape.vocab, (1, T), seed=1)
    with torch.cuda.stream(stream):
        river.prefill(m, kv, torch.from_numpy(toks).cuda(), river.Policy.tau_(1.01), stream=stream)
    om.prefill(toks, one, OPolicy.tau_(1.01))
    kv.share_prefix()
    st = KVState(shape, B, cap)
    for l in range(shape.n_layers):
        st.K[l][:] = one.K[l]
        st.V[l][:] = one.V[l]
    st.pos = T
    tok = synth.gen_tokens(shape.vocab, (B,), seed=7)
    L = shape.n_layers
    steps(river, m, om, kv, st, stream, 8, B, tok, [L, 0, max(0, L - 1)], "behind a shared prefix")
    with pytest.raises(river.RiverError) as e:
        kv.set_position(T - 1, 0, stream)
    assert e.value.status == river.RL_ERR_STATE
    # the next prefill is an ordinary one again
    B2 = min(B, 2)
    t2 = synth.gen_tokens(shape.vocab, (B2, 5), seed=9)
    st2 = KVState(shape, B2, cap)
    with torch.cuda.stream(stream):
        out = river.prefill(m, kv, torch.from_numpy(t2).cuda(), river.Policy.tau_(1.01), stream=stream)
        kv.sync(stream)
    ref = om.prefill(t2, st2, OPolicy.tau_(1.01))
    check_step(out, ref, None, B2, "prefill after sharing")
    steps(river, m, om, kv, st2, stream, 2, B2, ref.logits.argmax(-1).astype(np.int32), [L], "after sharing")


def check_scores(shape, om, toks, got, exit_layer, top_k):
    """A scored prefill's outputs against the oracle's logits at every position."""
    B, T = toks.shape
    logits = om.recompute(toks, np.full(T, exit_layer)).astype(np.float64)
    lp = logits - np.log(np.sum(np.exp(logits - logits.max(-1, keepdims=True)), -1, keepdims=True)) - logits.max(-1, keepdims=True)
    g = got["logprob"].cpu().numpy().astype(np.float64)
    assert (g[:, 0] == 0).all()
    if T > 1:
        want = np.take_along_axis(lp[:, :-1], toks[:, 1:, None].astype(np.int64), -1)[..., 0]
        assert np.abs(g[:, 1:] - want).max() <= 2 * LOGIT_TOL
    # dH = -sum p (ln p + H) dx: at most the logits' error times E |ln p + H|, e^(2 tol) for the weights' own change
    p = np.exp(lp)
    H = -(p * lp).sum(-1)
    spread = (p * np.abs(lp + H[..., None])).sum(-1)
    dH = np.abs(got["entropy"].cpu().numpy() - H)
    assert (dH <= LOGIT_TOL * np.exp(2 * LOGIT_TOL) * (spread + 2 * LOGIT_TOL) + 1e-4).all()
    if top_k:
        ids = got["top_ids"].cpu().numpy()
        assert np.abs(np.take_along_axis(lp, ids.astype(np.int64), -1) - got["top_logprobs"].cpu().numpy()).max() <= 2 * LOGIT_TOL
        srt = np.sort(lp, -1)[..., ::-1]
        # the k-th reported one is as likely as the true k-th, up to the logits' error on both
        assert (np.take_along_axis(lp, ids.astype(np.int64), -1) >= srt[..., :top_k] - 4 * LOGIT_TOL).all()


@pytest.mark.parametrize("shape,B,T,top_k", [(TINY, 3, 17, 4), (TINY, 1, 1, 0), (TINY, 2, 300, 1), (HD64, 1, 33, 32)])
def test_scored_prefill(river, stream, shape, B, T, top_k):
    m, om = pair(shape, stream)
    kv = m.kv_cache_alloc(B, T + 2)
    toks = synth.gen_tokens(shape.vocab, (B, T), seed=3)
    t = torch.from_numpy(toks).cuda()
    sched = torch.tensor([shape.n_layers - 1], dtype=torch.int32, device="cuda")
    with torch.cuda.stream(stream):
        plain = river.prefill(m, kv, t, river.Policy.forced(sched), stream=stream)
        got = river.prefill_score(m, kv, t, river.Policy.forced(sched), top_k=top_k, stream=stream)
        kv.sync(stream)
    for n in ("logits", "next_token", "exit_layer", "min_cos"):
        assert torch.equal(plain[n], got[n]), n
    check_scores(shape, om, toks, got, shape.n_layers - 1, top_k)
    assert kv.position() == (T, 0)


def test_refusals(river, stream):
    m, _ = pair(TINY, stream)
    kv = m.kv_cache_alloc(2, 32)
    t = torch.from_numpy(synth.gen_tokens(TINY.vocab, (1, 8), seed=1)).cuda()
    for bad in (-1, 1):
        with pytest.raises(river.RiverError):
            kv.share_prefix(bad)  # nothing prefilled yet
    with pytest.raises(river.RiverError):
        kv.set_window(-1)
    with torch.cuda.stream(stream):
        river.prefill(m, kv, t, river.Policy.tau_(1.01), stream=stream)
    kv.share_prefix(8)
    with pytest.raises(river.RiverError) as e:
        kv.set_window(4)
    assert e.value.status == river.RL_ERR_STATE
    kv.share_prefix(0)
    kv.set_window(4, 1)
    with pytest.raises(river.RiverError) as e:
        kv.share_prefix(8)
    assert e.value.status == river.RL_ERR_STATE
    kv.set_window(0)
    o = torch.zeros((1, 8), device="cuda")
    with pytest.raises(river.RiverError) as e:
        river.prefill_score(m, kv, t, river.Policy.tau_(1.01), top_k=33, stream=stream)
    assert e.value.status == river.RL_ERR_INVALID_ARG
    river.rl_debug_fail_allocations(1)  # the prompt's workspace is there, the scores' is not
    try:
        with pytest.raises(river.RiverError) as e:
            river.prefill_score(m, kv, t, river.Policy.tau_(1.01), out={"logprob": o}, stream=stream)
        assert e.value.status == river.RL_ERR_OOM
    finally:
        river.rl_debug_fail_allocations(-1)
    with torch.cuda.stream(stream):
        river.prefill_score(m, kv, t, river.Policy.tau_(1.01), out={"logprob": o}, stream=stream)
        kv.sync(stream)
    assert torch.isfinite(o).all()


def test_many_continuations_of_one_prompt_scored(river, stream):
    """The operators together: a scored prompt, several sampled continuations
    behind its shared prefix, each step's log-probabilities from the step's
    logits, and the best one scored again as a whole."""
    m, om = pair(TINY, stream)
    B, T, n = 6, 29, 5
    kv = m.kv_cache_alloc(B, T + n + 1)
    prompt = synth.gen_tokens(TINY.vocab, (1, T), seed=11)
    sched = torch.tensor([TINY.n_layers], dtype=torch.int32, device="cuda")
    pol = river.Policy.forced(sched)
    with torch.cuda.stream(stream):
        first = river.prefill_score(m, kv, torch.from_numpy(prompt).cuda(), pol, top_k=B, stream=stream)
        kv.share_prefix()
        tok = first["top_ids"][0, -1].clone()          # the B likeliest first tokens
        total = first["top_logprobs"][0, -1].clone()
        seqs = [tok]
        for _ in range(n):
            out = river.decode_step(m, kv, tok, pol, stream=stream)
            s = river.token_logprobs(out["logits"], out["next_token"], top_k=1, stream=stream)
            tok = out["next_token"].clone()
            assert torch.equal(s["top_ids"][:, 0], tok)
            total = total + s["logprob"]
            seqs.append(tok)
        kv.sync(stream)
    cont = torch.stack(seqs, 1).cpu().numpy()
    best = int(total.argmax())
    whole = np.concatenate([prompt, cont[best:best + 1]], 1)
    kv2 = m.kv_cache_alloc(1, whole.shape[1] + 1)
    with torch.cuda.stream(stream):
        again = river.prefill_score(m, kv2, torch.from_numpy(whole).cuda(), pol, stream=stream)
        kv2.sync(stream)
    check_scores(TINY, om, whole, again, TINY.n_layers, 0)
    # each of the n + 1 terms may differ by twice the logits' tolerance
    assert abs(float(again["logprob"][0, T:].sum()) - float(total[best])) <= 2 * LOGIT_TOL * (n + 1)
