"""The operators and the model's paths over them where calls meet: other
streams at work, buffers a caller brings, failures half way."""
import numpy as np
import pytest

import synth
from tests.harness import build_pair

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
