"""The oracle's sliding window: against a float64 softmax over the keys a row
sees, and no change while everything is in sight."""
import numpy as np

import synth
from oracle.model import KVState, OracleModel, Policy, attention


def test_window_rows_are_softmaxes_over_what_they_see():
    rng = np.random.default_rng(0)
    q = rng.standard_normal((9, 4, 8)).astype(np.float32)
    k = rng.standard_normal((2, 9, 8)).astype(np.float32)
    v = rng.standard_normal((2, 9, 8)).astype(np.float32)
    got = attention(q, k, v, np.arange(9), window=3, sinks=2)
    for p in range(9):
        see = [j for j in range(p + 1) if p - j < 3 or j < 2]
        for h in range(4):
            s = np.array([q[p, h].astype(np.float64) @ k[h // 2, j] / np.sqrt(8) for j in see])
            w = np.exp(s - s.max())
            ref = (w / w.sum()) @ v[h // 2, see].astype(np.float64)
            assert np.abs(got[p, h] - ref).max() < 1e-6


def test_wide_window_changes_nothing_and_a_narrow_one_does():
    S = synth.TINY
    om = OracleModel(S, synth.weights_to_numpy(synth.gen_weights(S, seed=0, device="cpu")))
    toks = synth.gen_tokens(S.vocab, (1, 12), seed=1)
    outs = []
    for window in (0, 12, 4):
        st = KVState(S, 1, 16)
        st.window, st.sinks = window, 1
        outs.append(om.prefill(toks, st, Policy.tau_(1.01)).logits)
    assert np.array_equal(outs[0], outs[1]) and np.abs(outs[0] - outs[2]).max() > 1e-3
