"""The sampler's weights on the GPU are those of csrc/sample_weight.h with every
operation rounded by itself, unit for unit.

With u = 1/2 a row of the largest logit, x, the largest again and a ladder of
small logits gives id 1 where the ladder's weights sum to less than x's, and
else id 2: half of all, rounded down, is the first weight plus half of x's and
the ladder's.  A ladder one unit short of x's weight and one equal to it fix the
weight exactly (and the ladder's own)."""
import numpy as np
import pytest

from tests.test_gpu_attention_ops import river  # noqa: F401
from tests.weight_host import WeightHost

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    return WeightHost(str(tmp_path_factory.mktemp("weight")))


@pytest.mark.parametrize("m,T", [(14.32, 0.8), (7.3, 1.0), (-3.25, 1.7), (91.0, 0.3)])
def test_weights_on_the_gpu_are_the_headers(river, host, m, T):  # noqa: F811
    rng = np.random.default_rng(int(T * 100))
    unit = T / np.log2(np.e)  # of y, in logits
    m = np.float32(m)
    bank = (m - unit * np.linspace(0.01, 44.9, 6000)).astype(np.float32)
    value = host.weights(bank, m, T).astype(np.int64)
    order = np.argsort(-value, kind="stable")
    bank, value = bank[order], value[order]
    assert (value == 1).any()
    # anywhere, and where the table's step ends (|r| near 1 / 128)
    y = np.concatenate([rng.uniform(0, 44, 1500), (rng.integers(0, 2800, 1500) + 0.5 + rng.uniform(-0.03, 0.03, 1500)) / 64])
    x = (m - unit * y).astype(np.float32)
    rows, want = [], []
    for xx, w in zip(x, host.weights(x, m, T).astype(np.int64)):
        for goal, token in ((w - 1, 1), (w, 2)):
            row, left = [m, xx, m], int(goal)
            while left > 0:
                i = int(np.searchsorted(-value, -left))  # the largest that fits
                row.append(bank[i])
                left -= int(value[i])
            rows.append(row)
            want.append(token)
    V = max(map(len, rows))
    assert V < 200
    logits = np.full((len(rows), V), -np.inf, np.float32)
    for r, row in enumerate(rows):
        logits[r, :len(row)] = row
    u = torch.full((len(rows),), 0.5, device="cuda")
    got = river.sample(torch.from_numpy(logits).cuda(), u, temperature=float(T))["token"].cpu().numpy()
    wrong = np.nonzero(got != np.array(want))[0]
    assert wrong.size == 0, f"{wrong.size} of {got.size}, the first at y {y[wrong[0] // 2]}: token {got[wrong[0]]}"
