"""Sampling with a row in 1, 2, 4, 8 and 16 parts (few rows of 4,000 to 60,000 ids), with every kind of cut, against float64;
logits of a long tail, of few values, and of one far above the rest."""
import pytest

from tests.test_gpu_attention_ops import rnd, river  # noqa: F401
from tests.test_gpu_serving_ops import BF, F32, FP, SETTINGS, call, check_sample, uniform

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF, FP])
@pytest.mark.parametrize("V", [4000, 8000, 16000, 32000, 60000])
def test_every_split(river, dtype, V):  # noqa: F811
    rows = [rnd(1, V, dtype=F32, seed=V, scale=1.0), rnd(1, V, dtype=F32, seed=V + 1, scale=4.0), rnd(1, V, dtype=F32, seed=V + 2, scale=3.0).round()]
    rows.append(rows[0].clone())
    rows[3][0, V // 3] = 12.0
    x = torch.cat(rows).to(dtype)
    for i, s in enumerate([*SETTINGS, dict(k=97), dict(k=130, p=0.8), dict(T=2.0, k=1000, p=0.6, mp=0.001), dict(T=0.4, p=0.99)]):
        u = uniform(4, 3 * i + V)
        check_sample(call(river, x, u, **s), x, u, **s)
