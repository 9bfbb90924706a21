"""Where rl_sample's outputs may lie: beside the logits' rows, in the room between them."""
import pytest

from tests.test_gpu_attention_ops import river  # noqa: F401
from tests.test_gpu_serving_ops import check_sample, logits, uniform

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_outputs_between_the_rows(river):  # noqa: F811
    R, V, step = 4, 1000, 1016
    buf = torch.zeros(R * step, device="cuda")
    x = buf.as_strided((R, V), (step, 1))
    x.copy_(logits(R, V, torch.float32, 3))
    u = uniform(R, 4)
    want = river.sample(x, u, top_p=0.9)
    o = {"token": buf[step + V:step + V + R].view(torch.int32), "logprob": buf[V + 8:V + 8 + R]}
    got = river.sample(x, u, top_p=0.9, out=o)
    check_sample(got, x, u, p=0.9)
    assert torch.equal(got["token"], want["token"]) and torch.equal(got["logprob"], want["logprob"])
    for at in (step + V - 1, step * 2 - R + 1):  # into the row in front, the row behind
        with pytest.raises(river.RiverError):
            river.sample(x, u, out={"logprob": buf[at:at + R]})
