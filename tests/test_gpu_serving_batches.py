"""The largest batches the packed and paged operators take: 2^16 sequences, most of a row, some of none or a few.
Tolerances as in test_gpu_serving_ops."""
import pytest

from tests.test_gpu_attention_ops import compare, rnd, river, row_ref  # noqa: F401
from tests.test_gpu_serving_ops import held, i32, kv4_ref, make_cache, quantized, starts

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF = torch.bfloat16
B = 1 << 16


def lengths(seed, most):
    g = torch.Generator()
    g.manual_seed(seed)
    n = torch.ones(B, dtype=torch.int64)
    some = torch.randperm(B, generator=g)[:2000]
    n[some] = torch.randint(0, most + 1, (2000,), generator=g)
    n[0], n[1], n[-2], n[-1] = 0, most, most, 1
    return n.tolist(), sorted({0, 1, B - 2, B - 1, *some[:60].tolist(), *range(0, B, 1021)})


def test_packed_prompts_of_the_largest_batch(river):  # noqa: F811
    rows, look = lengths(1, 300)
    st = starts(rows)
    first = st.tolist()
    N, scale = first[-1], 0.125
    q, k, v = rnd(N, 4, 64, dtype=BF, seed=2).split((2, 1, 1), dim=1)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = river.packed_attention(q, k, v, st, max_rows=300, scale=scale, err=err)
    assert int(err) == 0
    for b in look:
        at, n = first[b], rows[b]
        ts = sorted({0, n // 2, n - 1}) if n else []
        refs = [row_ref(q[at + t], k[at:at + t + 1].transpose(0, 1), v[at:at + t + 1].transpose(0, 1), scale) for t in ts]
        if ts:
            compare(got["out"][[at + t for t in ts]], got["lse"][[at + t for t in ts]], refs, f"sequence {b} of {n}")
    # a row alone gives its value
    one = torch.tensor([first[b] for b in range(B) if rows[b] == 1], device="cuda")
    assert torch.equal(got["out"][one], v[one].expand(-1, 2, -1))


@pytest.mark.parametrize("drafts", [False, True])
def test_a_step_of_the_largest_batch(river, drafts):  # noqa: F811
    lens, look = lengths(3, 60)
    rows = [min(n, 1 + b % 3) for b, n in enumerate(lens)] if drafts else [1] * B
    lens = [max(n, r) for n, r in zip(lens, rows)]
    cache, table = make_cache(river, lens, 1, 64, 16, BF, 4)
    N, st, n = sum(rows), starts(rows), i32(lens)
    first = st.tolist()
    q, k, v = rnd(N, 4, 64, dtype=BF, seed=5).split((2, 1, 1), dim=1)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = dict(start=st) if drafts else {}
    river.kv4_append(cache, table, n, k, v, err=err, **args)
    back = river.kv4_read(cache, table, n, err=err, **(dict(start=st, rows=N) if drafts else {}))
    c, s = quantized(k)
    assert torch.equal(back["k"], (s[..., 1:].float() + s[..., :1].float() * torch.stack([c & 15, c >> 4], -1).flatten(-2).float()).to(BF))
    got = river.kv4_attention(q, cache, table, n, max_rows=3 if drafts else None, err=err, **args)
    assert int(err) == 0
    for b in look:
        kv = held(cache, table, b, lens[b])
        r = rows[b]
        refs = [kv4_ref(q[first[b] + t], [tuple(x[:, :lens[b] - r + t + 1] for x in y) for y in kv], 0.125) for t in range(r)]
        if refs:
            compare(got["out"][first[b]:first[b] + r], got["lse"][first[b]:first[b] + r], refs, f"sequence {b}")
