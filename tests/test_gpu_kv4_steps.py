"""kv4_attention where the steps of the values differ from key to key: zeros in
front of, between and behind ordinary ones, the largest there are, negative
ones.  Tolerances as in test_gpu_serving_ops (which count steps by their size)."""
import math

import pytest

from tests.test_gpu_attention_ops import compare, rnd, river  # noqa: F401
from tests.test_gpu_serving_ops import check_kv4, held, i32, kv4_ref, make_cache, starts

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


def set_steps(cache, table, b, positions, value, minimum=None):
    """v's steps (and minima) of a sequence's positions, in every head."""
    page = cache.v_codes.shape[2]
    pos = torch.tensor(list(positions), dtype=torch.int64, device="cuda")
    cache.v_scale[table[b, pos // page].long(), :, pos % page, 0] = value
    if minimum is not None:
        cache.v_scale[table[b, pos // page].long(), :, pos % page, 1] = minimum


ZEROS = [range(32), range(128), range(256), range(1, 33), range(700), range(300, 700), [*range(64), *range(500, 900)], range(1000)]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D,Hq,rows", [(64, 4, 1), (128, 8, 1), (64, 4, 5), (128, 8, 4), (128, 32, 1)])
@pytest.mark.parametrize("zeros", ZEROS, ids=lambda z: f"{z[0]}-{z[-1]}-{len(z)}")
def test_steps_of_zero_beside_others(river, dtype, D, Hq, rows, zeros):  # noqa: F811
    """Flat scores, so that nothing else makes the kernel scale anew."""
    lens = [1024, 33, 1001]
    cache, table = make_cache(river, lens, 2, D, 16, dtype, 11)
    cache.k_scale.mul_(0.02)
    for b, n in enumerate(lens):
        set_steps(cache, table, b, [p for p in zeros if p < n], 0.0)
    q = rnd(3 * rows, Hq, D, dtype=dtype, seed=12)
    args = dict(start=starts([rows] * 3), max_rows=rows) if rows > 1 else {}
    check_kv4(river.kv4_attention(q, cache, table, i32(lens), **args), q, cache, table, lens, [rows] * 3)
    # rows of zeros as an append leaves them
    for b, n in enumerate(lens):
        set_steps(cache, table, b, [p for p in zeros if p < n], 0.0, 0.0)
    check_kv4(river.kv4_attention(q, cache, table, i32(lens), **args), q, cache, table, lens, [rows] * 3)


@pytest.mark.parametrize("rows", [1, 9])
def test_shares_that_start_among_steps_of_zero(river, rows):  # noqa: F811
    lens = [20000, 700, 9000]
    cache, table = make_cache(river, lens, 2, 128, 64, BF, 21)
    cache.k_scale.mul_(0.02)
    for b, n in enumerate(lens):
        set_steps(cache, table, b, [p for p in range(n) if p % 3000 < 1500], 0.0)
    q = rnd(3 * rows, 4, 128, dtype=BF, seed=22)
    got = river.kv4_attention(q, cache, table, i32(lens), start=starts([rows] * 3), max_rows=rows)
    check_kv4(got, q, cache, table, lens, [rows] * 3, most=3)


def test_zeros_first_give_what_they_give_last(river):  # noqa: F811
    """A sequence's output does not hang on what else is in the call."""
    lens = [640] + [100] * 40
    cache, table = make_cache(river, lens, 2, 64, 32, BF, 31)
    cache.k_scale.mul_(0.02)
    set_steps(cache, table, 0, range(320), 0.0)
    q = rnd(len(lens), 8, 64, dtype=BF, seed=32)
    alone = river.kv4_attention(q[:1], cache, table[:1].contiguous(), i32(lens[:1]))
    check_kv4(alone, q[:1], cache, table, lens[:1], [1])
    check_kv4(river.kv4_attention(q, cache, table, i32(lens)), q, cache, table, lens, [1] * len(lens))


@pytest.mark.parametrize("big", [1e33, 1e35, 1e36])
@pytest.mark.parametrize("rows", [1, 6])
def test_the_largest_steps(river, big, rows):  # noqa: F811
    """Values up to 15 times `big`, whose weighted sums stay in fp32's range (41 keys: 41 x 15 x 1e35; 9 with 1e36)."""
    lens = [41, 17, 9] if big < 1e36 else [9, 9, 3]
    lens = [max(n, rows) for n in lens]
    cache, table = make_cache(river, lens, 2, 64, 16, BF, 41)
    g = torch.Generator(device="cuda")
    g.manual_seed(42)
    s = (torch.rand(cache.v_scale.shape[:3], device="cuda", generator=g) * 0.9 + 0.1) * big
    cache.v_scale[..., 0] = s.to(BF)
    cache.v_scale[..., 1] = (-7.0 * s * torch.rand(s.shape, device="cuda", generator=g)).to(BF)
    q = rnd(3 * rows, 4, 64, dtype=BF, seed=43)
    args = dict(start=starts([rows] * 3), max_rows=rows) if rows > 1 else {}
    got = river.kv4_attention(q, cache, table, i32(lens), **args)
    assert torch.isfinite(got["out"]).all()
    check_kv4(got, q, cache, table, lens, [rows] * 3)


def test_a_row_over_the_types_whole_range(river):  # noqa: F811
    """The largest steps an append can leave, one key a sequence."""
    cache, table = make_cache(river, [1, 1], 2, 64, 16, BF, 51)
    k = rnd(2, 2, 64, dtype=BF, seed=52)
    v = (rnd(2, 2, 64, dtype=torch.float32, seed=53).tanh() * 1.6e38).to(BF)
    v[..., 0], v[..., 1] = -1.69e38, 1.69e38
    river.kv4_append(cache, table, i32([1, 1]), k, v)
    q = rnd(2, 4, 64, dtype=BF, seed=54)
    got = river.kv4_attention(q, cache, table, i32([1, 1]))
    assert torch.isfinite(got["out"]).all()
    check_kv4(got, q, cache, table, [1, 1], [1, 1])


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D,Hq,rows", [(64, 4, 1), (128, 8, 4)])
def test_steps_below_zero(river, dtype, D, Hq, rows):  # noqa: F811
    """A cache whose rows count down from their largest value, the sizes of the steps growing on the way."""
    lens = [600, 41]
    cache, table = make_cache(river, lens, 2, D, 16, dtype, 61)
    cache.k_scale.mul_(0.02)
    for b, n in enumerate(lens):
        set_steps(cache, table, b, range(0, n), -0.4)
        set_steps(cache, table, b, range(0, n // 2), -1e-4)
        set_steps(cache, table, b, range(n * 3 // 4, n), -300.0, 4000.0)
    q = rnd(2 * rows, Hq, D, dtype=dtype, seed=62)
    args = dict(start=starts([rows] * 2), max_rows=rows) if rows > 1 else {}
    got = river.kv4_attention(q, cache, table, i32(lens), **args)
    for b, n in enumerate(lens):
        (k, ks), (v, vs) = held(cache, table, b, n)
        refs = [kv4_ref(q[b * rows + t], [(k[:, : n - rows + t + 1], ks[:, : n - rows + t + 1]), (v[:, : n - rows + t + 1], vs[:, : n - rows + t + 1].abs())],
                        1 / math.sqrt(D)) for t in range(rows)]
        compare(got["out"][b * rows:(b + 1) * rows], got["lse"][b * rows:(b + 1) * rows], refs, f"sequence {b}")
