"""kv4_append, kv4_read, kv4_attention, packed_attention and sample against
float64.

Tolerances, from the arithmetic (u: a step's half as finfo.eps / 2 gives it,
bf16 2^-8, fp16 2^-11):
  appended queries   one rounding of a sum of two products: u |x| and 2 steps of
                     fp32 of the products' sizes
  appended codes     equal to the documented fp32 arithmetic's, bit for bit
  kv4_attention      q.k is a sum of head_dim products of q (to fp16: exact but
                     for head_dim values 2^-24 below the largest) and codes, times
                     s, plus m times a sum of q: off by at most
                     (2 head_dim + 8) 2^-24 A with A = max scale sum |q| (15 s + |m|),
                     which moves weights by twice that; the weights times s are
                     rounded to fp16 for the product with codes taken from 8:
                     2^-11 sum p 8 s, and those below 2^-14 of the largest by
                     2^-24 of it each; fp32 sums 1e-5; the result once, u |out|
  packed_attention   as window_attention
  sample             tokens are equal unless u or a filter's border is within
                     (vocab 2^-44 + 2^-36) of the sums in float64; logprob is the
                     logarithm of a quotient of two rounded numbers: 2^-22 (1 + |lp|)"""
import math

import pytest

from tests.test_gpu_attention_ops import compare, rnd, river, row_ref  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F64 = torch.float64
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
NAN, INF = float("nan"), float("inf")


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def starts(rows):
    s = [0]
    for n in rows:
        s.append(s[-1] + n)
    return i32(s)


def make_cache(river, lens, Hkv, D, page, dtype, seed, spare=2, width=None):
    """A cache of random codes and scales, pages dealt out at random."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    pages = [(n + page - 1) // page for n in lens]
    n_pages = sum(pages) + spare
    free = torch.randperm(n_pages, device="cuda", generator=g).to(torch.int32)
    W = width or max(1, max(pages))
    table = torch.full((len(lens), W), -7, dtype=torch.int32, device="cuda")  # (unused entries name no page)
    at = 0
    for b, p in enumerate(pages):
        table[b, :p] = free[at:at + p]
        at += p
    ts = []
    for _ in "kv":
        ts.append(torch.randint(0, 256, (n_pages, Hkv, page, D // 2), dtype=torch.uint8, device="cuda", generator=g))
        s = torch.rand((n_pages, Hkv, page), device="cuda", generator=g) * 0.4 + 0.1
        ts.append(torch.stack([s, -7.5 * s + 0.3 * torch.randn(s.shape, device="cuda", generator=g)], -1).to(dtype))
    return river.KV4Cache(*ts), table


def held(cache, table, b, n):
    """float64 [Hkv][n][D] values (and steps, minima) of k and v of sequence b."""
    out = []
    for c, s in (cache[:2], cache[2:]):
        page = c.shape[2]
        used = table[b, : (n + page - 1) // page].long()
        c, s = c[used], s[used].to(F64)
        v = torch.stack([c & 15, c >> 4], -1).flatten(-2).to(F64) * s[..., :1] + s[..., 1:]
        out.append(tuple(x.transpose(0, 1).flatten(1, 2)[:, :n] for x in (v, s)))
    return out


def kv4_ref(q, kv, scale):
    """One query row of every head: q [Hq][D] -> out, lse, tolerances."""
    (k, ks), (v, vs) = kv
    Hq, D = q.shape
    Hkv, n, _ = k.shape
    if n == 0:
        z = torch.zeros((Hq, D), dtype=F64, device="cuda")
        return z, torch.full((Hq,), -INF, dtype=F64, device="cuda"), z, z[:, 0]
    u = torch.finfo(q.dtype).eps / 2
    qq = q.to(F64).view(Hkv, Hq // Hkv, D)
    s = qq @ k.transpose(1, 2) * scale
    A = qq.abs().sum(-1, keepdim=True) * (15 * ks[..., 0].abs() + ks[..., 1].abs()).amax(-1)[:, None, None] * scale
    lse = torch.logsumexp(s, -1, keepdim=True)
    p = torch.exp(s - lse)
    out = p @ v
    size = (15 * vs[..., 0] + vs[..., 1].abs())[:, :, None]
    W, W8 = p @ size, p @ (8 * vs[..., :1])
    ds = (2 * D + 8) * 2.0 ** -24 * A
    top = (p * vs[..., 0][:, None]).amax(-1, keepdim=True)
    tol = u * out.abs() + 2.0 ** -11 * W8 + n * 2.0 ** -24 * 8 * top + (2 * ds + 1e-5) * W
    return out.reshape(Hq, D), lse.reshape(Hq), tol.reshape(Hq, D), (ds + 1e-5 + 2.0 ** -21 * lse.abs()).reshape(Hq)


def check_kv4(got, q, cache, table, lens, rows, scale=None, most=12):
    scale = 1 / math.sqrt(q.shape[2]) if scale is None else scale
    at = 0
    for b, (n, r) in enumerate(zip(lens, rows)):
        kv = held(cache, table, b, n)
        ts = sorted({i * r // most for i in range(most)} | {r - 1}) if r else []
        refs = [kv4_ref(q[at + t], [tuple(x[:, : max(0, n - r + t + 1)] for x in y) for y in kv], scale) for t in ts]
        if ts:
            compare(got["out"][[at + t for t in ts]], got["lse"][[at + t for t in ts]], refs, f"sequence {b} (n {n}, rows {r})")
        at += r


# ---------------------------------------------------------------- the cache's rows

def rotated(x, rope, pos):
    D = x.shape[-1]
    a, b = x.float()[..., : D // 2], x.float()[..., D // 2:]
    c, s = rope[pos, None, :, 0], rope[pos, None, :, 1]
    return torch.cat([a * c - b * s, b * c + a * s], -1).to(x.dtype)


def quantized(x):
    """The documented arithmetic in fp32: codes, (s, m)."""
    f = x.float()
    lo, hi = f.amin(-1, keepdim=True), f.amax(-1, keepdim=True)
    s = ((hi - lo) / 15).to(x.dtype).float()
    s = torch.where(s < 2.0 ** -100, 0.0, s)
    c = torch.where(s > 0, torch.round((f - lo) / torch.where(s > 0, s, 1.0)), 0.0).clamp(0, 15).to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4), torch.cat([s, lo], -1).to(x.dtype)


def check_append(river, rows, old, Hq, Hkv, D, page, dtype, seed, use_rope=True, with_q=True):
    lens = [a + b for a, b in zip(rows, old)]
    cache, table = make_cache(river, lens, Hkv, D, page, dtype, seed)
    before = [t.clone() for t in cache]
    N = sum(rows)
    qkv = rnd(N + 3, Hq + 2 * Hkv, D, dtype=dtype, seed=seed + 1, scale=2.0)
    q, k, v = qkv.split((Hq, Hkv, Hkv), dim=1)
    rope = river.rope_table(max(lens) + 1, D, 10000.0) if use_rope else None
    pos = torch.tensor([o + t for r, o in zip(rows, old) for t in range(r)], device="cuda")
    seq = torch.tensor([b for b, r in enumerate(rows) for _ in range(r)], device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    start = starts(rows)
    qo = rnd(*q.shape, dtype=dtype, seed=9)
    keep = qo.clone()
    got = river.kv4_append(cache, table, i32(lens), k, v, q=q if with_q else None, rope=rope, start=start, out={"q": qo} if with_q else None, err=err)
    assert int(err) == 0
    if with_q:
        assert got["q"] is qo and torch.equal(qo[N:], keep[N:])
        if use_rope and N:
            a, c = q[:N].to(F64).chunk(2, -1)
            cs, sn = (rope[pos, None, :, i].to(F64) for i in (0, 1))
            want = torch.cat([a * cs - c * sn, c * cs + a * sn], -1)
            size = torch.cat([(a * cs).abs() + (c * sn).abs(), (c * cs).abs() + (a * sn).abs()], -1)
            assert ((qo[:N].to(F64) - want).abs() <= torch.finfo(dtype).eps / 2 * want.abs() + 2 * 2.0 ** -24 * size + (2.0 ** -25 if dtype == FP else 0)).all()
        elif N:
            assert torch.equal(qo[:N], q[:N])
    kk = rotated(k[:N], rope, pos) if use_rope else k[:N]
    expect = before
    if N:
        at, row = table[seq, pos // page].long(), pos % page
        for i, x in ((0, kk), (2, v[:N])):
            expect[i][at, :, row], expect[i + 1][at, :, row] = quantized(x)
    for g, w in zip(cache, expect):
        assert torch.equal(g.view(torch.uint8), w.view(torch.uint8))
    # and back
    o = {x: rnd(N + 3, Hkv, D, dtype=dtype, seed=5 + i) for i, x in enumerate("kv")}
    keep = {x: t.clone() for x, t in o.items()}
    back = river.kv4_read(cache, table, i32(lens), start=start, rows=N + 3, out=o, err=err)
    assert int(err) == 0
    for i, x in ((0, "k"), (2, "v")):
        assert torch.equal(back[x][N:], keep[x][N:])
        if N:
            c, s = expect[i][at, :, row], expect[i + 1][at, :, row].float()
            assert torch.equal(back[x][:N], (s[..., 1:] + s[..., :1] * torch.stack([c & 15, c >> 4], -1).flatten(-2).float()).to(dtype))
    return cache, table, lens


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D,Hq,Hkv,page", [(64, 4, 2, 16), (128, 6, 3, 64), (64, 3, 1, 32), (128, 8, 8, 256), (128, 1, 1, 128)])
def test_append_and_read(river, dtype, D, Hq, Hkv, page):
    check_append(river, [3, 0, 40, 1, 17], [0, 5, 250, 63, 1], Hq, Hkv, D, page, dtype, 1)
    check_append(river, [1] * 33, list(range(33)), Hq, Hkv, D, page, dtype, 2)
    check_append(river, [1], [0], Hq, Hkv, D, page, dtype, 3, use_rope=False)
    check_append(river, [0, 0, 7], [0, 1, 2], Hq, Hkv, D, page, dtype, 4, with_q=False)


def test_append_many_rows(river):
    """Enough rows that a warp takes all of a row's heads."""
    check_append(river, [2500, 33, 501], [0, 1001, 7], 6, 2, 64, 32, BF, 11)
    check_append(river, [2499, 1, 0, 700], [3, 0, 0, 90], 5, 5, 128, 128, FP, 12)


def test_append_one_row_each_without_start(river):
    lens = [5, 1, 300]
    cache, table = make_cache(river, lens, 2, 64, 16, BF, 21)
    qkv = rnd(3, 8, 64, dtype=BF, seed=22)
    q, k, v = qkv.split((4, 2, 2), dim=1)
    rope = river.rope_table(300, 64, 500000.0)
    two = river.KV4Cache(*(t.clone() for t in cache))
    a = river.kv4_append(cache, table, i32(lens), k, v, q=q, rope=rope)
    b = river.kv4_append(two, table, i32(lens), k, v, q=q, rope=rope, start=i32(range(4)))
    assert torch.equal(a["q"], b["q"]) and all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(cache, two))
    x, y = river.kv4_read(cache, table, i32(lens)), river.kv4_read(cache, table, i32(lens), start=i32(range(4)), rows=3)
    assert torch.equal(x["k"], y["k"]) and torch.equal(x["v"], y["v"])
    # in q's place
    c = river.kv4_append(two, table, i32(lens), k, v, q=q, rope=rope, out={"q": q})
    assert torch.equal(c["q"], b["q"])


def test_rows_of_one_value_and_without_a_finite_range(river):
    cache, table = make_cache(river, [40], 1, 64, 16, BF, 31)
    k = rnd(40, 1, 64, dtype=BF, seed=32)
    k[0] = 3.25
    k[1] = 0.0
    k[2] = -0.0
    k[3] = 1e30
    k[4, 0, :32], k[4, 0, 32:] = -3e38, 3e38  # (their difference is infinite)
    k[5, 0, 7] = NAN
    k[6, 0, 7] = INF
    k[7, 0, 7] = -INF
    k[8, 0, 3] = 2.0 ** -120                   # a step below 2^-100
    k[8, 0, 4:] = k[8, 0, :3] = 0.0
    k[9, 0] = 1e-38 * torch.arange(64, device="cuda").to(BF)
    river.kv4_append(cache, table, i32([40]), k, k, start=i32([0, 40]))
    got = river.kv4_read(cache, table, i32([40]), start=i32([0, 40]), rows=40)["k"]
    for r in (0, 1, 2, 3):
        assert (got[r] == k[r]).all()
    for r in (4, 5, 6, 7):
        assert torch.isnan(got[r]).all(), r
    assert (got[8] == 0).all() and (got[9].float() - k[9].float()).abs().max() <= 64e-38
    s = (k[10:].float().amax(-1) - k[10:].float().amin(-1)) / 15
    assert ((got[10:].float() - k[10:].float()).abs() <= (s * (0.5 + 15 * 2.0 ** -8))[..., None] + 2.0 ** -8 * k[10:].float().abs()).all()


def test_append_refuses_places_outside_on_the_device(river):
    lens = [64, 65, 10, 200]
    cache, table = make_cache(river, [64, 64, 64, 64], 2, 64, 16, BF, 41, width=4)
    table[2, 0] = 10 ** 6
    before = [t.clone() for t in cache]
    k = rnd(4, 2, 64, dtype=BF, seed=42)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = torch.full((4, 4, 64), 7.0, dtype=BF, device="cuda")
    out = {"q": torch.zeros_like(q)}
    river.kv4_append(cache, table, i32(lens), k, k, q=q, out=out, err=err)
    assert int(err) == river.RL_DEVERR_CAPACITY
    assert (out["q"][0] == 7).all() and (out["q"][1:] == 0).all()
    expect = before
    for i in (0, 2):
        expect[i][table[0, 3].long(), :, 15], expect[i + 1][table[0, 3].long(), :, 15] = quantized(k[0])
    assert all(torch.equal(g.view(torch.uint8), w.view(torch.uint8)) for g, w in zip(cache, expect))
    err.zero_()
    river.kv4_append(cache, table, i32([64, 0, -5, 3]), k, k, rope=river.rope_table(64, 64, 1e4), err=err)
    assert int(err) == river.RL_DEVERR_CAPACITY
    err.zero_()
    river.kv4_append(cache, table, i32([64] * 4), k, k, rope=river.rope_table(63, 64, 1e4), err=err)  # (position 63)
    assert int(err) == river.RL_DEVERR_CAPACITY
    for start in ([0, 5, 2, 3, 4], [0, 1, 2, 3, 9], [-1, 1, 2, 3, 4]):
        err.zero_()
        river.kv4_append(cache, table, i32([64, 64, 1, 64]), k, k, start=i32(start), err=err)
        assert int(err) == river.RL_DEVERR_CAPACITY, start


# ---------------------------------------------------------------- attention over the cache

@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D,Hq,Hkv,page", [(64, 4, 4, 16), (64, 8, 2, 32), (128, 8, 1, 16), (128, 12, 4, 64), (128, 24, 2, 128), (64, 20, 1, 256)])
def test_kv4_single_tokens(river, dtype, D, Hq, Hkv, page):
    lens = [0, 1, 2, 15, 16, 17, 129, 700, 513, 255]
    cache, table = make_cache(river, lens, Hkv, D, page, dtype, 51)
    q = rnd(len(lens), Hq, D, dtype=dtype, seed=52, scale=1.5)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = river.kv4_attention(q, cache, table, i32(lens), err=err)
    assert int(err) == 0
    check_kv4(got, q, cache, table, lens, [1] * len(lens))
    got = river.kv4_attention(q, cache, table, i32(lens), scale=0.31)
    check_kv4(got, q, cache, table, lens, [1] * len(lens), scale=0.31)


@pytest.mark.parametrize("D,Hq,Hkv,page", [(64, 4, 2, 16), (128, 8, 2, 32), (128, 3, 1, 64), (64, 32, 2, 128)])
def test_kv4_drafts(river, D, Hq, Hkv, page):
    for dtype in (BF, FP):
        rows, lens = [2, 5, 0, 1, 16, 7, 3], [2, 900, 10, 77, 401, 4, 0]
        cache, table = make_cache(river, lens, Hkv, D, page, dtype, 61)
        N = sum(rows)
        q = rnd(N + 2, Hq, D, dtype=dtype, seed=62, scale=1.5)
        for most in (16, None):
            o = {"out": rnd(N + 2, Hq, D, dtype=dtype, seed=63), "lse": rnd(N + 2, Hq, dtype=F32, seed=64)}
            keep = {x: t.clone() for x, t in o.items()}
            got = river.kv4_attention(q, cache, table, i32(lens), start=starts(rows), max_rows=most, out=o)
            check_kv4(got, q, cache, table, lens, rows)
            assert all(torch.equal(o[x][N:], keep[x][N:]) for x in o)


def test_kv4_long_contexts(river):
    for lens, rows, D, Hq, Hkv, page, dtype in (([70001, 8192], [1, 1], 128, 8, 2, 128, BF), ([33333], [4], 64, 4, 2, 16, FP),
                                                ([9000] * 40 + [5] * 30, [1] * 70, 64, 4, 4, 64, BF)):
        cache, table = make_cache(river, lens, Hkv, D, page, dtype, 71)
        q = rnd(sum(rows), Hq, D, dtype=dtype, seed=72, scale=1.5)
        got = river.kv4_attention(q, cache, table, i32(lens), start=starts(rows), max_rows=max(rows))
        check_kv4(got, q, cache, table, lens, rows)
        assert all(torch.equal(got[x], y) for x, y in river.kv4_attention(q, cache, table, i32(lens), start=starts(rows), max_rows=max(rows)).items())


def test_kv4_scales_of_every_size(river):
    """Steps and minima over the whole range of the type, peaked rows, steps of 0."""
    for dtype, big in ((BF, 1e30), (FP, 3000.0)):
        lens = [300, 41]
        cache, table = make_cache(river, lens, 2, 64, 16, dtype, 81)
        q = rnd(2, 4, 64, dtype=dtype, seed=82)
        g = torch.Generator(device="cuda")
        g.manual_seed(3)
        small = 1e-30 if dtype == BF else 1e-6
        span = torch.exp(torch.rand(cache.v_scale.shape[:3], device="cuda", generator=g) * (math.log(big) - math.log(small)) + math.log(small))
        cache.v_scale[..., 0] = span.to(dtype)
        cache.v_scale[..., 1] = (span * torch.randn(span.shape, device="cuda", generator=g)).to(dtype)
        check_kv4(river.kv4_attention(q, cache, table, i32(lens)), q, cache, table, lens, [1, 1])
        cache.v_scale[..., 0] = 0  # a step of 0: every value the minimum
        check_kv4(river.kv4_attention(q, cache, table, i32(lens)), q, cache, table, lens, [1, 1])
        cache.v_scale[..., 0] = span.to(dtype)
        cache.k_scale[..., 0] *= 30  # one key takes nearly all
        check_kv4(river.kv4_attention(q, cache, table, i32(lens)), q, cache, table, lens, [1, 1])
        cache.k_scale[..., 0] = 0
        cache.k_scale[..., 1] = 0  # all alike
        check_kv4(river.kv4_attention(q, cache, table, i32(lens)), q, cache, table, lens, [1, 1])


def test_kv4_queries_of_every_size(river):
    lens = [200] * 6
    for dtype, sizes in ((BF, [1e-30, 1e-8, 1e-3, 1.0, 50.0, 0.0]), (FP, [1e-7, 1e-5, 1e-3, 1.0, 50.0, 0.0])):
        cache, table = make_cache(river, lens, 2, 64, 32, dtype, 91)
        q = (rnd(6, 4, 64, dtype=F32, seed=92) * torch.tensor(sizes, device="cuda")[:, None, None]).to(dtype)
        q[3, 0, 1] = 1e-5  # beside values around 1
        check_kv4(river.kv4_attention(q, cache, table, i32(lens)), q, cache, table, lens, [1] * 6)


@pytest.mark.parametrize("bad", [NAN, INF])
def test_kv4_positions_behind_have_no_part(river, bad):
    lens, rows = [333, 40, 17, 64], [1, 5, 1, 3]
    for D, Hq in ((64, 4), (128, 32)):
        cache, table = make_cache(river, lens, 2, D, 32, BF, 101)
        q = rnd(sum(rows), Hq, D, dtype=BF, seed=102)
        clean = river.kv4_attention(q, cache, table, i32(lens), start=starts(rows), max_rows=5)
        for b, n in enumerate(lens):
            p = table[b, (n - 1) // 32].long()
            if n % 32:
                cache.k_scale[p, :, n % 32:] = bad
                cache.v_scale[p, :, n % 32:] = bad
        got = river.kv4_attention(q, cache, table, i32(lens), start=starts(rows), max_rows=5)
        assert torch.equal(got["out"], clean["out"]) and torch.equal(got["lse"], clean["lse"])
        # a key that only the last row of a draft sees
        cache.v_scale[table[1, 1].long(), 0, 39 % 32, 1] = bad
        got = river.kv4_attention(q, cache, table, i32(lens), start=starts(rows), max_rows=5)
        h = Hq // 2
        assert not torch.isfinite(got["out"][5, :h]).any()
        mask = torch.ones_like(got["out"], dtype=torch.bool)
        mask[5, :h] = False
        assert torch.equal(got["out"][mask], clean["out"][mask]) and torch.equal(got["lse"], clean["lse"])


def test_kv4_device_errors_and_bounds(river):
    lens = [30, 31, 32]
    cache, table = make_cache(river, lens, 2, 64, 16, BF, 111, width=2)
    q = rnd(3, 4, 64, dtype=BF, seed=112)
    want = river.kv4_attention(q, cache, table, i32(lens))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = river.kv4_attention(q, cache, table, i32([30, 10 ** 9, -4]), err=err)
    assert int(err) == river.RL_DEVERR_CAPACITY
    assert torch.equal(got["out"][0], want["out"][0]) and (got["out"][2] == 0).all() and (got["lse"][2] == -INF).all()
    check_kv4(got, q, cache, table, [30, 32], [1, 1])
    err.zero_()
    bad = table.clone()
    bad[1, 1] = -1
    got = river.kv4_attention(q, cache, bad, i32(lens), err=err)
    assert int(err) == river.RL_DEVERR_CAPACITY and torch.equal(got["out"][0], want["out"][0]) and torch.equal(got["out"][2], want["out"][2])
    bad[1, 1] = 0  # (page 0 is read instead)
    check_kv4(got, q, cache, bad, lens, [1] * 3)
    # more rows than max_rows says
    rows = [3, 5, 1]
    q = rnd(9, 4, 64, dtype=BF, seed=113)
    err.zero_()
    o = {"out": torch.full_like(q, 9.0)}
    got = river.kv4_attention(q, cache, table, i32(lens), start=starts(rows), max_rows=3, out=o, err=err)
    assert int(err) == river.RL_DEVERR_CAPACITY and (got["out"][6:8] == 9).all()
    all_ = river.kv4_attention(q, cache, table, i32(lens), start=starts(rows))
    check_kv4(all_, q, cache, table, lens, rows)
    for r in (0, 1, 2, 3, 4, 5, 8):
        assert (got["out"][r].float() - all_["out"][r].float()).abs().max() < 0.05, r


def test_kv4_starts_that_overlap(river):
    """Reported, and the next call is right: with more units than all rows have (five
    sequences, three of them of all rows), and with fewer."""
    rows, lens = [16, 0, 0, 0, 0], [64, 0, 70, 0, 80]
    cache, table = make_cache(river, [64, 64, 70, 70, 80], 2, 64, 16, BF, 114, width=5)
    q = rnd(16, 16, 64, dtype=BF, seed=115)
    want = river.kv4_attention(q, cache, table, i32(lens), start=starts(rows))
    check_kv4(want, q, cache, table, lens, rows)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for start in ([0, 16, 0, 16, 0, 16], [0, 10, 5, 12, 12, 16]):
        err.zero_()
        river.kv4_attention(q, cache, table, i32(lens), start=i32(start), err=err)
        assert int(err) == river.RL_DEVERR_CAPACITY, start
        got = river.kv4_attention(q, cache, table, i32(lens), start=starts(rows))
        assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])


def test_kv4_strides_and_views(river):
    """Heads cut out of a fused projection; the cache one layer of a pool."""
    lens = [100, 47]
    pool, table = make_cache(river, [200, 200], 2, 128, 16, BF, 121)
    n = pool.k_codes.shape[0] // 2
    cache = river.KV4Cache(*(t[1:2 * n:2] for t in pool))
    table = (table % n).contiguous()
    wide = torch.cat([table, table], 1)[:, : table.shape[1]]
    fused = rnd(2, 16, 128, dtype=BF, seed=122)
    q = fused[:, 4:12]
    out = torch.zeros((2, 12, 128), dtype=BF, device="cuda")
    got = river.kv4_attention(q, cache, wide, i32(lens), out={"out": out[:, 2:10]})
    check_kv4(got, q, cache, wide, lens, [1, 1])
    assert (out[:, :2] == 0).all() and (out[:, 10:] == 0).all()
    k = rnd(2, 2, 128, dtype=BF, seed=123)
    keep = [t.clone() for t in pool]
    river.kv4_append(cache, wide, i32(lens), k, k)
    assert all(torch.equal(t[0::2].view(torch.uint8), x[0::2].view(torch.uint8)) for t, x in zip(pool, keep))


# ---------------------------------------------------------------- packed prompts

def check_packed(got, q, k, v, rows, scale=None, most=24):
    scale = 1 / math.sqrt(q.shape[2]) if scale is None else scale
    at = 0
    for b, n in enumerate(rows):
        ts = sorted({i * n // most for i in range(most)} | {n - 1}) if n else []
        refs = [row_ref(q[at + t], k[at:at + t + 1].transpose(0, 1), v[at:at + t + 1].transpose(0, 1), scale) for t in ts]
        if ts:
            compare(got["out"][[at + t for t in ts]], got["lse"][[at + t for t in ts]], refs, f"sequence {b} of {n}")
        at += n


def packed_case(rows, Hq, Hkv, D, dtype, seed, extra=0):
    qkv = rnd(sum(rows) + extra, Hq + 2 * Hkv, D, dtype=dtype, seed=seed, scale=1.3)
    return qkv.split((Hq, Hkv, Hkv), dim=1)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 4), (128, 8, 2), (64, 12, 4), (128, 8, 1), (64, 32, 2), (128, 3, 1)])
def test_packed_prompts(river, dtype, D, Hq, Hkv):
    for rows in ([1], [0, 1, 2, 0, 33, 64, 0], [128, 129, 127, 1, 300], [256, 512, 11], [1] * 70):
        q, k, v = packed_case(rows, Hq, Hkv, D, dtype, 131, extra=5)
        N = sum(rows)
        for most in (max(rows), None):
            o = {"out": rnd(*q.shape, dtype=dtype, seed=3), "lse": rnd(N + 5, Hq, dtype=F32, seed=4)}
            keep = {x: t.clone() for x, t in o.items()}
            err = torch.zeros(1, dtype=torch.int32, device="cuda")
            got = river.packed_attention(q, k, v, starts(rows), max_rows=most, out=o, err=err)
            assert int(err) == 0
            check_packed(got, q, k, v, rows, most=9)
            assert all(torch.equal(o[x][N:], keep[x][N:]) for x in o)


def test_packed_long(river):
    rows = [5003, 2048, 1, 777]
    q, k, v = packed_case(rows, 8, 2, 128, BF, 141)
    got = river.packed_attention(q, k, v, starts(rows), scale=0.2)
    check_packed(got, q, k, v, rows, scale=0.2)
    again = river.packed_attention(q, k, v, starts(rows), scale=0.2)
    assert all(torch.equal(got[x], again[x]) for x in got)
    # one sequence alone
    s0, s1 = 5003, 5003 + 2048
    one = river.packed_attention(q[s0:s1], k[s0:s1], v[s0:s1], i32([0, 2048]), scale=0.2)
    check_packed(one, q[s0:s1], k[s0:s1], v[s0:s1], [2048], scale=0.2)


def test_packed_many_sequences(river):
    g = torch.Generator()
    g.manual_seed(1)
    rows = torch.randint(0, 40, (1200,), generator=g).tolist()
    q, k, v = packed_case(rows, 4, 2, 64, FP, 151)
    check_packed(river.packed_attention(q, k, v, starts(rows), max_rows=40), q, k, v, rows, most=2)


@pytest.mark.parametrize("bad", [NAN, INF])
@pytest.mark.parametrize("D", [64, 128])
def test_packed_rows_see_their_own_sequence_only(river, bad, D):
    """Values of other sequences, and of later rows, have no part."""
    rows = [200, 77, 130, 300]
    q, k, v = packed_case(rows, 4, 2, D, BF, 161, extra=40)
    k, v = k.contiguous(), v.contiguous()
    clean = river.packed_attention(q, k, v, starts(rows))
    kb, vb = k.clone(), v.clone()
    for x in (kb, vb):
        x[277:407] = bad          # the third sequence
        x[707:] = bad             # behind the last
    got = river.packed_attention(q, kb, vb, starts(rows))
    for s in (slice(0, 277), slice(407, 707)):
        assert torch.equal(got["out"][s], clean["out"][s]) and torch.equal(got["lse"][s], clean["lse"][s])
    vb = v.clone()
    vb[100, 0, 3] = bad           # rows from 100 on of the first see it
    got = river.packed_attention(q, k, vb, starts(rows))
    assert not torch.isfinite(got["out"][100:200, :2, 3]).any()
    same = torch.ones_like(clean["out"], dtype=torch.bool)
    same[:200, :2] = False
    same[707:] = False
    assert torch.equal(got["out"][same], clean["out"][same])
    check_packed({"out": got["out"][:100], "lse": got["lse"][:100]}, q, k, vb, [100])


def test_packed_strides_device_errors(river):
    rows = [40, 50]
    q, k, v = packed_case(rows, 4, 2, 64, BF, 171)
    want = river.packed_attention(q, k, v, starts(rows))
    kt, vt = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (k, v))  # head-major
    out = torch.zeros((90, 7, 64), dtype=BF, device="cuda")
    got = river.packed_attention(q.contiguous(), kt, vt, starts(rows), out={"out": out[:, 2:6]})
    assert torch.equal(got["out"], want["out"]) and (out[:, :2] == 0).all() and (out[:, 6] == 0).all()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for start in ([0, 40, 95], [-3, 40, 90], [0, 60, 50], [90, 0, 90]):
        err.zero_()
        river.packed_attention(q, k, v, i32(start), err=err)
        assert int(err) == river.RL_DEVERR_CAPACITY, start
    err.zero_()
    o = {"out": torch.full_like(want["out"], 5.0)}
    got = river.packed_attention(q, k, v, starts(rows), max_rows=45, out=o, err=err)
    assert int(err) == river.RL_DEVERR_CAPACITY and (got["out"][85:] == 5).all()
    check_packed(got, q, k, v, [40, 45])


# ---------------------------------------------------------------- sampling

def sample_ref(x, u, T, k, p, mp):
    """Token, logprob, and whether every border is far enough to be sure."""
    x = x.to(F64)
    V = x.numel()
    m, first = float(x.max()), int((x == x.max()).nonzero()[0, 0])
    if not T > 0:
        return first, 0.0, True
    w = torch.exp((x - m) / T)
    order = torch.sort(x, descending=True, stable=True).indices
    ws = w[order]
    keep = torch.ones(V, dtype=torch.bool, device="cuda")
    if 1 <= k < V:
        keep[k:] = False
    eps = V * 2.0 ** -44 + 2.0 ** -36
    sure = True
    S = float(ws[keep].sum())
    if p < 1:
        before = torch.cat([torch.zeros(1, dtype=F64, device="cuda"), ws.cumsum(0)[:-1]])
        sure = sure and not ((before[1:] - p * S).abs() < eps * S)[keep[1:]].any()
        keep &= before < p * S
    if mp > 0:
        keep &= ws >= mp
    keep[0] = True
    ids = order[keep].sort().values
    c = w[ids].cumsum(0)
    at = min(max(u, 0.0), 1 - 2.0 ** -24) * float(c[-1])
    i = int((c <= at).sum())
    edge = [float(c[j]) for j in (i - 1, i) if 0 <= j < len(ids)]
    # (u 0 is the first id whose weight is not 0, exactly; weights around 2^-44 may round either way)
    sure = sure and all(abs(e - at) > eps * float(c[-1]) or e == at == 0 for e in edge)
    if at == 0:
        sure = sure and bool((w[ids[:i]] == 0).all())
    return int(ids[i]), math.log(float(w[ids[i]]) / float(c[-1])), sure


def check_sample(got, x, u, T=1.0, k=0, p=1.0, mp=0.0):
    R = x.shape[0]

    def each(a):
        return a.tolist() if isinstance(a, torch.Tensor) else [float(torch.tensor(a, dtype=F32)) if isinstance(a, float) else a] * R
    seen = 0
    for r, (uu, t, kk, pp, m) in enumerate(zip(u.tolist(), each(T), each(k), each(p), each(mp))):
        tok, lp, sure = sample_ref(x[r], uu, t, kk, pp, m)
        if sure:
            seen += 1
            assert int(got["token"][r]) == tok, (r, uu, t, kk, pp, m, int(got["token"][r]), tok)
            assert abs(float(got["logprob"][r]) - lp) <= 2.0 ** -22 * (1 + abs(lp)), (r, float(got["logprob"][r]), lp)
    assert seen >= 0.8 * R  # (the check has not run empty)


def logits(R, V, dtype, seed, scale=2.0):
    x = rnd(R, V, dtype=F32, seed=seed, scale=scale)
    if V > 20:
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        x.scatter_add_(1, torch.randint(0, V, (R, 6), device="cuda", generator=g), torch.rand((R, 6), device="cuda", generator=g) * 10)
    return x.to(dtype)


def uniform(R, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.rand(R, device="cuda", generator=g)


SETTINGS = [dict(), dict(T=0.7), dict(T=1.7, k=50), dict(k=1), dict(p=0.9), dict(T=0.8, k=40, p=0.95), dict(mp=0.05), dict(T=1.3, p=0.5, mp=0.01),
            dict(k=7, p=0.3, mp=0.2), dict(T=0.0), dict(p=0.0), dict(mp=1.0), dict(k=10 ** 9, p=1.5), dict(T=5.0, p=0.999), dict(k=3000), dict(mp=3.0)]


def call(river, x, u, T=1.0, k=0, p=1.0, mp=0.0, **kw):
    return river.sample(x, u, temperature=T, top_k=k, top_p=p, min_p=mp, **kw)


@pytest.mark.parametrize("dtype", [F32, BF, FP])
@pytest.mark.parametrize("R,V", [(1, 1), (3, 2), (5, 33), (4, 1000), (2, 50257), (1, 128256), (9, 7001), (200, 3001)])
def test_sample(river, dtype, R, V):
    x = logits(R, V, dtype, R + V)
    for i, s in enumerate(SETTINGS if R < 10 else SETTINGS[5:8]):
        u = uniform(R, 7 * i + V)
        check_sample(call(river, x, u, **s), x, u, **s)


def test_sample_largest_vocabulary(river):
    x = logits(3, 2 ** 19, F32, 3)
    for i, s in enumerate((dict(), dict(T=3.0, p=0.97), dict(k=100000, p=0.5))):
        u = uniform(3, i)
        check_sample(call(river, x, u, **s), x, u, **s)


def test_sample_settings_of_each_row(river):
    R, V = 64, 20011
    x, u = logits(R, V, F32, 1), uniform(R, 2)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    T = torch.rand(R, device="cuda", generator=g) * 2
    T[::7] = 0
    T[3] = -1.0
    k = torch.randint(-2, 60, (R,), device="cuda", generator=g).to(torch.int32)
    p = torch.rand(R, device="cuda", generator=g) * 1.2
    mp = torch.rand(R, device="cuda", generator=g) * 0.1 - 0.02
    check_sample(call(river, x, u, T, k, p, mp), x, u, T, k, p, mp)
    T[5], p[6], mp[7], p[8], T[9] = NAN, NAN, NAN, -1.0, INF
    x[9, ::3] = -INF
    got = call(river, x, u, T, k, p, mp)
    p[6], mp[7], p[8], T[9] = 1.0, 0.0, 0.0, 1e30
    check_sample(got, x, u, T, k, p, mp)


@pytest.mark.parametrize("R", [305, 1500, 2048, 2049])
def test_sample_many_rows_of_their_own_settings(river, R):
    """Rows in whatever order give what a few of them alone do; only the costliest, or none of a kind, too."""
    V = 16501  # (longer rows are put in order of their cost)
    x, u = logits(R, V, F32, 21), uniform(R, 22)
    g = torch.Generator(device="cuda")
    g.manual_seed(23)
    T = torch.rand(R, device="cuda", generator=g) + 0.3
    T[torch.rand(R, device="cuda", generator=g) < 0.2] = 0
    k = torch.randint(-150, 200, (R,), device="cuda", generator=g).to(torch.int32)
    p = torch.rand(R, device="cuda", generator=g) * 1.6
    full = torch.full((R,), 0.9, device="cuda")
    for s in (dict(T=T, k=k, p=p), dict(T=torch.zeros_like(T), k=k), dict(T=T), dict(p=full), dict(k=k, mp=0.01)):
        whole = call(river, x, u, **s)
        for i in range(0, R, 250):
            few = call(river, x[i:i + 250], u[i:i + 250], **{n: v[i:i + 250] if torch.is_tensor(v) else v for n, v in s.items()})
            assert torch.equal(whole["token"][i:i + 250], few["token"]) and torch.equal(whole["logprob"][i:i + 250], few["logprob"])
        check_sample({n: t[:60] for n, t in whole.items()}, x[:60], u[:60], **{n: v[:60] if torch.is_tensor(v) else v for n, v in s.items()})


@pytest.mark.parametrize("R,V", [(2, 40009), (40, 4003)])
def test_sample_orders_and_ties(river, R, V):
    """Ties at every border, all logits equal, sorted rows."""
    rows = [torch.full((V,), 0.25, device="cuda"), (torch.arange(V, device="cuda") % 3 == 0).float(), torch.linspace(-8, 8, V, device="cuda"),
            torch.linspace(8, -8, V, device="cuda"), torch.where(torch.arange(V, device="cuda") % 2 == 0, 0.0, -0.0)]
    for j, row in enumerate(rows):
        x = row.repeat(R, 1).contiguous()
        for i, s in enumerate((dict(), dict(k=100), dict(p=0.3), dict(k=1000, p=0.77), dict(T=0.5, mp=0.3), dict(k=V - 1), dict(T=0.0), dict(p=1e-30))):
            u = uniform(R, 31 * j + i)
            check_sample(call(river, x, u, **s), x, u, **s)


def test_sample_borders_of_u(river):
    V = 3000
    x = logits(8, V, F32, 5)
    x[:, :5] = -INF
    u = torch.tensor([0.0, 1 - 2.0 ** -24, 1.0, 7.0, -1.0, NAN, 2.0 ** -149, 2.0 ** -30], device="cuda")
    ref = torch.tensor([0.0, 1 - 2.0 ** -24, 1 - 2.0 ** -24, 1 - 2.0 ** -24, 0.0, 0.0, 0.0, 2.0 ** -30], device="cuda")
    for s in (dict(), dict(k=5), dict(p=0.8), dict(T=0.5)):
        check_sample(call(river, x, u, **s), x, ref, **s)


def test_sample_extremes(river):
    V = 2001
    x = logits(8, V, F32, 6)
    x[0] = -INF
    x[1, 9] = INF
    x[1, 10] = INF
    x[2, 77] = NAN
    x[3] = -torch.finfo(F32).max
    x[4, 1] = 3e38
    x[5, :2000] = -INF
    x[6] = x[6] * 1e-30
    u = uniform(8, 9)
    for s in (dict(), dict(k=3), dict(p=0.7, mp=0.01), dict(T=0.0)):
        got = call(river, x, u, **s)
        assert got["token"][:3].tolist() == [0, 9, 77] and torch.isnan(got["logprob"][:3]).all()
        check_sample({n: t[3:] for n, t in got.items()}, x[3:], u[3:], **s)
    got = call(river, x[6:], u[6:], T=1e-30)
    check_sample(got, x[6:], u[6:], T=1e-30)


def test_sample_temperatures_without_an_end(river):
    """An infinite one is the largest finite one: every id weighs the same, and is below 1."""
    x, u = logits(6, 999, F32, 16), uniform(6, 17)
    T = torch.full((6,), INF, device="cuda")
    check_sample(call(river, x, u, T=T), x, u, T=torch.finfo(F32).max)
    check_sample(call(river, x, u, T=T, k=3), x, u, T=torch.finfo(F32).max, k=3)
    got = call(river, x, u, T=T, mp=1.0)
    assert torch.equal(got["token"].long(), x.argmax(1)) and (got["logprob"] == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_sample_strided_rows_and_odd_starts(river, dtype):
    flat = logits(9, 2011, dtype, 8).view(-1)
    for off, V in ((0, 1999), (1, 2000), (3, 517), (5, 64), (7, 9)):
        x = torch.as_strided(flat, (8, V), (2011, 1), off)
        u = uniform(8, V)
        check_sample(call(river, x, u, k=20, p=0.9), x, u, k=20, p=0.9)


def test_sample_shares_follow_the_weights(river):
    """Evenly spaced u: every token as often as its share, to one."""
    x = torch.tensor([[0.5, -1.0, 2.0, 0.0, 1.0, -INF]], device="cuda").repeat(1000, 1)
    u = (torch.arange(1000, device="cuda") + 0.5) / 1000
    n = torch.bincount(call(river, x, u)["token"].long(), minlength=6)
    assert ((n - 1000 * torch.softmax(x[0], 0)).abs() <= 1).all()


def test_sample_buffers_and_refusals(river):
    x, u = logits(2, 64, F32, 1), uniform(2, 1)
    o = {"token": torch.full((2,), -1, dtype=torch.int32, device="cuda")}
    got = river.sample(x, u, out=o)
    assert got["token"] is o["token"]
    check_sample(got, x, u)
    for kw in (dict(temperature=-1.0), dict(temperature=NAN), dict(top_k=-1), dict(top_p=-0.1), dict(min_p=INF),
               dict(temperature=torch.ones(3, device="cuda")), dict(top_k=torch.ones(2, device="cuda")), dict(out={"logprob": torch.zeros(3, device="cuda")})):
        with pytest.raises(river.RiverError):
            river.sample(x, u, **kw)
    for bad in (u[:1], u.double(), u.cpu()):
        with pytest.raises(river.RiverError):
            river.sample(x, bad)
    with pytest.raises(river.RiverError) as e:
        river.sample(torch.zeros((1, 2 ** 19 + 1), device="cuda"), u[:1])
    assert e.value.status == river.RL_ERR_UNSUPPORTED


# ---------------------------------------------------------------- together

def test_a_serving_loop(river):
    """Prompts packed, appended, attended to; then steps and drafts over the cache; tokens drawn."""
    Hq, Hkv, D, page = 8, 2, 64, 16
    rows = [37, 5, 120, 1]
    dtype = BF
    lens = list(rows)
    cache, table = make_cache(river, [n + 30 for n in lens], Hkv, D, page, dtype, 201)
    rope = river.rope_table(256, D, 10000.0)
    q, k, v = packed_case(rows, Hq, Hkv, D, dtype, 202)
    st = starts(rows)
    qr = river.kv4_append(cache, table, i32(lens), k, v, q=q, rope=rope, start=st)["q"]
    kv = river.kv4_read(cache, table, i32(lens), start=st, rows=sum(rows))
    prompt = river.packed_attention(qr, kv["k"], kv["v"], st, max_rows=max(rows))
    check_packed(prompt, qr, kv["k"], kv["v"], rows)
    # the same rows over the cache itself (whose values the read rounds once more)
    direct = river.kv4_attention(qr, cache, table, i32(lens), start=st, max_rows=max(rows))
    check_kv4(direct, qr, cache, table, lens, rows)
    W = rnd(Hq * D, 500, dtype=F32, seed=203, scale=0.1)
    for step, new in enumerate(([1, 1, 1, 1], [1, 1, 1, 1], [3, 1, 2, 4], [1, 0, 1, 1])):
        lens = [a + b for a, b in zip(lens, new)]
        q, k, v = packed_case(new, Hq, Hkv, D, dtype, 210 + step)
        one = new == [1, 1, 1, 1]
        st = None if one else starts(new)
        qr = river.kv4_append(cache, table, i32(lens), k, v, q=q, rope=rope, start=st)["q"]
        got = river.kv4_attention(qr, cache, table, i32(lens), start=st, max_rows=None if one else 4)
        check_kv4(got, qr, cache, table, lens, new)
        x = got["out"].float().flatten(1) @ W
        u = uniform(x.shape[0], step)
        check_sample(river.sample(x, u, temperature=0.9, top_k=40, top_p=0.95), x, u, T=0.9, k=40, p=0.95)


def test_streams_capture_and_repeat(river):
    lens, rows = [900, 33, 2000], [1, 2, 4]
    cache, table = make_cache(river, [n + 16 for n in lens], 2, 64, 16, BF, 301)
    rope = river.rope_table(4096, 64, 10000.0)
    st, n = starts(rows), i32(lens)
    qkv = rnd(7, 8, 64, dtype=BF, seed=302)
    W = rnd(256, 5000, dtype=F32, seed=303, scale=0.2)
    u = uniform(7, 304)

    def chain(stream=None):
        q, k, v = qkv.split((4, 2, 2), dim=1)
        qr = river.kv4_append(cache, table, n, k, v, q=q, rope=rope, start=st, stream=stream)["q"]
        kv = river.kv4_read(cache, table, n, start=st, rows=7, stream=stream)
        att = river.kv4_attention(qr, cache, table, n, start=st, max_rows=4, stream=stream)
        p = river.packed_attention(qr, kv["k"], kv["v"], st, max_rows=4, stream=stream)
        return qr, kv["k"], kv["v"], att["out"], att["lse"], p["out"], p["lse"]

    def drawn(x, stream=None):
        return river.sample(x, u, top_k=50, top_p=0.9, stream=stream)

    want = chain()
    x = want[3].float().flatten(1) @ W
    tok = drawn(x)
    check_sample(tok, x, u, k=50, p=0.9)
    assert all(torch.equal(a, b) for a, b in zip(want, chain()))
    assert all(torch.equal(tok[y], t) for y, t in drawn(x).items())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other, ot = chain(s), drawn(x, s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, other)) and all(torch.equal(tok[y], ot[y]) for y in tok)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = chain()
        gt = drawn(x)
    qkv.copy_(rnd(7, 8, 64, dtype=BF, seed=305))
    n.copy_(i32([905, 40, 2011]))
    x.copy_(rnd(7, 5000, dtype=F32, seed=306, scale=2.0))
    g.replay()
    torch.cuda.synchronize()
    check_kv4({"out": got[3], "lse": got[4]}, got[0], cache, table, [905, 40, 2011], rows)
    assert all(torch.equal(a, b) for a, b in zip(chain(), got))
    check_sample(gt, x, u, k=50, p=0.9)


def test_offsets_past_32_bits(river):
    """Pages, rows of operands and rows of logits 2^31 bytes and more apart give what compact ones do, bit for bit."""
    if torch.cuda.get_device_properties(0).total_memory < 1 << 36:
        pytest.skip("needs 64 GB")
    lens, rows = [33, 40], [2, 3]
    small, table = make_cache(river, lens, 2, 128, 16, BF, 131)
    n, st, pages = i32(lens), starts(rows), small.k_codes.shape[0]
    cs, ss = (1 << 31) - 4096, (1 << 30) - 4096
    codes = torch.empty((pages - 1) * cs + 4096, dtype=torch.uint8, device="cuda")
    scales = torch.empty((pages - 1) * ss + 256, dtype=BF, device="cuda")
    far = river.KV4Cache(*(b.as_strided(t.shape, (step, *t.stride()[1:]), at) for t, b, step, at in zip(
        small, (codes, scales) * 2, (cs, ss) * 2, (0, 0, 2048, 128))))
    for x, y in zip(far, small):
        x.copy_(y)
    step = 1 << 30
    wide = torch.empty(4 * step + 4096, dtype=BF, device="cuda")
    q, out = (wide.as_strided((5, 8, 128), (step, 128, 1), at) for at in (0, 1024))
    k, v = (wide.as_strided((5, 2, 128), (step, 128, 1), at) for at in (2048, 2304))
    for x, seed in ((q, 132), (k, 133), (v, 134)):
        x.copy_(rnd(*x.shape, dtype=BF, seed=seed))
    cq, ck, cv = (x.clone(memory_format=torch.contiguous_format) for x in (q, k, v))
    want = river.kv4_append(small, table, n, ck, cv, q=cq, start=st)["q"]
    assert torch.equal(river.kv4_append(far, table, n, k, v, q=q, start=st, out={"q": out})["q"], want)
    assert all(torch.equal(x.contiguous().view(torch.uint8), y.view(torch.uint8)) for x, y in zip(far, small))
    want = river.kv4_attention(cq, small, table, n, start=st)
    check_kv4(want, cq, small, table, lens, rows)
    got = river.kv4_attention(q, far, table, n, start=st, out={"out": out})
    assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])
    want = river.packed_attention(cq, ck, cv, st)
    assert torch.equal(river.packed_attention(q, k, v, st, out={"out": out})["out"], want["out"])
    want = river.kv4_read(small, table, n, start=st, rows=5)
    river.kv4_read(far, table, n, start=st, rows=5, out={"k": k, "v": v})
    assert torch.equal(k, want["k"]) and torch.equal(v, want["v"])
    del far, codes, scales, q, out, k, v, wide
    x, u = logits(3, 9001, BF, 135), uniform(3, 136)
    wide = torch.empty(2 * (1 << 31) + 9001, dtype=BF, device="cuda")
    y = wide.as_strided(x.shape, (1 << 31, 1))
    y.copy_(x)
    assert all(torch.equal(a, b) for a, b in zip(call(river, x, u, p=0.9).values(), call(river, y, u, p=0.9).values()))


def test_two_calls_at_once(river):
    """Several streams with calls in flight together."""
    lens = [3000, 1234, 77, 8000]
    cache, table = make_cache(river, lens, 2, 128, 64, BF, 401)
    q = rnd(4, 8, 128, dtype=BF, seed=402)
    rows = [500, 300]
    pq, pk, pv = packed_case(rows, 8, 2, 128, BF, 403)
    x, u = logits(8, 128256, F32, 404), uniform(8, 405)
    n, st = i32(lens), starts(rows)
    want = (river.kv4_attention(q, cache, table, n), river.packed_attention(pq, pk, pv, st), river.sample(x, u, top_p=0.9))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(6)]
    got = []
    for i in range(18):
        s = streams[i % 6]
        got.append((i % 3, river.kv4_attention(q, cache, table, n, stream=s) if i % 3 == 0 else
                    river.packed_attention(pq, pk, pv, st, stream=s) if i % 3 == 1 else river.sample(x, u, top_p=0.9, stream=s)))
    torch.cuda.synchronize()
    for i, o in got:
        assert all(torch.equal(o[y], want[i][y]) for y in o)


def test_derivatives_are_refused(river):
    from tests.test_ops_edges import derivatives_refused
    cache, table = make_cache(river, [20], 2, 64, 16, BF, 501)
    n, z = i32([20]), torch.zeros((1, 2, 64), dtype=BF, device="cuda")
    q = torch.zeros((1, 4, 64), dtype=BF, device="cuda")
    u = torch.zeros(1, device="cuda")
    for call_, ops in ((lambda q, k, v: river.packed_attention(q, k, v, i32([0, 1])), [q, z, z]),
                       (lambda q: river.kv4_attention(q, cache, table, n), [q]),
                       (lambda k, v, q: river.kv4_append(cache, table, n, k, v, q=q), [z, z, q]),
                       (lambda x, u: river.sample(x, u), [torch.zeros((1, 9), device="cuda"), u])):
        derivatives_refused(river, call_, ops, range(len(ops)), lambda c: c())
