"""window_attention and shared_prefix_attention against float64.

Tolerances, from the arithmetic.  With u = half a step of the type (2^-9 ... as
eps / 2: bf16 2^-8, fp16 2^-11), p the exact weights and W = sum p |v|: the
result is rounded once (u |out|) and the weights once for the product with v
(u W).  A score is a sum of head_dim fp32 products: off by at most
head_dim 2^-24 A with A = max_j sum_i |q_i k_ji| scale, which moves every
weight by that relative amount and the normalised ones by twice it; fp32 sums
over n keys and the exponential add less than 1e-5 W.  fp16 weights below
2^-14 of a row's largest (2^-24 steps) add at most n 2^-24 max |v|."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F64 = torch.float64
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def river():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import __graft_entry__
    __graft_entry__.build()
    import early_exit_decoding_gb300 as r
    return r


def rnd(*shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, device="cuda", generator=g) * scale).to(dtype)


def row_ref(q, k, v, scale):
    """One query row of every head: q [Hq][D], k, v [Hkv][n][D] -> out, lse, tolerances."""
    Hq, D = q.shape
    Hkv, n, _ = k.shape
    rep = Hq // Hkv
    if n == 0:
        z = torch.zeros((Hq, D), dtype=F64, device="cuda")
        return z, torch.full((Hq,), float("-inf"), dtype=F64, device="cuda"), z, z[:, 0]
    u = torch.finfo(v.dtype).eps / 2
    q = q.to(v.dtype).to(F64).view(Hkv, rep, D)
    k, v = k.to(F64), v.to(F64)
    s = q @ k.transpose(1, 2) * scale
    A = (q.abs() @ k.abs().transpose(1, 2)).amax(-1, keepdim=True) * scale
    lse = torch.logsumexp(s, -1, keepdim=True)
    p = torch.exp(s - lse)
    out, W = p @ v, p @ v.abs()
    ds = D * 2.0 ** -24 * A
    tol = u * (out.abs() + W) + (2 * ds + 1e-5) * W
    if u == 2.0 ** -11:
        tol = tol + n * 2.0 ** -24 * v.abs().amax() * p.amax(-1, keepdim=True)
    return out.reshape(Hq, D), lse.reshape(Hq), tol.reshape(Hq, D), (ds + 1e-5 + 2.0 ** -21 * lse.abs()).reshape(Hq)


def compare(got_o, got_l, refs, label):
    o, l, to, tl = (torch.stack(x) for x in zip(*refs))
    d = (got_o.to(F64) - o).abs()
    assert torch.isfinite(got_o).all(), f"{label}: not finite"
    assert (d <= to).all(), f"{label}: out off by {d.max()} ({(d / to.clamp(min=1e-30)).max()} of the tolerance)"
    dead = torch.isinf(l)
    assert torch.equal(got_l.to(F64)[dead], l[dead]), label
    dl = (got_l.to(F64) - l).abs()
    assert (dl[~dead] <= tl[~dead]).all(), f"{label}: lse off by {dl[~dead].max()}"


def check_window(got, q, k, v, kv_len, q_len, window, sinks, scale=None, rows=40, before=None):
    B, T, Hq, D = q.shape
    scale = 1 / math.sqrt(D) if scale is None else scale
    for b in range(B):
        n, ql = int(kv_len[b]), T if q_len is None else int(q_len[b])
        if before is not None:
            assert torch.equal(got["out"][b, ql:], before["out"][b, ql:]) and torch.equal(got["lse"][b, ql:], before["lse"][b, ql:])
        ts = sorted({min(ql - 1, i * ql // rows) for i in range(rows)} | {ql - 1, max(0, ql - 2)}) if ql else []
        refs = []
        for t in ts:
            p = n - ql + t
            j = torch.arange(max(0, p + 1), device="cuda")
            j = j[(p - j < window) | (j < sinks)]
            refs.append(row_ref(q[b, t], k[b][:, j], v[b][:, j], scale))
        if ts:
            compare(got["out"][b, ts], got["lse"][b, ts], refs, f"sequence {b} (n {n}, ql {ql})")


def window_case(B, T, Hq, Hkv, D, cap, dtype, seed, q_dtype=None):
    q = rnd(B, T, Hq, D, dtype=q_dtype or dtype, seed=seed, scale=1.5)
    k = rnd(B, Hkv, cap, D, dtype=dtype, seed=seed + 1)
    v = rnd(B, Hkv, cap, D, dtype=dtype, seed=seed + 2)
    return q, k, v


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (4, 2), (12, 4), (8, 1), (20, 1)])
def test_window_single_tokens(river, dtype, D, Hq, Hkv):
    cap = 700
    q, k, v = window_case(8, 1, Hq, Hkv, D, cap, dtype, 1)
    n = i32(0, 1, 2, 16, 129, 513, 699, 700)
    for window, sinks in ((1, 0), (16, 4), (128, 0), (300, 17), (700, 3), (5000, 9000), (64, 200)):
        got = river.window_attention(q, k, v, n, window, sinks)
        check_window(got, q, k, v, n, None, window, sinks)


@pytest.mark.parametrize("window,sinks", [(1, 0), (7, 2), (100, 4), (128, 130), (2000, 0)])
@pytest.mark.parametrize("T,D,Hq,Hkv", [(2, 64, 4, 2), (5, 128, 8, 2), (17, 128, 4, 4), (65, 64, 8, 2), (300, 128, 6, 2), (257, 64, 3, 1)])
def test_window_queries(river, T, D, Hq, Hkv, window, sinks):
    cap = 1000
    for dtype in (BF, FP):
        q, k, v = window_case(5, T, Hq, Hkv, D, cap, dtype, 11)
        n = i32(T, T + 1, 1000, max(0, T - 3), 0)
        ql = i32(T, T - 1, T, T, min(2, T))
        before = {"out": rnd(*q.shape, dtype=dtype, seed=3), "lse": rnd(5, T, Hq, dtype=torch.float32, seed=4)}
        got = river.window_attention(q, k, v, n, window, sinks, q_len=ql, out={a: t.clone() for a, t in before.items()})
        check_window(got, q, k, v, n, ql, window, sinks, before=before)


def test_window_long_prompt_and_context(river):
    q, k, v = window_case(1, 3001, 8, 2, 128, 5003, BF, 21)
    n = i32(5003)
    for window, sinks in ((1024, 4), (5003, 0), (130, 300)):
        check_window(river.window_attention(q, k, v, n, window, sinks), q, k, v, n, None, window, sinks)
    q, k, v = window_case(2, 1, 8, 2, 64, 40000, FP, 22)
    n = i32(39999, 20011)
    for window, sinks in ((40000, 0), (9000, 33)):
        check_window(river.window_attention(q, k, v, n, window, sinks), q, k, v, n, None, window, sinks)


def test_window_fp32_queries_and_scale(river):
    for T in (1, 40):
        q, k, v = window_case(2, T, 8, 2, 64, 200, BF, 31, q_dtype=torch.float32)
        n = i32(200, 77)
        got = river.window_attention(q, k, v, n, 50, 2, scale=0.3)
        check_window(got, q, k, v, n, None, 50, 2, scale=0.3)


@pytest.mark.parametrize("T", [1, 6, 150])
def test_window_strides(river, T):
    """Token-major caches, heads cut out of a fused projection, one cache shared by all sequences."""
    Hq, Hkv, D, cap = 4, 2, 64, 300
    fused = rnd(3, T, Hq + 2 * Hkv, D, dtype=BF, seed=41)
    q = fused[:, :, :Hq]
    kv = rnd(3, cap, 2, Hkv, D, dtype=BF, seed=42)
    k, v = kv[:, :, 0].permute(0, 2, 1, 3), kv[:, :, 1].permute(0, 2, 1, 3)
    out = torch.zeros((3, T, Hq + 2, D), dtype=BF, device="cuda")
    n = i32(300, 151, T)
    got = river.window_attention(q, k, v, n, 90, 5, out={"out": out[:, :, 1:1 + Hq]})
    check_window(got, q, k, v, n, None, 90, 5)
    assert (out[:, :, 0] == 0).all() and (out[:, :, -1] == 0).all()
    k1, v1 = k[:1].expand(3, -1, -1, -1), v[:1, :1].expand(3, Hkv, -1, -1)
    check_window(river.window_attention(q, k1, v1, n, 90, 5), q, k1, v1, n, None, 90, 5)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("T", [1, 4, 200])
def test_window_masked_keys_have_no_part(river, T, bad):
    """NaN and infinities where no row, or only some rows, look."""
    q, k, v = window_case(2, T, 4, 2, 64, 600, BF, 51)
    n = i32(400, 333)
    clean = river.window_attention(q, k, v, n, 60, 3)
    kb, vb = k.clone(), v.clone()
    for b in range(2):
        for x in (kb, vb):
            x[b, :, int(n[b]):] = bad                        # behind the sequence
            x[b, :, 3:int(n[b]) - T - 60 + 1] = bad          # before every row's window
    got = river.window_attention(q, kb, vb, n, 60, 3)
    assert torch.equal(got["out"], clean["out"]) and torch.equal(got["lse"], clean["lse"])
    if T > 1:
        # a key that only the first rows see: they are not finite, the others are untouched
        j = int(n[0]) - T - 60 + 2
        vb[0, 0, j, 5] = bad
        got = river.window_attention(q, kb, vb, n, 60, 3)
        p = int(n[0]) - T + torch.arange(T)
        sees = (p - j < 60) & (p >= j)
        assert sees.any() and not sees.all()
        assert not torch.isfinite(got["out"][0, sees.cuda(), :2, 5]).any()
        check_window(got, q, k, v, i32(0, int(n[1])), i32(0, T), 60, 3)
        ts = [t for t in range(T) if not sees[t]]
        refs = []
        for t in ts:
            jj = torch.arange(int(p[t]) + 1, device="cuda")
            jj = jj[(int(p[t]) - jj < 60) | (jj < 3)]
            refs.append(row_ref(q[0, t], k[0][:, jj], v[0][:, jj], 0.125))
        compare(got["out"][0, ts], got["lse"][0, ts], refs, "rows that do not see it")


@pytest.mark.parametrize("D,dtype", [(64, FP), (128, BF)])
def test_window_masked_keys_of_many_sequences(river, D, dtype):
    """As above with more row tiles than the GPU holds at once (no tile's keys
    are split): the first row sees a NaN, the other rows of its tile do not."""
    B, T, W = 40, 64, 50
    q, k, v = window_case(B, T, 8, 8, D, 150, dtype, 61)
    n = torch.arange(B, dtype=torch.int32, device="cuda") + 105
    ql = torch.full((B,), T, dtype=torch.int32, device="cuda")
    ql[::3] = 33
    clean = river.window_attention(q, k, v, n, W, 2, q_len=ql)
    check_window(clean, q, k, v, n, ql, W, 2, rows=4)
    vb = v.clone()
    for b in range(B):
        # the first row's oldest key in the window (below 0, with no such key: a slot behind the sequence)
        j = int(n[b]) - int(ql[b]) - W + 1
        vb[b, :, j, 1] = float("nan")
    got = river.window_attention(q, k, vb, n, W, 2, q_len=ql)
    hit = (n - ql - W + 1 >= 0)[:, None].expand(B, 8)
    assert hit.any() and not hit.all() and torch.equal(torch.isnan(got["out"][:, 0, :, 1]), hit)
    refs = []
    for b in range(B):
        for t in (0, 1 + b % 7):
            p = int(n[b]) - int(ql[b]) + t
            jj = torch.arange(p + 1, device="cuda")
            jj = jj[(p - jj < W) | (jj < 2)]
            ref = row_ref(q[b, t], k[b][:, jj], v[b][:, jj], 1 / math.sqrt(D))
            if t == 0:  # (its other dims)
                assert ((got["out"][b, 0].to(F64) - ref[0]).abs() <= ref[2])[:, 2:].all()
            elif b == 8:  # (its key is a sink: every row sees it)
                assert int(n[b]) - int(ql[b]) - W + 1 == 0 and torch.isnan(got["out"][b, t, :, 1]).all()
            else:
                refs.append(ref)
    ar = torch.tensor([b for b in range(B) if b != 8], device="cuda")
    compare(got["out"][ar, 1 + ar % 7], got["lse"][ar, 1 + ar % 7], refs, "rows that do not see it")


def test_window_wider_than_any_length(river):
    """Windows and sinks beyond 32 bits are plain causal attention."""
    q, k, v = window_case(2, 3, 4, 2, 64, 90, BF, 71)
    n = i32(90, 41)
    want = river.window_attention(q, k, v, n, 90)
    for w, s in ((2**31 - 1, 0), (2**32 + 5, 0), (7, 2**40)):
        got = river.window_attention(q, k, v, n, w, s)
        check_window(got, q, k, v, n, None, w, s)
        assert s or (torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"]))


def test_buffers_that_overlap_themselves(river):
    q, k, v = window_case(2, 3, 4, 2, 64, 40, BF, 81)
    n = i32(40, 11)
    for out in (torch.empty((1, 3, 4, 64), dtype=BF, device="cuda").expand(2, 3, 4, 64),
                torch.empty(2000, dtype=BF, device="cuda").as_strided((2, 3, 4, 64), (768, 256, 32, 1))):
        with pytest.raises(river.RiverError):
            river.window_attention(q, k, v, n, 8, out={"out": out})
    qp, kp, vp, kq, vq = prefix_case(2, 4, 2, 64, 64, 20, BF, 91)
    with pytest.raises(river.RiverError):
        river.shared_prefix_attention(qp, kp, vp, kq, vq, i32(20, 3),
                                      workspace=torch.empty(1, dtype=torch.uint8, device="cuda").expand(1 << 20))


def test_window_lengths_outside_the_buffers(river):
    q, k, v = window_case(3, 4, 4, 2, 64, 100, BF, 61)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = river.window_attention(q, k, v, i32(100, 50, 0), 30, q_len=i32(4, 4, 0), err=err)
    assert int(err) == 0
    for n, ql in ((i32(101, 50, 0), i32(4, 4, 0)), (i32(100, -3, 0), i32(4, 4, 0)), (i32(100, 50, 0), i32(5, 4, 0)), (i32(100, 50, 0), i32(4, -1, 0))):
        err.zero_()
        o = {"out": torch.zeros_like(q), "lse": torch.zeros((3, 4, 4), device="cuda")}
        o = river.window_attention(q, k, v, n, 30, q_len=ql, err=err, out=o)
        assert int(err) == river.RL_DEVERR_CAPACITY
        check_window(o, q, k, v, n.clamp(0, 100), ql.clamp(0, 4), 30, 0)
    assert torch.isfinite(got["out"][:2]).all()


def test_window_offsets_past_32_bits(river):
    """A cache whose last sequence starts 2^32 elements in."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 20 GB")
    cap, D = 1 << 22, 128
    k = torch.empty((5, 2, cap, D), dtype=BF, device="cuda")
    k[4, :, :300] = rnd(2, 300, D, dtype=BF, seed=71)
    k[4, :, cap - 300:] = rnd(2, 300, D, dtype=BF, seed=72)
    assert k.stride(0) * 4 >= 1 << 32
    for T in (1, 200):
        q = rnd(5, T, 4, D, dtype=BF, seed=73)
        n = i32(0, 0, 0, 0, cap)
        got = river.window_attention(q, k, k, n, 100, 20)
        check_window({a: t[4:] for a, t in got.items()}, q[4:], k[4:], k[4:], n[4:], None, 100, 20, rows=5)
        assert (got["out"][:4] == 0).all()


@pytest.mark.parametrize("T", [1, 5, 300])
def test_window_streams_capture_and_repeat(river, T):
    q, k, v = window_case(3, T, 8, 2, 128, 2000, BF, 81)
    n = i32(2000, 1000, 333)
    want = river.window_attention(q, k, v, n, 512, 4)
    again = river.window_attention(q, k, v, n, 512, 4)
    assert all(torch.equal(want[a], again[a]) for a in want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = river.window_attention(q, k, v, n, 512, 4, stream=s)
    s.synchronize()
    assert all(torch.equal(want[a], other[a]) for a in want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = river.window_attention(q, k, v, n, 512, 4)
    n.copy_(i32(1999, 400, 301))
    g.replay()
    torch.cuda.synchronize()
    check_window(got, q, k, v, n, None, 512, 4, rows=8)


# ------------------------------------------------------------- shared prefix

def check_prefix(got, q, kp, vp, k, v, n, scale=None, prefix=None):
    B, Hq, D = q.shape
    scale = 1 / math.sqrt(D) if scale is None else scale
    refs = []
    for b in range(B):
        m = int(n[b])
        refs.append(row_ref(q[b], torch.cat([kp, k[b, :, :m]], 1), torch.cat([vp, v[b, :, :m]], 1), scale))
    compare(got["out"], got["lse"], refs, "shared prefix")


def prefix_case(B, Hq, Hkv, D, P, cap, dtype, seed, q_dtype=None):
    return (rnd(B, Hq, D, dtype=q_dtype or dtype, seed=seed, scale=1.5), rnd(Hkv, P, D, dtype=dtype, seed=seed + 1),
            rnd(Hkv, P, D, dtype=dtype, seed=seed + 2), rnd(B, Hkv, cap, D, dtype=dtype, seed=seed + 3),
            rnd(B, Hkv, cap, D, dtype=dtype, seed=seed + 4))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,Hq,Hkv,P,cap", [(1, 1, 1, 1, 1), (1, 4, 2, 127, 40), (3, 8, 2, 128, 70), (5, 12, 4, 1000, 64), (33, 8, 1, 300, 33),
                                            (64, 8, 2, 2049, 130), (130, 4, 1, 129, 20), (9, 20, 1, 5000, 300)])
def test_prefix_values(river, dtype, D, B, Hq, Hkv, P, cap):
    q, kp, vp, k, v = prefix_case(B, Hq, Hkv, D, P, cap, dtype, 91)
    n = torch.tensor([cap * b // max(1, B - 1) if B > 1 else cap for b in range(B)], dtype=torch.int32, device="cuda")
    check_prefix(river.shared_prefix_attention(q, kp, vp, k, v, n), q, kp, vp, k, v, n)


@pytest.mark.parametrize("B,Hq,Hkv,D,P,cap,dtype", [(160, 8, 4, 64, 300, 40, BF), (620, 3, 1, 128, 130, 17, FP), (80, 72, 4, 128, 513, 33, BF),
                                                    (320, 8, 2, 128, 1, 300, BF), (640, 1, 1, 64, 2000, 5, FP)])
def test_prefix_many_sequences(river, B, Hq, Hkv, D, P, cap, dtype):
    """More own-key tiles than the GPU holds at once: a third launch joins."""
    q, kp, vp, k, v = prefix_case(B, Hq, Hkv, D, P, cap, dtype, 171)
    n = (torch.arange(B, device="cuda") * 7 % (cap + 1)).to(torch.int32)
    got = river.shared_prefix_attention(q, kp, vp, k, v, n)
    check_prefix(got, q, kp, vp, k, v, n)
    again = river.shared_prefix_attention(q, kp, vp, k, v, n)
    assert torch.equal(got["out"], again["out"]) and torch.equal(got["lse"], again["lse"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        o = river.shared_prefix_attention(q, kp, vp, k, v, n)
    for t in o.values():
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got["out"], o["out"]) and torch.equal(got["lse"], o["lse"])


@pytest.mark.parametrize("Hq", [64, 128, 256])
def test_many_heads_of_one_kv_head(river, Hq):
    for T in (1, 5):
        q, k, v = window_case(2, T, Hq, 1, 64, 300, BF, 181)
        n = i32(300, 7)
        check_window(river.window_attention(q, k, v, n, 90, 5), q, k, v, n, None, 90, 5)
    c = prefix_case(3, Hq, 1, 64, 200, 20, BF, 183)
    check_prefix(river.shared_prefix_attention(*c, i32(20, 0, 9)), *c, i32(20, 0, 9))


def test_window_queries_shared_by_sequences_or_heads(river):
    q, k, v = window_case(3, 40, 4, 2, 128, 200, BF, 185)
    n = i32(200, 50, 3)
    for x in (q[:1].expand(3, -1, -1, -1), q[:, :, :1].expand(-1, -1, 4, -1), q[:, :1].expand(-1, 40, -1, -1)):
        check_window(river.window_attention(x, k, v, n, 60, 2), x, k, v, n, None, 60, 2)


def test_prefix_alone_own_keys_alone_and_nothing(river):
    q, kp, vp, k, v = prefix_case(4, 8, 2, 64, 200, 50, BF, 101)
    zero = i32(0, 0, 0, 0)
    check_prefix(river.shared_prefix_attention(q, kp, vp, k, v, zero), q, kp, vp, k, v, zero)
    n = i32(50, 1, 0, 17)
    got = river.shared_prefix_attention(q, kp[:, :0], vp[:, :0], k, v, n)
    check_prefix(got, q, kp[:, :0], vp[:, :0], k, v, n)
    assert (got["out"][2] == 0).all() and (got["lse"][2] == float("-inf")).all()


def test_prefix_strides_fp32_queries_and_garbage_behind(river):
    """The prefix in a cache's first sequence, rows behind the lengths NaN."""
    Hq, Hkv, D, cap = 8, 2, 128, 900
    cache_k, cache_v = rnd(6, Hkv, cap, D, dtype=BF, seed=111), rnd(6, Hkv, cap, D, dtype=BF, seed=112)
    P = 700
    n = i32(1, 200, 33, 0, 64, 7)
    for b in range(6):
        cache_k[b, :, P + int(n[b]):] = float("nan")
        cache_v[b, :, P + int(n[b]):] = float("nan")
        if b:
            cache_k[b, :, :P] = float("nan")
            cache_v[b, :, :P] = float("nan")
    q = rnd(6, Hq, D, dtype=torch.float32, seed=113, scale=1.5)
    args = (cache_k[0, :, :P], cache_v[0, :, :P], cache_k[:, :, P:], cache_v[:, :, P:], n)
    got = river.shared_prefix_attention(q, *args, scale=0.1)
    check_prefix(got, q, *args, scale=0.1)
    # a prefix whose last tile is followed by NaN rows
    cache_k[0, :, 650:], cache_v[0, :, 650:] = float("nan"), float("nan")
    args = (cache_k[0, :, :650], cache_v[0, :, :650], *prefix_case(6, Hq, Hkv, D, 1, 250, BF, 114)[3:], n)
    check_prefix(river.shared_prefix_attention(q, *args), q, *args)


def test_prefix_not_finite_stays_in_its_sequence(river):
    q, kp, vp, k, v = prefix_case(3, 4, 2, 64, 100, 20, BF, 121)
    n = i32(20, 20, 20)
    clean = river.shared_prefix_attention(q, kp, vp, k, v, n)
    v[1, :, 3] = float("inf")
    got = river.shared_prefix_attention(q, kp, vp, k, v, n)
    assert torch.equal(got["out"][::2], clean["out"][::2]) and not torch.isfinite(got["out"][1]).any()


def test_prefix_lengths_workspace_and_refusals(river):
    q, kp, vp, k, v = prefix_case(2, 4, 2, 64, 64, 20, BF, 131)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = river.shared_prefix_attention(q, kp, vp, k, v, i32(21, -1), err=err)
    assert int(err) == river.RL_DEVERR_CAPACITY
    check_prefix(got, q, kp, vp, k, v, i32(20, 0))
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    got = river.shared_prefix_attention(q, kp, vp, k, v, i32(20, 3), workspace=ws)
    check_prefix(got, q, kp, vp, k, v, i32(20, 3))
    with pytest.raises(river.RiverError):
        river.shared_prefix_attention(q, kp, vp, k, v, i32(20, 3), workspace=ws[:16])
    with pytest.raises(river.RiverError):
        river.shared_prefix_attention(q, kp[:1], vp, k, v, i32(20, 3))
    with pytest.raises(river.RiverError):
        river.shared_prefix_attention(q, kp, vp, k, v, i32(20, 3, 4))


def test_prefix_two_graphs_and_streams(river):
    """Two captured calls replayed at the same time do not share a workspace."""
    cases = [prefix_case(16, 8, 2, 128, 3000 + i, 64, BF, 141 + 7 * i) for i in range(2)]
    n = torch.arange(16, dtype=torch.int32, device="cuda") * 4
    want = [river.shared_prefix_attention(*c, n) for c in cases]
    assert all(torch.equal(a, b) for a, b in zip(want[0].values(), river.shared_prefix_attention(*cases[0], n).values()))
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(river.shared_prefix_attention(*c, n))
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(o[a], w[a]) for a in w)
