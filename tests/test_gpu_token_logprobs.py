"""token_logprobs against float64.

Tolerances, from the arithmetic (u = 2^-24): the terms exp(x - m) carry a
relative error of at most |x - m| 2u + 4u, the fp32 sums at most n_seq u with
n_seq <= 300 sequential additions a thread, so ln s is off by less than
300 u + 2u E + 8u < 2e-5 (1 + E / 100) with E = sum |x - m| e / s; the entropy
adds the same relative error of its second term, (2e-5)(1 + 2 E); results are
rounded once more, 2u of their size."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F64 = torch.float64


@pytest.fixture(scope="module")
def river():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import __graft_entry__
    __graft_entry__.build()
    import early_exit_decoding_gb300 as r
    return r


def check(logits, tokens, top_k, got):
    x = logits.to(F64)
    m = x.amax(1, keepdim=True)
    y = x - m  # shifted first: at the lowest finite value lse itself rounds to m
    ln_s = torch.logsumexp(y, 1)
    lse = m[:, 0] + ln_s
    d = torch.where(torch.isinf(y), 0.0, y)
    p = torch.exp(y - ln_s[:, None])
    E = (d.abs() * p).sum(1)
    ent = ln_s - (d * p).sum(1)
    tol = 2e-5 * (1 + E / 100) + 4 * U * lse.abs()
    assert got["lse"].dtype == torch.float32
    assert ((got["lse"].to(F64) - lse).abs() <= tol).all(), (got["lse"].to(F64) - lse).abs().max()
    assert ((got["entropy"].to(F64) - ent).abs() <= 2e-5 * (1 + 2 * E) + 4 * U * ent.abs()).all()
    if tokens is not None:
        t = tokens.view(len(x), -1).long()
        ref = y.gather(1, t) - ln_s[:, None]
        g = got["logprob"].to(F64).view_as(ref)
        fin = torch.isfinite(ref)
        assert torch.equal(g[~fin], ref[~fin])
        assert ((g - ref).abs()[fin] <= (tol[:, None] + 4 * U * (ref.abs() + ln_s.abs()[:, None]))[fin]).all()
    if top_k:
        val, ids = torch.sort(x, dim=1, descending=True, stable=True)
        assert torch.equal(got["top_ids"].long(), ids[:, :top_k])
        ref = val[:, :top_k] - m - ln_s[:, None]
        g = got["top_logprobs"].to(F64)
        fin = torch.isfinite(ref)
        assert torch.equal(g[~fin], ref[~fin])
        assert ((g - ref).abs()[fin] <= (tol[:, None] + 4 * U * (ref.abs() + ln_s.abs()[:, None]))[fin]).all()


def make(R, V, dtype, seed=0, scale=3.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn((R, V), device="cuda", generator=g) * scale).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("R,V,n,k", [(1, 1, 1, 1), (1, 2, 1, 2), (3, 31, 2, 31), (5, 33, 0, 32), (2, 1000, 3, 5), (1, 4096, 1, 0),
                                     (1, 128256, 1, 20), (7, 50257, 4, 32), (64, 32001, 1, 1), (700, 5003, 256, 7), (1300, 129, 1, 9)])
def test_values(river, R, V, n, k, dtype):
    x = make(R, V, dtype, seed=R + V)
    tok = torch.randint(0, V, (R, n), dtype=torch.int32, device="cuda") if n else None
    got = river.token_logprobs(x, tok, top_k=k)
    assert set(got) == {"lse", "entropy"} | ({"logprob"} if n else set()) | ({"top_ids", "top_logprobs"} if k else set())
    check(x, tok, k, got)


@pytest.mark.parametrize("R", [1, 20, 400])
@pytest.mark.parametrize("order", ["ascending", "descending", "constant", "two values"])
def test_orders_that_defeat_a_running_threshold(river, R, order):
    V = 40009
    if order == "constant":
        x = torch.full((R, V), 0.25, device="cuda")
    elif order == "two values":
        x = (torch.arange(V, device="cuda") % 3 == 0).float().repeat(R, 1)
    else:
        x = torch.linspace(-8, 8, V, device="cuda").repeat(R, 1)
        if order == "descending":
            x = x.flip(1).contiguous()
    check(x, None, 32, river.token_logprobs(x, top_k=32))


def test_masked_ids_and_extremes(river):
    x = make(6, 3001, torch.float32, seed=5)
    x[0, :3000] = float("-inf")           # one id left
    x[1] = -torch.finfo(torch.float32).max  # the lowest value everywhere: uniform
    x[2, ::2] = -torch.finfo(torch.float32).max
    x[3, 7] = 3e38                          # one huge logit
    x[4, 100:] = float("-inf")
    x[5] = -0.0
    x[5, ::7] = 0.0                         # -0 equals +0: ids in order
    tok = torch.tensor([[3000, 5], [1, 2], [1, 2], [7, 8], [99, 100], [0, 3000]], dtype=torch.int32, device="cuda")
    got = river.token_logprobs(x, tok, top_k=32)
    check(x, tok, 32, got)
    assert float(got["entropy"][0]) == 0.0 and float(got["logprob"][0, 0]) == 0.0
    assert float(got["logprob"][0, 1]) == float("-inf")
    assert got["top_ids"][5].tolist() == list(range(32))


def test_rows_without_a_distribution(river):
    x = make(4, 777, torch.float32, seed=6)
    x[0] = float("-inf")
    x[1, 5] = float("nan")
    x[2, 9] = float("inf")
    tok = torch.full((4,), 3, dtype=torch.int32, device="cuda")
    got = river.token_logprobs(x, tok, top_k=3)
    assert float(got["lse"][0]) == float("-inf") and torch.isnan(got["entropy"][0]) and torch.isnan(got["logprob"][0])
    assert got["top_ids"][0].tolist() == [0, 1, 2]
    for r in (1, 2):
        assert torch.isnan(got["lse"][r]) and torch.isnan(got["entropy"][r]) and torch.isnan(got["logprob"][r])
    assert int(got["top_ids"][1, 0]) == 5 and int(got["top_ids"][2, 0]) == 9
    check(x[3:], tok[3:], 3, {k: v[3:] for k, v in got.items()})


def test_token_ids_outside_the_vocabulary(river):
    x = make(3, 100, torch.bfloat16, seed=7)
    tok = torch.tensor([[5, -1], [100, 6], [7, 8]], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = river.token_logprobs(x, tok, err=err)
    assert int(err) == river.RL_DEVERR_TOKEN
    assert torch.isnan(got["logprob"]).tolist() == [[False, True], [True, False], [False, False]]
    err.zero_()
    river.token_logprobs(x, tok.clamp(0, 99), err=err)
    assert int(err) == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_rows_and_odd_starts(river, dtype):
    big = make(9, 2011, dtype, seed=8)
    flat = big.view(-1)
    for off, V in ((0, 1999), (1, 2000), (3, 517), (5, 64), (7, 9)):
        x = torch.as_strided(flat, (8, V), (2011, 1), off)
        check(x, None, min(V, 5), river.token_logprobs(x, top_k=min(V, 5)))


def test_stream_capture_and_repeat(river):
    x = make(3, 128256, torch.float32, seed=9)
    tok = torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda")
    want = river.token_logprobs(x, tok, top_k=8)
    again = river.token_logprobs(x, tok, top_k=8)
    assert all(torch.equal(want[k], again[k]) for k in want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = river.token_logprobs(x, tok, top_k=8, stream=s)
    s.synchronize()
    assert all(torch.equal(want[k], other[k]) for k in want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = river.token_logprobs(x, tok, top_k=8)
    x.copy_(make(3, 128256, torch.float32, seed=10))
    g.replay()
    torch.cuda.synchronize()
    check(x, tok, 8, got)


def test_given_buffers_and_their_refusal(river):
    x = make(2, 64, torch.float32)
    o = {"lse": torch.full((2,), 9.0, device="cuda")}
    got = river.token_logprobs(x, out=o)
    assert got["lse"] is o["lse"] and set(o) == {"lse"}
    check(x, None, 0, got)
    with pytest.raises(river.RiverError):
        river.token_logprobs(x, out={"lse": torch.zeros(3, device="cuda")})
    with pytest.raises(river.RiverError):
        river.token_logprobs(x, top_k=33)
    with pytest.raises(river.RiverError):
        river.token_logprobs(x, torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(river.RiverError) as e:
        river.token_logprobs(x.requires_grad_())
    assert e.value.status == river.RL_ERR_UNSUPPORTED
