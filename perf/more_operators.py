"""A serving loop's operators beside the decode path, measured: the paged cache
held in 4 bits (rows appended with the position rotation and read back,
attention over its pages), causal attention over packed prompts, and sampling
from given random numbers.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits, sampling's weights in 64) or, where ``own`` is true, through the
framework's entry points.

The cache: a page holds `page` token rows of every KV head, a row of head_dim
values is one group with a step s and a minimum m of the cache's 16-bit type and
a code c in 0 .. 15 for each value, which stands for m + s c.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one decode step of a batch: its rows rotated and appended (latency counts)
        {"name": "cache-step-32", "op": "cache", "batch": 32, "new_lo": 1, "new_hi": 1, "old_lo": 7, "old_hi": 4095, "page": 16,
         "heads": 32, "kv_heads": 8, "dim": 64, "dtype": "bf16"},
        # prompts of different lengths behind what their sequences hold already
        {"name": "cache-prompts", "op": "cache", "batch": 7, "new_lo": 33, "new_hi": 2301, "old_lo": 0, "old_hi": 1001, "page": 64,
         "heads": 32, "kv_heads": 8, "dim": 128, "dtype": "bf16"},
        # one sequence's step (latency counts)
        {"name": "kv4-step-1", "op": "kv4", "batch": 1, "q_lo": 1, "q_hi": 1, "len_lo": 1001, "len_hi": 1001, "page": 16,
         "heads": 32, "kv_heads": 8, "dim": 64, "dtype": "bf16"},
        # a full decode batch with ragged contexts
        {"name": "kv4-step-64", "op": "kv4", "batch": 64, "q_lo": 1, "q_hi": 1, "len_lo": 130, "len_hi": 8191, "page": 64,
         "heads": 32, "kv_heads": 8, "dim": 128, "dtype": "bf16"},
        # verifying a few drafted tokens a sequence, in fp16
        {"name": "kv4-draft-8", "op": "kv4", "batch": 8, "q_lo": 2, "q_hi": 5, "len_lo": 901, "len_hi": 6007, "page": 32,
         "heads": 32, "kv_heads": 8, "dim": 128, "dtype": "fp16"},
        # one long document
        {"name": "kv4-long-2", "op": "kv4", "batch": 2, "q_lo": 1, "q_hi": 1, "len_lo": 99999, "len_hi": 131072, "page": 128,
         "heads": 32, "kv_heads": 8, "dim": 128, "dtype": "bf16"},
        # many short prompts in fp16, one of a single token (latency counts)
        {"name": "packed-short-17", "op": "packed", "batch": 17, "len_lo": 1, "len_hi": 97, "heads": 32, "kv_heads": 8, "dim": 64,
         "dtype": "fp16"},
        # a batch of ordinary prompts
        {"name": "packed-ragged-12", "op": "packed", "batch": 12, "len_lo": 37, "len_hi": 2999, "heads": 32, "kv_heads": 8, "dim": 128,
         "dtype": "bf16"},
        # two long ones
        {"name": "packed-long-2", "op": "packed", "batch": 2, "len_lo": 5001, "len_hi": 8192, "heads": 32, "kv_heads": 8, "dim": 128,
         "dtype": "bf16"},
        # one decode step of one sequence, the usual filters (latency counts)
        {"name": "sample-step-1", "op": "sample", "rows": 1, "vocab": 128256, "dtype": "fp32", "temperature": 0.8, "top_k": 50,
         "top_p": 0.95, "min_p": 0.0, "each": False},
        # a decode batch, cut by probability mass alone
        {"name": "sample-step-64", "op": "sample", "rows": 64, "vocab": 128256, "dtype": "fp32", "temperature": 1.0, "top_k": 0,
         "top_p": 0.9, "min_p": 0.0, "each": False},
        # many samples in bf16 over an odd vocabulary, every row with settings of its own (some greedy, some unfiltered)
        {"name": "sample-each-500", "op": "sample", "rows": 500, "vocab": 50257, "dtype": "bf16", "temperature": 0.9, "top_k": 40,
         "top_p": 0.9, "min_p": 0.02, "each": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["cache", "kv4", "kv4", "packed", "sample"])
    if op == "sample":
        vocab = rng.choice([128256, _log_int(rng, 1000, 160000)])
        return {"op": op, "rows": _log_int(rng, 1, min(1000, 25_000_000 // vocab)), "vocab": vocab, "dtype": rng.choice(["fp32", "bf16", "fp16"]),
                "temperature": rng.choice([0.0, 1.0, round(rng.uniform(0.3, 2.0), 3)]), "top_k": rng.choice([0, 0, 1, 50, _log_int(rng, 2, 5000)]),
                "top_p": rng.choice([1.0, 0.95, round(rng.uniform(0.05, 0.999), 4)]), "min_p": rng.choice([0.0, 0.0, 0.05, round(rng.uniform(0.001, 0.3), 4)]),
                "each": rng.random() < 0.4}
    dim, dtype = rng.choice([64, 128]), rng.choice(["bf16", "fp16"])
    kv_heads = rng.choice([1, 2, 4, 8])
    case = {"op": op, "heads": min(32, kv_heads * rng.choice([1, 2, 3, 4, 8])), "kv_heads": kv_heads, "dim": dim, "dtype": dtype}
    if op == "packed":
        hi = _log_int(rng, 1, 8192)
        batch = _log_int(rng, 1, max(1, min(64, 8192 * 8192 // (hi * hi), 18_000 // hi)))
        return {**case, "batch": batch, "len_lo": rng.randint(1, hi), "len_hi": hi}
    case["page"] = rng.choice([16, 32, 64, 128])
    if op == "cache":
        hi = rng.choice([1, _log_int(rng, 1, 4000)])
        batch = _log_int(rng, 1, max(1, min(64, 8000 // hi)))
        old = _log_int(rng, 1, 4000)
        return {**case, "batch": batch, "new_lo": rng.randint(0, hi), "new_hi": hi, "old_lo": rng.randint(0, old), "old_hi": old}
    batch, q_hi = _log_int(rng, 1, 64), rng.choice([1, 1, rng.randint(2, 16)])
    hi = _log_int(rng, q_hi, max(q_hi, 266_000 // batch // (2 if q_hi > 1 else 1)))
    hi = min(hi, 131072)
    return {**case, "batch": batch, "q_lo": rng.randint(1, q_hi), "q_hi": q_hi, "len_lo": rng.randint(min(q_hi, hi), hi), "len_hi": hi}


def _spread(lo, hi, n):
    """n whole numbers from lo to hi (the last one the largest)."""
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _sizes(case):
    """Rows of each sequence in the call, and its length with them."""
    B = case["batch"]
    if case["op"] == "packed":
        n = _spread(case["len_lo"], case["len_hi"], B)
        return n, n
    if case["op"] == "cache":
        new, old = _spread(case["new_lo"], case["new_hi"], B), _spread(case["old_lo"], case["old_hi"], B)[::-1]
        return new, [a + b for a, b in zip(new, old)]
    return _spread(case["q_lo"], case["q_hi"], B), _spread(case["len_lo"], case["len_hi"], B)


def _rope(n, dim):
    """(cos, sin) of position x frequency, the angles in 64 bits: [n][dim / 2][2]."""
    f = 500000.0 ** (-2.0 * torch.arange(dim // 2, dtype=torch.float64, device="cuda") / dim)
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.stack([a.cos(), a.sin()], dim=-1).float()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, dtype, scale=1.0):
        t = torch.empty(shape, dtype=torch.float32, device="cuda")
        t.normal_(0.0, scale, generator=g)
        return t.to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.empty(shape, dtype=torch.float32, device="cuda").uniform_(lo, hi, generator=g)

    dt = _DT[case["dtype"]]
    state = {"case": dict(case)}
    if case["op"] == "sample":
        R, V = case["rows"], case["vocab"]
        logits = torch.empty((R, V), dtype=torch.float32, device="cuda").normal_(0.0, 2.0, generator=g)
        # a few likely continuations a row, and ids that no row may produce
        likely = torch.randint(0, V, (R, 8), device="cuda", generator=g)
        logits.scatter_add_(1, likely, uniform(R, 8, lo=4.0, hi=14.0))
        logits[:, : max(1, V // 1000)] = float("-inf")
        state["logits"] = logits.to(dt)
        state["u"] = torch.rand(R, device="cuda", generator=g)
        set_ = {k: case[k] for k in ("temperature", "top_k", "top_p", "min_p")}
        if case["each"]:  # requests of different users in one batch
            def some(p, a, b):
                return torch.where(torch.rand(R, device="cuda", generator=g) < p, a, b)
            set_["temperature"] = some(0.15, torch.zeros(R, device="cuda"), uniform(R, lo=0.3, hi=1.5))
            set_["top_k"] = some(0.4, torch.zeros(R, dtype=torch.int32, device="cuda"),
                                 torch.randint(1, max(2, 2 * case["top_k"] + 2), (R,), device="cuda", generator=g).to(torch.int32))
            set_["top_p"] = some(0.4, torch.ones(R, device="cuda"), uniform(R, lo=0.3, hi=1.0))
            set_["min_p"] = some(0.5, torch.zeros(R, device="cuda"), uniform(R, lo=0.0, hi=2 * case["min_p"] + 0.01))
        state["settings"] = set_
        return state
    B, Hq, Hkv, D = case["batch"], case["heads"], case["kv_heads"], case["dim"]
    new, lens = _sizes(case)
    order = torch.randperm(B, device="cuda", generator=g)
    rows = torch.tensor(new, dtype=torch.int64, device="cuda")[order]
    N = sum(new)
    state["start"] = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), rows.cumsum(0)]).to(torch.int32)
    state["max_rows"] = max(new)
    if case["op"] in ("cache", "packed"):
        # one projection's output: queries, keys and values of every row side by side
        state["qkv"] = normal(max(N, 1), Hq + 2 * Hkv, D, dtype=dt)
        if case["op"] == "packed":
            state["qkv"][:, :Hq] *= 1.5
            return state
        # a few channels of the keys are larger, as models' keys have them
        state["qkv"][:, Hq:Hq + Hkv, ::17] *= 4.0
        state["rope"] = _rope(max(lens) + 1, D)
    else:
        state["q"] = normal(max(N, 1), Hq, D, dtype=dt, scale=1.5)
    page = case["page"]
    state["kv_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")[order].contiguous()
    width = max(1, (max(lens) + page - 1) // page)
    pages = [(n + page - 1) // page for n in lens]
    n_pages = sum(pages) + 3
    free = torch.randperm(n_pages, device="cuda", generator=g).to(torch.int32)
    first = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), torch.tensor(pages, device="cuda")[order].cumsum(0)])
    at = first[:-1, None] + torch.arange(width, device="cuda")
    # (entries behind a sequence's last page name some page of another)
    state["table"] = free[at.clamp(max=n_pages - 1)].contiguous()
    for x in ("k", "v"):
        state[x + "_codes"] = torch.randint(0, 256, (n_pages, Hkv, page, D // 2), dtype=torch.uint8, device="cuda", generator=g)
        s = uniform(n_pages, Hkv, page, lo=0.1, hi=0.5)
        state[x + "_scale"] = torch.stack([s, -7.5 * s + normal(n_pages, Hkv, page, dtype=torch.float32, scale=0.2)], dim=-1).to(dt)
    state["cache"] = tuple(state[x + y] for x in ("k", "v") for y in ("_codes", "_scale"))
    return state


def _row_places(start, kv_len, n_rows):
    """Sequence and position of every packed row."""
    r = torch.arange(n_rows, device=start.device)
    b = torch.searchsorted(start[1:].long(), r, right=True).clamp(max=kv_len.numel() - 1)
    return b, kv_len.long()[b] - start.long()[b + 1] + r


def _quantize(x, dt):
    """Rows of 16-bit values [..., D] -> codes, (step, minimum) of the same type."""
    f = x.float()
    lo, hi = f.amin(dim=-1, keepdim=True), f.amax(dim=-1, keepdim=True)
    s = ((hi - lo) / 15.0).to(dt).float()
    s = torch.where(s < 2.0 ** -100, 0.0, s)
    c = torch.round(torch.where(s > 0, (f - lo) / torch.where(s > 0, s, 1.0), 0.0)).clamp(0, 15).to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4), torch.cat([s, lo], dim=-1).to(dt)


def _values(codes, scale):
    """What codes [..., D / 2] with (step, minimum) [..., 2] stand for, in 32 bits."""
    c = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).float()
    return scale[..., 1:].float() + scale[..., :1].float() * c


def _plain_cache(q, k, v, rope, start, kv_len, table, page, cache):
    b, pos = _row_places(start, kv_len, q.shape[0])
    cos, sin = rope[pos, None, :, 0], rope[pos, None, :, 1]

    def rotate(x):
        a, c = x.float().chunk(2, dim=-1)
        return torch.cat([a * cos - c * sin, c * cos + a * sin], dim=-1).to(x.dtype)

    at, row = table[b, pos // page].long(), pos % page
    out = {"q": rotate(q)}
    for name, x, codes, scale in (("k", rotate(k), *cache[:2]), ("v", v, *cache[2:])):
        codes[at, :, row], scale[at, :, row] = _quantize(x, x.dtype)
        out[name] = _values(codes[at, :, row], scale[at, :, row]).to(x.dtype)
    return out


def _plain_attention(q, k, v, visible):
    """q [..., R, D], k and v [..., S, D], visible [..., R, S] -> (outputs, ln of the weights' sums), in 32 bits."""
    s = torch.matmul(q.float(), k.float().transpose(-1, -2)) * (1.0 / math.sqrt(q.shape[-1]))
    s = s.masked_fill(~visible, float("-inf"))
    m = s.amax(dim=-1, keepdim=True)
    m = torch.where(torch.isinf(m), 0.0, m)
    e = torch.exp(s - m)
    del s
    l = e.sum(dim=-1, keepdim=True)
    return torch.matmul(e, v.float()) / torch.where(l > 0, l, 1.0), (m + torch.log(l))[..., 0]


def _padded(x, start, width):
    """Packed rows [N, H, D] -> [B, width, H, D] (rows behind a sequence's last: some other row)."""
    at = start[:-1, None].long() + torch.arange(width, device=x.device)
    return x[at.clamp(max=x.shape[0] - 1)]


def _plain_rows(q, start, width, Hkv, pos, k, v):
    """Packed queries at positions `pos` [B, width] of k, v [B, Hkv, S, D]."""
    N, Hq, D = q.shape
    B, rep = start.numel() - 1, Hq // Hkv
    qq = _padded(q, start, width).view(B, width, Hkv, rep, D).permute(0, 2, 3, 1, 4)
    vis = torch.arange(k.shape[2], device=q.device) <= pos[..., None]
    o, lse = _plain_attention(qq, k[:, :, None], v[:, :, None], vis[:, None, None])
    o, lse = o.permute(0, 3, 1, 2, 4).reshape(B, width, Hq, D), lse.permute(0, 3, 1, 2).reshape(B, width, Hq)
    live = torch.arange(width, device=q.device) < (start[1:] - start[:-1])[:, None]
    return {"out": o[live].to(q.dtype), "lse": lse[live]}


def _plain_kv4(q, cache, table, kv_len, start, width):
    def gathered(c, s):  # [B, pages, Hkv, page, D] -> [B, Hkv, tokens, D]
        return _values(c[table.long()], s[table.long()]).transpose(1, 2).flatten(2, 3)

    k, v = gathered(*cache[:2]), gathered(*cache[2:])
    v = v.masked_fill((torch.arange(v.shape[2], device=v.device) >= kv_len[:, None])[:, None, :, None], 0.0)
    rows = (start[1:] - start[:-1])[:, None]
    pos = kv_len[:, None] - rows + torch.arange(width, device=q.device)
    return _plain_rows(q, start, width, k.shape[1], pos, k, v)


def _plain_packed(q, k, v, start, width):
    kk, vv = _padded(k, start, width).transpose(1, 2), _padded(v, start, width).transpose(1, 2)
    pos = torch.arange(width, device=q.device).expand(start.numel() - 1, width)
    return _plain_rows(q, start, width, k.shape[1], pos, kk, vv)


def _plain_sample(logits, u, temperature, top_k, top_p, min_p):
    R, V = logits.shape

    def column(x, dt):  # (a setting as the call takes it: one value a row, or one for all)
        return x[:, None] if isinstance(x, torch.Tensor) else torch.full((R, 1), x, dtype=dt, device=logits.device)

    T, p, mp = (column(x, torch.float32).to(torch.float64) for x in (temperature, top_p, min_p))
    k = column(top_k, torch.int32)
    x = logits.to(torch.float64)
    greedy = T <= 0
    m = x.amax(dim=1, keepdim=True)
    w = torch.exp((x - m) / torch.where(greedy, 1.0, T))
    ids = torch.sort(x, dim=1, descending=True, stable=True).indices
    ws = w.gather(1, ids)
    rank = torch.arange(V, device=x.device)
    keep = (rank < torch.where(k > 0, k, V)) & (rank < torch.where(greedy, 1, V))
    before = torch.where(keep, ws, 0.0).cumsum(1) - torch.where(keep, ws, 0.0)
    total = torch.where(keep, ws, 0.0).sum(dim=1, keepdim=True)
    keep = keep & ((rank == 0) | (p >= 1.0) | (before < p * total)) & ((rank == 0) | (ws >= mp))
    w = torch.where(torch.zeros_like(keep).scatter_(1, ids, keep), w, 0.0)
    cum = w.cumsum(1)
    token = (cum <= u.to(torch.float64)[:, None] * cum[:, -1:]).sum(dim=1)
    return {"token": token.to(torch.int32), "logprob": torch.log(w.gather(1, token[:, None]) / w.sum(dim=1, keepdim=True))[:, 0].float()}


def run(state):
    c = state["case"]
    if c["op"] == "sample":
        if own:
            import early_exit_decoding_gb300 as river
            return river.sample(state["logits"], state["u"], **state["settings"])
        return _plain_sample(state["logits"], state["u"], **state["settings"])
    start, width, Hq, Hkv = state["start"], state["max_rows"], c["heads"], c["kv_heads"]
    if c["op"] == "kv4":
        if own:
            import early_exit_decoding_gb300 as river
            return river.kv4_attention(state["q"], state["cache"], state["table"], state["kv_len"], start=start, max_rows=width)
        return _plain_kv4(state["q"], state["cache"], state["table"], state["kv_len"], start, width)
    q, k, v = state["qkv"].split((Hq, Hkv, Hkv), dim=1)
    if c["op"] == "packed":
        if own:
            import early_exit_decoding_gb300 as river
            return river.packed_attention(q, k, v, start, max_rows=width)
        return _plain_packed(q, k, v, start, width)
    if own:
        import early_exit_decoding_gb300 as river
        o = river.kv4_append(state["cache"], state["table"], state["kv_len"], k, v, q=q, rope=state["rope"], start=start)
        return {**o, **river.kv4_read(state["cache"], state["table"], state["kv_len"], start=start, rows=q.shape[0])}
    return _plain_cache(q, k, v, state["rope"], start, state["kv_len"], state["table"], c["page"], state["cache"])


def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "sample":
        R, V = case["rows"], case["vocab"]
        # maximum, difference, exponential, sum and a comparison a logit
        return {"bytes": R * V * size + R * (16 if case["each"] else 0) + R * 12, "flops": 5 * R * V}
    Hq, Hkv, D = case["heads"], case["kv_heads"], case["dim"]
    new, lens = _sizes(case)
    N = sum(new)
    if case["op"] == "cache":
        held = 2 * N * Hkv * (D // 2 + 2 * size)
        # rows in, queries out, the cache's rows written and read, their values out, a row of angles each
        return {"bytes": (2 * Hq + 4 * Hkv) * N * D * size + 2 * held + N * D * 4, "flops": N * (6 * (Hq + Hkv) + 8 * Hkv) * D}
    if case["op"] == "packed":
        return {"bytes": 2 * (Hq + Hkv) * N * D * size + N * Hq * 4, "flops": sum(2 * D * Hq * n * (n + 1) for n in new)}
    pairs = sum(sum(range(n - r + 1, n + 1)) for r, n in zip(new, lens))
    return {"bytes": 2 * sum(lens) * Hkv * (D // 2 + 2 * size) + N * Hq * (2 * D * size + 4) + 8 * len(lens)
            + 4 * sum((n + case["page"] - 1) // case["page"] for n in lens), "flops": 4 * D * Hq * pairs}


def exact(case, seed):
    state = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "sample":
        tokens, lps = [], []
        st = {k: (x.tolist() if isinstance(x, torch.Tensor) else [float(torch.tensor(x, dtype=torch.float32))] * case["rows"])
              for k, x in state["settings"].items()}
        u = state["u"].tolist()
        for r in range(case["rows"]):
            x = state["logits"][r].to(f64)
            if st["temperature"][r] <= 0:
                tokens.append(int((x == x.max()).nonzero()[0, 0]))
                lps.append(0.0)
                continue
            z = x / st["temperature"][r]
            order = torch.argsort(z, descending=True, stable=True)
            if st["top_k"][r] > 0:
                order = order[: int(st["top_k"][r])]
            p = torch.softmax(z[order], dim=0)
            n = order.numel()
            if st["top_p"][r] < 1.0:
                n = max(1, int(torch.searchsorted(p.cumsum(0), st["top_p"][r])) + 1)
            n = max(1, min(n, int((p >= st["min_p"][r] * p[0]).sum())))
            ids = order[:n].sort().values
            p = torch.softmax(z[ids], dim=0)
            i = min(int(torch.searchsorted(p.cumsum(0), u[r], right=True)), n - 1)
            tokens.append(int(ids[i]))
            lps.append(float(p[i].log()))
        return {"token": torch.tensor(tokens, dtype=torch.int32, device="cuda"), "logprob": torch.tensor(lps, dtype=f64, device="cuda")}
    Hq, Hkv, D, B = case["heads"], case["kv_heads"], case["dim"], case["batch"]
    rep, st = Hq // Hkv, state["start"].tolist()
    N = st[-1]
    if case["op"] == "cache":
        lens, page = state["kv_len"].tolist(), case["page"]
        x = state["qkv"].to(f64)
        seq = [b for b in range(B) for _ in range(st[b + 1] - st[b])]
        pos = torch.tensor([lens[seq[r]] - st[seq[r] + 1] + r for r in range(N)], device="cuda", dtype=torch.int64)
        half = D // 2
        z = torch.complex(x[..., :half], x[..., half:])
        turn = torch.view_as_complex(state["rope"].to(f64))[pos]
        z = z * turn[:, None]
        rot = torch.cat([z.real, z.imag], dim=-1)
        # the codes go by the keys as a 16-bit cache would hold them
        k16 = rot[:, Hq:Hq + Hkv].to(_DT[case["dtype"]]).to(f64)

        def held(y):
            lo, hi = y.min(dim=-1, keepdim=True).values, y.max(dim=-1, keepdim=True).values
            s = ((hi - lo) / 15).to(_DT[case["dtype"]]).to(f64)
            return lo + s * ((y - lo) / s.clamp(min=2.0 ** -100)).round().clamp(0, 15)
        return {"q": rot[:, :Hq], "k": held(k16), "v": held(x[:, Hq + Hkv:])}
    out = torch.zeros((N, Hq, D), dtype=f64, device="cuda")
    lse = torch.zeros((N, Hq), dtype=f64, device="cuda")
    lens = st if case["op"] == "packed" else state["kv_len"].tolist()
    for b in range(B):
        r0, r1 = st[b], st[b + 1]
        for h in range(Hkv):
            if case["op"] == "packed":
                n = r1 - r0
                kb, vb = (state["qkv"][r0:r1, Hq + o + h].to(f64) for o in (0, Hkv))
                q = state["qkv"]
            else:
                n = lens[b]
                used = state["table"][b, : (n + case["page"] - 1) // case["page"]].long()

                def rows(c, s):
                    c, s = c[used, h].reshape(-1, D // 2)[:n].to(torch.int64), s[used, h].reshape(-1, 2)[:n].to(f64)
                    return s[:, 1:] + s[:, :1] * torch.stack([c % 16, c // 16], dim=2).reshape(n, D)
                kb, vb = rows(state["k_codes"], state["k_scale"]), rows(state["v_codes"], state["v_scale"])
                q = state["q"]
            for lo in range(r0, r1, 1024):
                hi = min(r1, lo + 1024)
                qb = q[lo:hi, h * rep:(h + 1) * rep].to(f64).transpose(0, 1)
                last = n - r1 + torch.arange(lo, hi, device="cuda")
                end = n - r1 + hi
                sc = (qb @ kb[:end].T / math.sqrt(D)).masked_fill(torch.arange(end, device="cuda") > last[:, None], float("-inf"))
                z = torch.logsumexp(sc, dim=-1)
                out[lo:hi, h * rep:(h + 1) * rep] = (torch.exp(sc - z[..., None]) @ vb[:end]).transpose(0, 1)
                lse[lo:hi, h * rep:(h + 1) * rep] = z.transpose(0, 1)
    return {"out": out, "lse": lse}
