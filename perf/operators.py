"""The serving operators beside the decode path, measured: log-probabilities of
given tokens, sliding-window attention with sinks, and decode attention of a
batch over one shared prefix.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits) or, where ``own`` is true, through the framework's entry points.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one decode step of one sequence: fp32 logits as the step returns them, the sampled
        # token's log-probability and five alternatives (latency counts)
        {"name": "logprobs-step-1", "op": "logprobs", "rows": 1, "vocab": 128256, "dtype": "fp32", "n_tok": 1, "top_k": 5},
        # a decode batch asked for its sampled tokens and twenty alternatives
        {"name": "logprobs-step-64", "op": "logprobs", "rows": 64, "vocab": 128256, "dtype": "fp32", "n_tok": 1, "top_k": 20},
        # an odd vocabulary in bf16 (rows start off any 16-byte boundary), four candidate tokens a row
        {"name": "logprobs-odd-bf16", "op": "logprobs", "rows": 777, "vocab": 50257, "dtype": "bf16", "n_tok": 4, "top_k": 3},
        # scoring a prompt: every position's next token
        {"name": "logprobs-prompt", "op": "logprobs", "rows": 4096, "vocab": 128256, "dtype": "fp32", "n_tok": 1, "top_k": 1},
        # one sequence decoding past its window (latency counts)
        {"name": "window-step-1", "op": "window", "batch": 1, "q_cap": 1, "q_lo": 1, "len_lo": 3001, "len_hi": 3001, "capacity": 4096,
         "heads": 32, "kv_heads": 8, "dim": 64, "window": 1024, "sinks": 4, "dtype": "bf16"},
        # a full decode batch with ragged contexts, some still inside the window
        {"name": "window-step-64", "op": "window", "batch": 64, "q_cap": 1, "q_lo": 1, "len_lo": 130, "len_hi": 8191, "capacity": 8192,
         "heads": 32, "kv_heads": 8, "dim": 128, "window": 4096, "sinks": 4, "dtype": "bf16"},
        # verifying a few drafted tokens a sequence
        {"name": "window-draft-8", "op": "window", "batch": 8, "q_cap": 5, "q_lo": 2, "len_lo": 901, "len_hi": 6007, "capacity": 6144,
         "heads": 32, "kv_heads": 8, "dim": 128, "window": 2048, "sinks": 4, "dtype": "bf16"},
        # ragged prompts in fp16, the shortest with fewer cached rows than queries (rows that see nothing)
        {"name": "window-prompt-ragged", "op": "window", "batch": 5, "q_cap": 1003, "q_lo": 37, "len_lo": 30, "len_hi": 1401, "capacity": 1408,
         "heads": 32, "kv_heads": 8, "dim": 64, "window": 500, "sinks": 16, "dtype": "fp16"},
        # a long prompt in one call
        {"name": "window-prompt-8192", "op": "window", "batch": 1, "q_cap": 8192, "q_lo": 8192, "len_lo": 8192, "len_hi": 8192, "capacity": 8192,
         "heads": 32, "kv_heads": 8, "dim": 128, "window": 2048, "sinks": 4, "dtype": "bf16"},
        # a few continuations of one prompt, just begun
        {"name": "prefix-step-4", "op": "prefix", "batch": 4, "prefix": 1001, "len_lo": 0, "len_hi": 33, "capacity": 64,
         "heads": 32, "kv_heads": 8, "dim": 64, "dtype": "bf16"},
        # a decode batch behind one long instruction
        {"name": "prefix-step-64", "op": "prefix", "batch": 64, "prefix": 8192, "len_lo": 1, "len_hi": 257, "capacity": 288,
         "heads": 32, "kv_heads": 8, "dim": 128, "dtype": "bf16"},
        # many samples of one long document with long answers
        {"name": "prefix-step-256", "op": "prefix", "batch": 256, "prefix": 32768, "len_lo": 5, "len_hi": 1999, "capacity": 2000,
         "heads": 32, "kv_heads": 8, "dim": 128, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["logprobs", "window", "window", "prefix"])
    if op == "logprobs":
        vocab = rng.choice([128256, _log_int(rng, 1000, 160000)])
        rows = _log_int(rng, 1, min(4096, 500_000_000 // vocab))
        return {"op": op, "rows": rows, "vocab": vocab, "dtype": rng.choice(["fp32", "bf16", "fp16"]),
                "n_tok": rng.randint(0, 5), "top_k": rng.randint(0, 32)}
    dim, dtype = rng.choice([64, 128]), rng.choice(["bf16", "fp16"])
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 8])
    if op == "prefix":
        batch = _log_int(rng, 1, 256)
        hi = _log_int(rng, 1, 2000)
        return {"op": op, "batch": batch, "prefix": _log_int(rng, 1, 32768), "len_lo": rng.randint(0, hi), "len_hi": hi,
                "capacity": hi + rng.randint(0, 100), "heads": min(heads, 32), "kv_heads": min(kv_heads, 8) if heads <= 32 else 4,
                "dim": dim, "dtype": dtype}
    kind = rng.choice(["step", "draft", "prompt"])
    window, sinks = _log_int(rng, 16, 8192), rng.choice([0, 1, 4, 17, 150])
    if heads > 32:
        kv_heads, heads = 4, 32
    if kind == "step":
        batch, q_cap, hi = _log_int(rng, 1, 64), 1, _log_int(rng, 1, 8192)
    elif kind == "draft":
        batch, q_cap, hi = _log_int(rng, 1, 64), rng.randint(2, 16), _log_int(rng, 16, 8192)
    else:
        q_cap = _log_int(rng, 17, 8192)
        hi = min(8192, q_cap + rng.choice([0, _log_int(rng, 1, 4096)]))
        batch = _log_int(rng, 1, max(1, min(16, (8192 * 8192) // (q_cap * hi) // 2)))
    return {"op": op, "batch": batch, "q_cap": q_cap, "q_lo": rng.randint(1, q_cap), "len_lo": rng.randint(0, hi), "len_hi": hi,
            "capacity": hi + rng.randint(0, 200), "heads": heads, "kv_heads": kv_heads, "dim": dim, "window": window, "sinks": sinks,
            "dtype": dtype}


def _spread(lo, hi, n):
    """n whole numbers from lo to hi: the sequences' lengths (the last one the longest)."""
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _lengths(case):
    lens = _spread(case["len_lo"], case["len_hi"], case["batch"])
    return (lens, _spread(case["q_lo"], case["q_cap"], case["batch"])) if case["op"] == "window" else (lens, None)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, dtype, scale=1.0):
        t = torch.empty(shape, dtype=torch.float32, device="cuda")
        t.normal_(0.0, scale, generator=g)
        return t.to(dtype)

    dt = _DT[case["dtype"]]
    state = {"case": dict(case)}
    if case["op"] == "logprobs":
        R, V = case["rows"], case["vocab"]
        logits = torch.empty((R, V), dtype=torch.float32, device="cuda").normal_(0.0, 2.0, generator=g)
        # a few likely continuations a row, and ids that no row may produce
        likely = torch.randint(0, V, (R, 8), device="cuda", generator=g)
        logits.scatter_add_(1, likely, torch.empty((R, 8), device="cuda").uniform_(4.0, 14.0, generator=g))
        logits[:, : max(1, V // 1000)] = float("-inf")
        state["logits"] = logits.to(dt)
        if case["n_tok"]:
            other = torch.randint(V // 1000 + 1, V, (R, case["n_tok"]), device="cuda", generator=g)
            pick = torch.rand((R, case["n_tok"]), device="cuda", generator=g) < 0.6
            mine = likely[:, torch.arange(case["n_tok"], device="cuda") % 8].clamp(min=V // 1000 + 1)
            state["tokens"] = torch.where(pick, mine, other).to(torch.int32)
        return state
    B, Hq, Hkv, D = case["batch"], case["heads"], case["kv_heads"], case["dim"]
    lens, qlens = _lengths(case)
    order = torch.randperm(B, device="cuda", generator=g)
    state["kv_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")[order].contiguous()
    state["k"] = normal(B, Hkv, case["capacity"], D, dtype=dt)
    state["v"] = normal(B, Hkv, case["capacity"], D, dtype=dt)
    if case["op"] == "window":
        state["q"] = normal(B, case["q_cap"], Hq, D, dtype=dt, scale=1.5)
        state["q_len"] = torch.tensor(qlens, dtype=torch.int32, device="cuda")[order].contiguous()
        # rows behind a sequence's last query stay as the caller left them
        state["out"] = {"out": torch.zeros_like(state["q"]),
                        "lse": torch.zeros((B, case["q_cap"], Hq), dtype=torch.float32, device="cuda")}
    else:
        state["q"] = normal(B, Hq, D, dtype=dt, scale=1.5)
        state["k_prefix"] = normal(Hkv, case["prefix"], D, dtype=dt)
        state["v_prefix"] = normal(Hkv, case["prefix"], D, dtype=dt)
    return state


def _ordered_keys(x):
    """64-bit keys that order fp32 values, equal ones by the lower index first."""
    i = (x + 0.0).view(torch.int32)
    o = (i ^ ((i >> 31) & 0x7FFFFFFF)).to(torch.int64)
    idx = torch.arange(x.shape[1], device=x.device, dtype=torch.int64)
    return o * (1 << 32) + ((1 << 32) - 1 - idx)


def _plain_logprobs(logits, tokens, top_k):
    x = logits.float()
    m = x.amax(dim=1, keepdim=True)
    e = torch.exp(x - m)
    s = e.sum(dim=1, keepdim=True)
    lse = m + torch.log(s)
    out = {"lse": lse[:, 0]}
    d = torch.where(e > 0, x - m, 0.0)
    out["entropy"] = (torch.log(s) - (d * e).sum(dim=1, keepdim=True) / s)[:, 0]
    if tokens is not None:
        out["logprob"] = x.gather(1, tokens.long()) - lse
    if top_k:
        key = _ordered_keys(x).topk(top_k, dim=1).values
        ids = (1 << 32) - 1 - (key & 0xFFFFFFFF)
        out["top_ids"] = ids.to(torch.int32)
        out["top_logprobs"] = x.gather(1, ids) - lse
    return out


def _plain_attention(q, k, v, visible):
    """q [..., R, D], k and v [..., S, D], visible [..., R, S] -> (weighted sums, row maxima, row sums), in 32 bits."""
    s = torch.matmul(q.float(), k.float().transpose(-1, -2)) * (1.0 / math.sqrt(q.shape[-1]))
    s = s.masked_fill(~visible, float("-inf"))
    m = s.amax(dim=-1, keepdim=True)
    e = torch.exp(s - torch.where(torch.isinf(m), 0.0, m))
    return torch.matmul(e, v.float()), m, e.sum(dim=-1, keepdim=True)


def _plain_window(q, k, v, kv_len, q_len, window, sinks, out):
    B, T, Hq, D = q.shape
    Hkv, S = k.shape[1], k.shape[2]
    rep = Hq // Hkv
    t = torch.arange(T, device=q.device)
    j = torch.arange(S, device=q.device)
    p = (kv_len - q_len)[:, None] + t[None, :]
    vis = (j <= p[..., None]) & ((p[..., None] - j < window) | (j < sinks))  # [B, T, S]
    qq = q.view(B, T, Hkv, rep, D).permute(0, 2, 3, 1, 4)  # [B, Hkv, rep, T, D]
    o, m, l = _plain_attention(qq, k[:, :, None], v[:, :, None], vis[:, None, None])
    o = torch.where(l > 0, o / torch.where(l > 0, l, 1.0), 0.0)
    lse = torch.where(l > 0, m + torch.log(l), float("-inf"))
    o = o.permute(0, 3, 1, 2, 4).reshape(B, T, Hq, D).to(q.dtype)
    lse = lse[..., 0].permute(0, 3, 1, 2).reshape(B, T, Hq)
    live = t[None, :] < q_len[:, None]
    return {"out": torch.where(live[..., None, None], o, out["out"]), "lse": torch.where(live[..., None], lse, out["lse"])}


def _plain_prefix(q, kp, vp, k, v, kv_len):
    B, Hq, D = q.shape
    Hkv, S = k.shape[1], k.shape[2]
    rep = Hq // Hkv
    qq = q.view(B, Hkv, rep, D)
    # the prefix once for all rows of a KV head, the sequences' own rows each
    qp = qq.permute(1, 0, 2, 3).reshape(Hkv, B * rep, D)
    o1, m1, l1 = _plain_attention(qp, kp, vp, torch.ones((1, 1, 1), dtype=torch.bool, device=q.device))
    o1, m1, l1 = (x.view(Hkv, B, rep, -1).permute(1, 0, 2, 3) for x in (o1, m1, l1))
    vis = torch.arange(S, device=q.device)[None, :] < kv_len[:, None]
    o2, m2, l2 = _plain_attention(qq, k, v, vis[:, None, None, :])
    m = torch.maximum(m1, m2)
    a1, a2 = torch.exp(m1 - m), torch.exp(m2 - m)
    l = a1 * l1 + a2 * l2
    o = (a1 * o1 + a2 * o2) / l
    return {"out": o.reshape(B, Hq, D).to(q.dtype), "lse": (m + torch.log(l)).reshape(B, Hq)}


def run(state):
    c = state["case"]
    if own:
        import early_exit_decoding_gb300 as river
        if c["op"] == "logprobs":
            return river.token_logprobs(state["logits"], state.get("tokens"), top_k=c["top_k"])
        if c["op"] == "window":
            return river.window_attention(state["q"], state["k"], state["v"], state["kv_len"], window=c["window"], sinks=c["sinks"],
                                          q_len=state["q_len"], out=state["out"])
        return river.shared_prefix_attention(state["q"], state["k_prefix"], state["v_prefix"], state["k"], state["v"], state["kv_len"])
    if c["op"] == "logprobs":
        return _plain_logprobs(state["logits"], state.get("tokens"), c["top_k"])
    if c["op"] == "window":
        return _plain_window(state["q"], state["k"], state["v"], state["kv_len"], state["q_len"], c["window"], c["sinks"], state["out"])
    return _plain_prefix(state["q"], state["k_prefix"], state["v_prefix"], state["k"], state["v"], state["kv_len"])


def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "logprobs":
        R, V = case["rows"], case["vocab"]
        # maximum, difference, exponential, two sums and a comparison a logit
        return {"bytes": R * V * size + R * case["n_tok"] * 8 + R * case["top_k"] * 8 + R * 8, "flops": 7 * R * V}
    Hq, Hkv, D = case["heads"], case["kv_heads"], case["dim"]
    lens, qlens = _lengths(case)
    if case["op"] == "prefix":
        B, P = case["batch"], case["prefix"]
        keys = Hkv * (P + sum(lens))
        return {"bytes": keys * D * 2 * size + B * Hq * (2 * D * size + 4) + 4 * B, "flops": 4 * D * Hq * (B * P + sum(lens))}
    pairs = keys = 0
    w, n_sink = case["window"], case["sinks"]
    for n, ql in zip(lens, qlens):
        p = np.arange(n - ql, n, dtype=np.int64)
        p = p[p >= 0]
        pairs += int(np.minimum(p + 1, w + np.minimum(n_sink, np.maximum(p + 1 - w, 0))).sum())
        if p.size:
            first = max(0, int(p[0]) - w + 1)
            keys += n - first + min(first, n_sink)
    rows = sum(qlens) * Hq
    return {"bytes": Hkv * keys * D * 2 * size + rows * (2 * D * size + 4) + 8 * len(lens), "flops": 4 * D * Hq * pairs}


def exact(case, seed):
    state = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "logprobs":
        cols = {"lse": [], "entropy": [], "logprob": [], "top_ids": [], "top_logprobs": []}
        for lo in range(0, case["rows"], 256):
            x = state["logits"][lo:lo + 256].to(f64)
            lse = torch.logsumexp(x, dim=1)
            lp = x - lse[:, None]
            cols["lse"].append(lse)
            cols["entropy"].append(-torch.where(torch.isinf(lp), 0.0, lp * lp.exp()).sum(dim=1))
            if case["n_tok"]:
                cols["logprob"].append(torch.gather(lp, 1, state["tokens"][lo:lo + 256].long()))
            if case["top_k"]:
                val, ids = torch.sort(lp, dim=1, descending=True, stable=True)
                cols["top_ids"].append(ids[:, : case["top_k"]].to(torch.int32))
                cols["top_logprobs"].append(val[:, : case["top_k"]])
        return {k: torch.cat(v) for k, v in cols.items() if v}
    Hq, Hkv, D, B = case["heads"], case["kv_heads"], case["dim"], case["batch"]
    rep = Hq // Hkv
    lens = state["kv_len"].tolist()

    def softmax_rows(sc, v):
        lse = torch.logsumexp(sc, dim=-1)
        w = torch.exp(sc - torch.where(torch.isinf(lse), 0.0, lse)[..., None])
        return w @ v, lse

    if case["op"] == "prefix":
        out = torch.zeros((B, Hq, D), dtype=f64, device="cuda")
        lse = torch.zeros((B, Hq), dtype=f64, device="cuda")
        for b in range(B):
            kb = torch.cat([state["k_prefix"], state["k"][b, :, : lens[b]]], dim=1).to(f64)
            vb = torch.cat([state["v_prefix"], state["v"][b, :, : lens[b]]], dim=1).to(f64)
            qb = state["q"][b].to(f64).view(Hkv, rep, D)
            o, z = softmax_rows(qb @ kb.transpose(1, 2) / math.sqrt(D), vb)
            out[b], lse[b] = o.reshape(Hq, D), z.reshape(Hq)
        return {"out": out, "lse": lse}
    out = torch.zeros((B, case["q_cap"], Hq, D), dtype=f64, device="cuda")
    lse = torch.zeros((B, case["q_cap"], Hq), dtype=f64, device="cuda")
    qlens = state["q_len"].tolist()
    for b in range(B):
        n, ql = lens[b], qlens[b]
        for lo in range(0, ql, 1024):  # blocks of queries against the keys that any of them may see
            hi = min(ql, lo + 1024)
            pos = torch.arange(n - ql + lo, n - ql + hi, device="cuda")
            end = max(0, n - ql + hi)
            j = torch.arange(end, device="cuda")
            first = max(0, n - ql + lo - case["window"] + 1)
            keep = (j >= first) | (j < case["sinks"])
            j = j[keep]
            back = pos[:, None] - j[None, :]
            hide = (back < 0) | ((back >= case["window"]) & (j[None, :] >= case["sinks"]))
            for h in range(Hkv):
                kb, vb = state["k"][b, h, :end][keep].to(f64), state["v"][b, h, :end][keep].to(f64)
                qb = state["q"][b, lo:hi, h * rep:(h + 1) * rep].to(f64).transpose(0, 1)
                sc = (qb @ kb.T / math.sqrt(D)).masked_fill(hide, float("-inf"))
                if j.numel():
                    o, z = softmax_rows(sc, vb)
                else:
                    o, z = torch.zeros_like(qb), torch.full(qb.shape[:-1], float("-inf"), dtype=f64, device="cuda")
                out[b, lo:hi, h * rep:(h + 1) * rep] = o.transpose(0, 1)
                lse[b, lo:hi, h * rep:(h + 1) * rep] = z.transpose(0, 1)
    return {"out": out, "lse": lse}
