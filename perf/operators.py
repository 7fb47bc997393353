"""Measured cases of the serving operators around the recurrent-state pool.

Five operators, reached through ``quantized_recurrent_state_gated_amd.sq``:

  tables   sq_block_tables         block tables and slot maps from request lengths
  append   sq_kv_append            keys and values into the paged cache
  attend   sq_paged_attention      one new token per request over the paged cache
  prefill  sq_prefill              chunked prompt form of the recurrent layers
  step     sq_decode_step_linear   single-token form with a plain decay

Where ``own`` is false, ``run`` computes each in its plain form: elementary
torch operations in 32 bits, rounded once at the end.
"""
import math

import torch

own = False

DEV = "cuda"
CHUNK = 64  # tokens per chunk of the plain prompt form
PAGES = (16, 32, 64)
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of the serving batch: every request gets one slot
        {"name": "tables_decode", "op": "tables", "n": 70, "ctx": 8192, "new": 1, "page": 16, "spread": 1.0},
        # admission of a large batch of prompts, part of them already cached
        {"name": "tables_prompts", "op": "tables", "n": 257, "ctx": 500, "new": 4096, "page": 64, "spread": 1.0},
        # the new tokens of one decode step
        {"name": "append_decode", "op": "append", "n": 70, "new": 1, "kv": 8, "d": 128, "page": 16, "dtype": "bf16"},
        # four long prompts
        {"name": "append_prompt", "op": "append", "n": 4, "new": 8191, "kv": 8, "d": 128, "page": 64, "dtype": "bf16"},
        # a single short conversation: latency counts
        {"name": "attend_one", "op": "attend", "n": 1, "len": 201, "q": 16, "kv": 2, "d": 128, "page": 16,
         "dtype": "bf16", "window": 0, "spread": 0.0},
        # the serving batch, contexts up to 16 Ki tokens
        {"name": "attend_serving", "op": "attend", "n": 70, "len": 16384, "q": 32, "kv": 8, "d": 128, "page": 16,
         "dtype": "bf16", "window": 0, "spread": 1.0},
        # few long contexts in full precision, odd group of query heads
        {"name": "attend_long_f32", "op": "attend", "n": 3, "len": 30001, "q": 20, "kv": 4, "d": 64, "page": 32,
         "dtype": "f32", "window": 0, "spread": 0.3},
        # a layer's prompts: 8 ragged sequences x 48 heads, the rule that sq_decode_step continues
        {"name": "prefill_delta", "op": "prefill", "n": 8, "len": 4096, "heads": 48, "d": 128, "dtype": "bf16",
         "rule": "delta", "init": False, "spread": 1.0},
        # one long prompt through a plain-decay layer
        {"name": "prefill_linear_long", "op": "prefill", "n": 1, "len": 16384, "heads": 48, "d": 128, "dtype": "bf16",
         "rule": "linear", "init": False, "spread": 0.0},
        # a few more tokens onto states that exist (a multi-turn request), full precision
        {"name": "prefill_more_f32", "op": "prefill", "n": 3, "len": 77, "heads": 12, "d": 128, "dtype": "f32",
         "rule": "delta", "init": True, "spread": 0.6},
        # one request, one layer's heads, full-precision states: latency counts
        {"name": "step_one_f32", "op": "step", "n": 1, "heads": 48, "state": "f32", "dtype": "bf16"},
        # the serving batch over 576 heads with bfloat16 states
        {"name": "step_serving_bf16", "op": "step", "n": 70, "heads": 576, "state": "bf16", "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["tables", "append", "attend", "attend", "prefill", "prefill", "step"])
    if op == "tables":
        n = _log(rng, 1, 400)
        decode = rng.random() < 0.4
        return {"op": op, "n": n, "ctx": _log(rng, 1, 16384), "new": 1 if decode else _log(rng, 1, 4096),
                "page": rng.choice(PAGES), "spread": rng.choice([0.0, 0.5, 1.0])}
    if op == "append":
        n = _log(rng, 1, 128)
        return {"op": op, "n": n, "new": _log(rng, 1, max(1, 32768 // n)), "kv": rng.randint(1, 8),
                "d": rng.choice([64, 128, 256]), "page": rng.choice(PAGES), "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if op == "attend":
        d, kv, dtype = rng.choice([64, 128, 256]), rng.randint(1, 8), rng.choice(["bf16", "bf16", "f32"])
        n = _log(rng, 1, 128)
        most = int(70 * 8192 * 8 * 128 * 2 / (n * kv * d * (2 if dtype == "bf16" else 4)))
        ln = _log(rng, 1, max(1, min(131072, most)))
        return {"op": op, "n": n, "len": ln, "q": kv * rng.randint(1, 16), "kv": kv, "d": d,
                "page": rng.choice(PAGES), "dtype": dtype, "window": rng.choice([0, 0, 0, _log(rng, 1, 8192)]),
                "spread": rng.choice([0.0, 0.5, 1.0])}
    if op == "prefill":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        n, heads = _log(rng, 1, 32), _log(rng, 1, 48)
        most = 8 * 2048 * 48 // (n * heads) if dtype == "bf16" else 98304 // (n * heads)
        top = 16384 if dtype == "bf16" else 2048
        return {"op": op, "n": n, "len": _log(rng, 1, max(1, min(top, most))), "heads": heads,
                "d": 128 if dtype == "bf16" else rng.choice([64, 128]), "dtype": dtype,
                "rule": rng.choice(["delta", "delta", "linear"]), "init": rng.random() < 0.5,
                "spread": rng.choice([0.0, 0.5, 1.0])}
    n = _log(rng, 1, 70)
    return {"op": op, "n": n, "heads": _log(rng, 1, 576), "state": rng.choice(["f32", "bf16"]),
            "dtype": rng.choice(["f32", "bf16"])}


def _lens(case, most, salt=0):
    """Ragged lengths of a case, at most `most` and one of them `most`: the
    same for every seed, so that a case is one amount of work.  spread 0: all
    equal; 1: down to a single token, the mean about half."""
    n, spread = case["n"], case.get("spread", 0.0)
    out = [most - int(spread * (most - 1) * ((i * 0.6180339887 + 0.37 * salt) % 1.0)) for i in range(n)]
    out[n // 2] = most
    return out


# ------------------------------------------------------------------ inputs

def _unit(shape, g):
    x = torch.randn(shape, generator=g, device=DEV)
    return x / x.norm(dim=-1, keepdim=True)


def _gates(lead, heads, g):
    """Gates around each head's half-life, log-uniform over 1 to 1000 tokens,
    and write strengths over (0.05, 0.95)."""
    life = torch.exp(torch.rand(heads, generator=g, device=DEV) * math.log(1000.0))
    z = torch.randn(lead + (heads,), generator=g, device=DEV)
    alpha = torch.exp(-(math.log(2.0) / life) * torch.exp(0.5 * z - 0.125))
    return alpha, 0.05 + 0.9 * torch.rand(lead + (heads,), generator=g, device=DEV)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _tables(lens, page, extra, g):
    """A fragmented cache: every request's pages lie anywhere in the pool."""
    need = [-(-x // page) for x in lens]
    pages = sum(need) + extra
    perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    cols = max(1, max(need))
    at, col = torch.tensor([0] + need, device=DEV).cumsum(0), torch.arange(cols, device=DEV)
    idx = (at[:-1, None] + col).clamp(max=pages - 1)
    held = col < torch.tensor(need, device=DEV)[:, None]
    return torch.where(held, perm[idx], 0).to(torch.int32).contiguous(), pages


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1000003 + 17)
    return {"tables": _prepare_tables, "append": _prepare_append, "attend": _prepare_attend,
            "prefill": _prepare_prefill, "step": _prepare_step}[case["op"]](dict(case), g)


def _prepare_tables(c, g):
    page, n = c["page"], c["n"]
    ctx, new = _lens(c, c["ctx"], 1), _lens(c, c["new"], 2)
    held = [-(-x // page) for x in ctx]
    need = [-(-(x + y) // page) - h for x, y, h in zip(ctx, new, held)]
    cols = max(h + m for h, m in zip(held, need)) + 1
    pages = sum(held) + sum(need) + 13
    perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    at, col = torch.tensor([0] + held, device=DEV).cumsum(0), torch.arange(cols, device=DEV)
    table = torch.where(col < torch.tensor(held, device=DEV)[:, None],
                        perm[(at[:-1, None] + col).clamp(max=pages - 1)], -1).to(torch.int32).contiguous()
    total = sum(new)
    i32 = {"dtype": torch.int32, "device": DEV}
    return {"c": c, "ctx": _ints(ctx), "new": _ints(new), "free": perm[sum(held):].contiguous(), "table": table,
            "total": total, "seq": torch.empty(n, **i32), "cu_new": torch.empty(n + 1, **i32),
            "cu_pages": torch.empty(n + 1, **i32), "result": torch.empty(1, **i32),
            "slots": torch.empty(total, dtype=torch.int64, device=DEV)}


def _cache(c, pages, g):
    dt, kv, d, page = DTYPES[c["dtype"]], c["kv"], c["d"], c["page"]
    k = torch.randn(pages, kv, page, d, generator=g, device=DEV, dtype=dt)
    v = torch.randn(pages, kv, d, page, generator=g, device=DEV, dtype=dt)
    if not own:
        return k, v, None
    from quantized_recurrent_state_gated_amd import sq
    return k, v, sq.SqKvCache(k, v)


def _prepare_append(c, g):
    page, n, new = c["page"], c["n"], c["new"]
    ctx = 3 if new > 1 else 5 * page + 3  # a prompt follows a few cached tokens, a decode step a context
    table, pages = _tables([ctx + new] * n, page, 3, g)
    pos = (ctx + torch.arange(new, device=DEV)).expand(n, new)
    slots = torch.gather(table.long(), 1, pos // page) * page + pos % page
    k, v, cache = _cache(c, pages, g)
    shape, dt = (n * new, c["kv"], c["d"]), DTYPES[c["dtype"]]
    return {"c": c, "kc": k, "vc": v, "cache": cache, "slots": slots.reshape(-1).contiguous(),
            "k": torch.randn(shape, generator=g, device=DEV, dtype=dt),
            "v": torch.randn(shape, generator=g, device=DEV, dtype=dt)}


def _prepare_attend(c, g):
    n, page, dt = c["n"], c["page"], DTYPES[c["dtype"]]
    lens = _lens(c, c["len"])
    table, pages = _tables(lens, page, 3, g)
    k, v, cache = _cache(c, pages, g)
    q = torch.randn(n, c["q"], c["d"], generator=g, device=DEV, dtype=dt)
    s = {"c": c, "kc": k, "vc": v, "cache": cache, "q": q, "table": table, "lens": _ints(lens), "most": max(lens)}
    if own:
        from quantized_recurrent_state_gated_amd import sq
        nb = sq.sq_paged_attention_workspace(cache, n, c["q"], max(lens))
        s |= {"ws": torch.empty(max(nb, 256), dtype=torch.uint8, device=DEV), "o": torch.empty_like(q),
              "lse": torch.empty(n, c["q"], device=DEV)}
    return s


def _prepare_prefill(c, g):
    n, H, d, dt = c["n"], c["heads"], c["d"], DTYPES[c["dtype"]]
    lens = _lens(c, c["len"])
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    N = cu[-1]
    alpha, beta = _gates((N,), H, g)
    s = {"c": c, "q": _unit((N, H, d), g).to(dt), "k": _unit((N, H, d), g).to(dt),
         "v": torch.randn(N, H, d, generator=g, device=DEV).to(dt), "alpha": alpha, "beta": beta,
         "cu": _ints(cu), "most": max(lens),
         "S0": torch.randn(n, H, d, d, generator=g, device=DEV) if c["init"] else None}
    if own:
        from quantized_recurrent_state_gated_amd import sq
        nb = sq.sq_prefill_workspace(n, N, H, d, d, dt, _rule(c))
        s |= {"ws": torch.empty(max(nb, 256), dtype=torch.uint8, device=DEV), "o": torch.empty_like(s["v"]),
              "S": torch.empty(n, H, d, d, device=DEV)}
    return s


def _prepare_step(c, g):
    n, H, d, dt = c["n"], c["heads"], 128, DTYPES[c["dtype"]]
    slots_n = n + 1
    state = torch.randn(slots_n, H, d, d, generator=g, device=DEV).mul_(0.5).to(DTYPES[c["state"]])
    alpha, beta = _gates((n,), H, g)
    s = {"c": c, "q": _unit((n, H, d), g).to(dt), "k": _unit((n, H, d), g).to(dt),
         "v": torch.randn(n, H, d, generator=g, device=DEV).to(dt), "alpha": alpha, "beta": beta,
         "ids": torch.randperm(slots_n, generator=g, device=DEV)[:n].to(torch.int32).contiguous()}
    if not own:
        # a plain program keeps its states row by row
        return s | {"state": state.view(slots_n, H, d // 4, 4, d // 4, 4)}
    # the pool keeps them in 4 x 4 blocks, column after column (the format in
    # include/sq.h): the same values, seen through a permuted view
    from quantized_recurrent_state_gated_amd import sq
    tiles = state.view(slots_n, H, d // 4, 4, d // 4, 4).permute(0, 1, 2, 4, 5, 3).contiguous()
    raw = tiles.view(-1).view(torch.uint8)
    ones = torch.ones(H, d, device=DEV)
    pool = sq.sq_pool_alloc(slots_n, H, d, d, [32 if c["state"] == "f32" else 144] * H, ones, ones, raw)
    return s | {"pool": pool, "state": tiles.permute(0, 1, 2, 5, 3, 4),
                "o": torch.empty(n, H, d, device=DEV)}


# ------------------------------------------------------------------ one pass

def _rule(c):
    from quantized_recurrent_state_gated_amd import sq
    return sq.SQ_RULE_DELTA if c["rule"] == "delta" else sq.SQ_RULE_LINEAR


def run(s):
    return (_run_own if own else _run_plain)[s["c"]["op"]](s)


def _own_tables(s):
    from quantized_recurrent_state_gated_amd import sq
    sq.sq_block_tables(s["ctx"], s["new"], s["c"]["page"], s["free"], s["table"], s["seq"], s["cu_new"],
                       s["cu_pages"], s["slots"], s["result"])
    return {k: s[k] for k in ("table", "seq", "cu_new", "cu_pages", "slots", "result")}


def _own_append(s):
    from quantized_recurrent_state_gated_amd import sq
    sq.sq_kv_append(s["cache"], s["k"], s["v"], s["slots"])
    return {"k": s["kc"], "v": s["vc"]}


def _own_attend(s):
    from quantized_recurrent_state_gated_amd import sq
    sq.sq_paged_attention(s["cache"], s["q"], s["table"], s["lens"], s["most"], s["o"], s["ws"],
                          window=s["c"]["window"], lse=s["lse"])
    return {"o": s["o"], "lse": s["lse"]}


def _own_prefill(s):
    from quantized_recurrent_state_gated_amd import sq
    sq.sq_prefill(s["q"], s["k"], s["v"], s["alpha"], s["beta"], s["cu"], s["o"], S=s["S"], S0=s["S0"],
                  rule=_rule(s["c"]), workspace=s["ws"])
    return {"o": s["o"], "S": s["S"]}


def _own_step(s):
    from quantized_recurrent_state_gated_amd import sq
    sq.sq_decode_step_linear(s["pool"], s["ids"], s["q"], s["k"], s["v"], s["alpha"], s["beta"], s["o"])
    return {"o": s["o"], "state": s["state"]}


def _plain_tables(s):
    page, n, ctx, new = s["c"]["page"], s["c"]["n"], s["ctx"], s["new"]
    seq = ctx + new
    held = (ctx + page - 1) // page
    need = (seq + page - 1) // page - held
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    cu_new = torch.cat([zero, new.cumsum(0, dtype=torch.int32)])
    cu_pages = torch.cat([zero, need.cumsum(0, dtype=torch.int32)])
    col = torch.arange(s["table"].shape[1], device=DEV)
    fresh = (col >= held[:, None]) & (col < (held + need)[:, None])
    pick = (cu_pages[:-1, None] + col - held[:, None]).clamp(0, s["free"].numel() - 1)
    table = torch.where(fresh, s["free"][pick.long()], s["table"])
    tok = torch.arange(s["total"], device=DEV)
    req = torch.searchsorted(cu_new, tok, right=True) - 1
    pos = ctx[req] + (tok - cu_new[req])
    slots = table[req, pos // page].long() * page + pos % page
    result = ((cu_pages[-1:] > s["free"].numel()).int() * 2).int()
    return {"table": table, "seq": seq, "cu_new": cu_new, "cu_pages": cu_pages, "slots": slots, "result": result}


def _plain_append(s):
    page = s["c"]["page"]
    p, at = s["slots"] // page, s["slots"] % page
    s["kc"].permute(0, 2, 1, 3)[p, at] = s["k"]
    s["vc"].permute(0, 3, 1, 2)[p, at] = s["v"]
    return {"k": s["kc"], "v": s["vc"]}


def _plain_attend(s):
    c, t = s["c"], s["table"].long()
    n, kv, d, page = c["n"], c["kv"], c["d"], c["page"]
    L = t.shape[1] * page
    K = s["kc"][t].transpose(1, 2).reshape(n, kv, L, d).float()
    V = s["vc"][t].permute(0, 2, 1, 4, 3).reshape(n, kv, L, d).float()
    q = s["q"].float().view(n, kv, c["q"] // kv, d)
    x = torch.matmul(q, K.transpose(-1, -2)) / math.sqrt(d)
    pos, lens = torch.arange(L, device=DEV), s["lens"][:, None]
    seen = pos < lens
    if c["window"]:
        seen &= pos >= lens - c["window"]
    x = x.masked_fill(~seen[:, None, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - top)
    tot = e.sum(-1, keepdim=True)
    o = torch.matmul(e, V) / tot
    return {"o": o.reshape(n, c["q"], d).to(s["q"].dtype), "lse": (top + tot.log()).reshape(n, c["q"])}


def _plain_prefill(s):
    c, cu = s["c"], s["cu"].long()
    n, H, d, N = c["n"], c["heads"], c["d"], s["q"].shape[0]
    nc = -(-s["most"] // CHUNK)
    pos = torch.arange(nc * CHUNK, device=DEV)
    there = pos < (cu[1:] - cu[:-1])[:, None]
    tok = (cu[:-1, None] + pos).clamp(max=N - 1)

    def chunks(x, fill):  # [N][H](d) -> [n][H][chunk][CHUNK](d), padded with `fill`
        x = x[tok].float()
        m = there.view(there.shape + (1,) * (x.dim() - 2))
        x = torch.where(m, x, fill).transpose(1, 2)
        return x.reshape(x.shape[:2] + (nc, CHUNK) + x.shape[3:])

    q, k, v = chunks(s["q"], 0.0), chunks(s["k"], 0.0), chunks(s["v"], 0.0)
    beta = chunks(s["beta"], 0.0)[..., None]
    G = chunks(s["alpha"], 1.0).log().cumsum(-1)[..., None]
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=DEV).tril()
    D = torch.where(low, (G - G.transpose(-1, -2)).clamp(max=0.0).exp(), 0.0)
    gam, last = G.exp(), (G[..., -1:, :] - G).exp()
    kt = k.transpose(-1, -2)
    P = torch.matmul(q, kt) * D
    W, X = beta * v, None
    if c["rule"] == "delta":
        # (I + M)^-1 as the product of I - M, I + M^2, I + M^4, ...: M^64 = 0
        M = (beta * torch.matmul(k, kt) * D).tril(-1)
        eye = torch.eye(CHUNK, device=DEV)
        inv, power = eye - M, torch.matmul(M, M)
        inv = torch.matmul(inv, eye + power)
        power = torch.matmul(power, power)
        inv = torch.matmul(inv, eye + power)
        power = torch.matmul(power, power)
        inv = torch.matmul(inv, eye + power)
        power = torch.matmul(power, power)
        inv = torch.matmul(inv, eye + power)
        power = torch.matmul(power, power)
        inv = torch.matmul(inv, eye + power)
        W, X = torch.matmul(inv, W), torch.matmul(inv, beta * gam * k)
    kd, qg = (k * last).transpose(-1, -2), q * gam
    S = torch.zeros(n, H, d, d, device=DEV) if s["S0"] is None else s["S0"]
    outs = []
    for j in range(nc):  # the state goes from chunk to chunk
        w = W[:, :, j] if X is None else W[:, :, j] - torch.matmul(X[:, :, j], S)
        outs.append(torch.matmul(qg[:, :, j], S) + torch.matmul(P[:, :, j], w))
        S = gam[:, :, j, -1:] * S + torch.matmul(kd[:, :, j], w)
    o = torch.stack(outs, 2).reshape(n, H, nc * CHUNK, d)
    t = torch.arange(N, device=DEV)
    seq = torch.searchsorted(cu, t, right=True) - 1
    return {"o": o.transpose(1, 2)[seq, t - cu[seq]].to(s["q"].dtype), "S": S}


def _plain_step(s):
    ids = s["ids"].long()
    n, H, d = s["q"].shape
    S = s["state"][ids].view(n, H, d, d).float()
    bk = s["beta"][..., None] * s["k"].float()
    S = s["alpha"][..., None, None] * S + bk[..., None] * s["v"].float()[..., None, :]
    o = (s["q"].float()[..., None] * S).sum(-2)
    s["state"][ids] = S.view(n, H, d // 4, 4, d // 4, 4).to(s["state"].dtype)
    return {"o": o, "state": s["state"]}


_run_plain = {"tables": _plain_tables, "append": _plain_append, "attend": _plain_attend,
              "prefill": _plain_prefill, "step": _plain_step}
_run_own = {"tables": _own_tables, "append": _own_append, "attend": _own_attend,
            "prefill": _own_prefill, "step": _own_step}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c, op = case, case["op"]
    es = 2 if c.get("dtype") == "bf16" else 4
    if op == "tables":
        ctx, new = _lens(c, c["ctx"], 1), _lens(c, c["new"], 2)
        pages = sum(-(-(x + y) // c["page"]) - -(-x // c["page"]) for x, y in zip(ctx, new))
        return {"bytes": 20 * c["n"] + 8 * pages + 8 * sum(new) + 12, "flops": 0}
    if op == "append":
        n = c["n"] * c["new"]
        return {"bytes": n * (8 + 4 * c["kv"] * c["d"] * es), "flops": 0}
    if op == "attend":
        seen = sum(min(x, c["window"]) if c["window"] else x for x in _lens(c, c["len"]))
        return {"bytes": 2 * seen * c["kv"] * c["d"] * es + 2 * c["n"] * c["q"] * c["d"] * es,
                "flops": 4 * seen * c["q"] * c["d"]}
    if op == "prefill":
        th, d = sum(_lens(c, c["len"])) * c["heads"], c["d"]
        states = c["n"] * c["heads"] * d * d * 4 * (2 if c["init"] else 1)
        return {"bytes": th * (4 * d * es + 8) + states, "flops": th * d * d * (8 if c["rule"] == "delta" else 5)}
    th, d = c["n"] * c["heads"], 128
    ss = 2 if c["state"] == "bf16" else 4
    return {"bytes": th * (2 * d * d * ss + 3 * d * es + 8 + 4 * d), "flops": 5 * th * d * d}


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "tables":
        return None  # whole numbers: both sides have to agree on all of them
    return {"append": _exact_append, "attend": _exact_attend, "prefill": _exact_prefill, "step": _exact_step}[op](s)


def _exact_append(s):
    page = s["c"]["page"]
    k, v = s["kc"].double(), s["vc"].double()
    kf = k.transpose(1, 2).reshape(-1, *s["k"].shape[1:])
    vf = v.permute(0, 3, 1, 2).reshape(-1, *s["v"].shape[1:])
    kf.index_copy_(0, s["slots"], s["k"].double())
    vf.index_copy_(0, s["slots"], s["v"].double())
    P = k.shape[0]
    return {"k": kf.view(P, page, *kf.shape[1:]).transpose(1, 2).contiguous(),
            "v": vf.view(P, page, *vf.shape[1:]).permute(0, 2, 3, 1).contiguous()}


def _exact_attend(s):
    c = s["c"]
    kv, d, G = c["kv"], c["d"], c["q"] // c["kv"]
    o, lse = [], []
    for r, n in enumerate(_lens(c, c["len"])):
        first = max(0, n - c["window"]) if c["window"] else 0
        pages = s["table"][r].long()
        K = s["kc"][pages].permute(1, 0, 2, 3).reshape(kv, -1, d)[:, first:n].double()
        V = s["vc"][pages].permute(1, 0, 3, 2).reshape(kv, -1, d)[:, first:n].double()
        q = s["q"][r].double().view(kv, G, d)
        x = (q @ K.mT) * d ** -0.5
        l = torch.logsumexp(x, -1)
        o.append((torch.exp(x - l[..., None]) @ V).reshape(kv * G, d))
        lse.append(l.reshape(-1))
    return {"o": torch.stack(o), "lse": torch.stack(lse)}


def _exact_prefill(s):
    """Token by token, as the recurrence is written."""
    c, cu = s["c"], s["cu"].tolist()
    n, H, d = c["n"], c["heads"], c["d"]
    S = torch.zeros(n, H, d, d, device=DEV, dtype=torch.float64) if s["S0"] is None else s["S0"].double()
    o = torch.zeros(s["q"].shape, device=DEV, dtype=torch.float64)
    order = sorted(range(n), key=lambda i: cu[i] - cu[i + 1])  # longest first: those still running are a prefix
    S = S[order]
    starts = torch.tensor([cu[i] for i in order], device=DEV)
    lens = [cu[i + 1] - cu[i] for i in order]
    for t in range(lens[0]):
        m = sum(x > t for x in lens)
        at = starts[:m] + t
        q, k, v = (s[x][at].double() for x in "qkv")
        a, b = s["alpha"][at].double()[..., None], s["beta"][at].double()[..., None]
        R = S[:m]
        w = b * v
        if c["rule"] == "delta":
            w -= a * b * torch.matmul(k[:, :, None], R)[:, :, 0]
        R.mul_(a[..., None]).addcmul_(k[..., None], w[:, :, None])
        o[at] = torch.matmul(q[:, :, None], R)[:, :, 0]
    back = torch.empty_like(S)
    back[order] = S
    return {"o": o, "S": back}


def _exact_step(s):
    ids, d = s["ids"].long(), 128
    n, H = s["alpha"].shape
    state = s["state"].reshape(-1, H, d, d).double()
    S = torch.einsum("nh,nhij->nhij", s["alpha"].double(), state[ids])
    S += torch.einsum("nh,nhi,nhj->nhij", s["beta"].double(), s["k"].double(), s["v"].double())
    o = torch.einsum("nhi,nhij->nhj", s["q"].double(), S)
    state[ids] = S
    return {"o": o, "state": state.view(-1, H, d // 4, 4, d // 4, 4)}
