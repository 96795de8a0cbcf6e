"""Cases for the operators of the prompt step: attention over packed prompts
(gk_prompt_attn) and block tables and slot maps built on the device
(gk_tables_step).

run() computes each in its plain form, elementary torch operations in fp32, or,
where `own` is true, through the library's calls.  A prompt case is one layer of
one step; a tables case is one step's bookkeeping.  Sizes follow the synthetic
workloads of this repository (Llama-3.1-8B: 32 query heads on 8 KV heads of 128;
Qwen-2.5-14B: 40 on 8; the tiny workload: 4 on 2 of 64) and a few generic ones.
"""
import random

import numpy as np
import torch

own = False

#: query heads, KV heads, head dim
GEOMETRY = {"tiny": (4, 2, 64), "small": (16, 4, 64), "single": (8, 8, 64), "mqa": (8, 1, 128), "mha": (8, 8, 128),
            "pairs": (16, 8, 128), "llama8b": (32, 8, 128), "qwen14b": (40, 8, 128)}


def _prompt(name, geo, b, lo, hi, n_prefix=0, plo=0, phi=0, clo=0, chi=0, page=16, fused=False, draw=1):
    c = dict(op="prompt", geo=geo, b=b, lo=lo, hi=hi, n_prefix=n_prefix, plo=plo, phi=phi, clo=clo, chi=chi, page=page,
             fused=fused, draw=draw)
    return dict(c, name=name) if name else c


def _tables(name, rows, page, llo, lhi, alo, ahi, release, short=False, draw=1):
    c = dict(op="tables", rows=rows, page=page, llo=llo, lhi=lhi, alo=alo, ahi=ahi, release=release, short=short, draw=draw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # the tiny workload's requests arriving: a few tokens each behind a 64-token shared prefix (latency)
        _prompt("tiny_prompts", "tiny", 4, 1, 48, n_prefix=1, plo=64, phi=64, page=1),
        # one short question, no cache (latency)
        _prompt("one_question", "llama8b", 1, 77, 77, fused=True),
        # a batch of fresh chat prompts of different lengths
        _prompt("chat_prompts", "llama8b", 24, 64, 1500, fused=True),
        # multi-agent turns: every agent's turn of a few hundred tokens behind one of four shared prefixes
        _prompt("agent_turns", "qwen14b", 32, 64, 600, n_prefix=4, plo=2048, phi=8192, clo=0, chi=1000, page=1),
        # a few tokens each (tool answers, drafted tokens) behind a long shared prefix and the agent's own history
        _prompt("drafted_tokens", "llama8b", 64, 1, 16, n_prefix=1, plo=16384, phi=16384, clo=256, chi=2048, page=1),
        # two chunks of long prompts whose earlier chunks are in the pages already
        _prompt("prompt_chunks", "llama8b", 2, 2040, 2048, clo=6000, chi=12000, page=16, fused=True),
        # half-width heads, one KV head for each four query heads, an odd length
        _prompt("narrow_heads", "small", 3, 2777, 4099),
        # a whole long prompt at once: the largest
        _prompt("long_prompt", "qwen14b", 1, 16384, 16384),
        # a decode step of the eight-prefix workload: every request one token, a few requests leave
        _tables("decode_step", 368, 1, 128, 4096, 1, 1, 8),
        # a batch of fresh prompts takes pages of 16 while others leave
        _tables("prompt_pages", 48, 16, 0, 2048, 64, 1500, 12),
        # long prompts into token-granular slots
        _tables("long_prompt_slots", 24, 1, 0, 8192, 2048, 16384, 6),
        # many short requests, and more asked for than is free: the rows behind the last block get nothing
        _tables("out_of_blocks", 1024, 4, 0, 300, 0, 40, 100, short=True),
    ]


def _log(r, lo, hi):
    return lo if lo >= hi else min(hi, max(lo, round((lo + 1) * ((hi + 1) / (lo + 1)) ** r.random() - 1)))


def _lengths(c):
    """new, prefix index, COLD context of each request; the prefixes' lengths."""
    r = random.Random(c["draw"])
    prefixes = [_log(r, c["plo"], c["phi"]) for _ in range(c["n_prefix"])]
    new = [_log(r, c["lo"], c["hi"]) for _ in range(c["b"])]
    which = [r.randrange(len(prefixes)) if prefixes else -1 for _ in range(c["b"])]
    cold = [_log(r, c["clo"], c["chi"]) for _ in range(c["b"])]
    return new, which, cold, prefixes


def _rows(c):
    """length, added tokens and leave flag of each row (one that leaves takes nothing in the same step); free blocks at the start."""
    r = random.Random(c["draw"])
    P, R = c["page"], c["rows"]
    length = [_log(r, c["llo"], c["lhi"]) for _ in range(R)]
    add = [_log(r, c["alo"], c["ahi"]) for _ in range(R)]
    leave = [0] * R
    for i in r.sample(range(R), min(R, c["release"])):
        leave[i], add[i] = 1, 0
    need = sum(-(-(n + a) // P) - -(-n // P) for n, a in zip(length, add))
    back = sum(-(-n // P) for n, x in zip(length, leave) if x)
    return length, add, leave, max(0, int(need * 0.7) - back) if c["short"] else need + 57


def draw(rng):
    while True:
        seed = rng.randrange(1 << 30)
        if rng.random() < 0.3:
            page = rng.choice([1, 4, 16, 16, 128])
            rows, ahi = _log(rng, 1, 1500), rng.choice([1, 1, 16, 700, 6000])
            lhi = _log(rng, 1, 8192)
            c = _tables(None, rows, page, rng.choice([0, lhi // 2]), lhi, rng.choice([0, 1, ahi // 2]), ahi, rng.randrange(rows // 2 + 1),
                        rng.random() < 0.25, seed)
            if rows * (ahi + lhi) < 1200000:
                return c
        else:
            geo = rng.choice(sorted(GEOMETRY))
            b, hi = _log(rng, 1, 64), _log(rng, 1, 16384)
            some = rng.random()
            phi, chi = (_log(rng, 1, 16384) if some < 0.6 else 0), (_log(rng, 1, 8192) if some > 0.3 else 0)
            c = _prompt(None, geo, b, rng.choice([0, hi // 2, hi]), hi, rng.randrange(1, 5) if phi else 0, (phi + 1) // 2, phi, chi // 3, chi,
                        rng.choice([1, 3, 16, 64]), rng.random() < 0.5, seed)
            new, which, cold, prefixes = _lengths(c)
            w = work(c)
            tokens = sum(new) + sum(cold) + sum(prefixes)
            if sum(new) and w["flops"] <= 2.7e12 and tokens * GEOMETRY[geo][0] * GEOMETRY[geo][2] <= 16384 * 40 * 128 * 2:
                return c


def work(c):
    if c["op"] == "prompt":
        hq, hkv, d = GEOMETRY[c["geo"]]
        new, which, cold, prefixes = _lengths(c)
        T = sum(new)
        used = sum(lp for p, lp in enumerate(prefixes) if any(w == p and n for w, n in zip(which, new)))
        past = [(prefixes[w] if w >= 0 else 0) + k for w, k in zip(which, cold)]
        pairs = sum(n * k + n * (n + 1) // 2 for n, k in zip(new, past))
        kept = used + sum(k for n, k in zip(new, cold) if n)
        blocks = sum(-(-k // c["page"]) for n, k in zip(new, cold) if n)
        return {"bytes": 4 * T * hq * d + 4 * T * hq + 4 * T * hkv * d + 4 * kept * hkv * d + 4 * blocks, "flops": 4 * d * hq * pairs}
    length, add, leave, free = _rows(c)
    P, asked = c["page"], sum(add)
    taken = sum(-(-((0 if x else n) + a) // P) - -(-(0 if x else n) // P) for n, a, x in zip(length, add, leave))
    back = sum(-(-n // P) for n, x in zip(length, leave) if x)
    taken = min(taken, free + back)
    return {"bytes": 20 * c["rows"] + 8 * back + 8 * taken + 8 * asked + 8, "flops": 10 * c["rows"] + 6 * asked}


class _Handles:
    """The library's pool (and plan) over a state's storage, for as long as the state lives."""

    def __init__(self, gk, pool):
        self.gk, self.pool, self.plan = gk, pool, None

    def __del__(self):
        if self.plan:
            self.gk.gk_prompt_plan_destroy(self.plan)
        self.gk.gk_pool_destroy(self.pool)


def _prepare_prompt(c, seed):
    dev, bf = "cuda", torch.bfloat16
    g = torch.Generator(device=dev).manual_seed(seed)
    hq, hkv, d = GEOMETRY[c["geo"]]
    new, which, cold, prefixes = _lengths(c)
    T, P, page_of = sum(new), c["page"], [-(-k // c["page"]) for k in cold]
    blocks = sum(page_of) + 7

    def kv(*shape):
        # channels with offsets of their own, as keys and values have
        x = torch.randn(*shape, d, generator=g, device=dev)
        return x.add_(0.4 * torch.randn(d, generator=g, device=dev)).to(bf)

    s = {"c": c, "new": new, "which": which, "cold": cold, "prefixes": prefixes}
    # HOT: prefix p owns rows [base, base + length) of every head, laid out [head][token][d] (one layer)
    s["bases"] = [sum(prefixes[:p]) for p in range(len(prefixes))]
    hot = max(1, sum(prefixes))
    s["hot_k"], s["hot_v"] = kv(hot * hkv), kv(hot * hkv)
    s["cold_k"], s["cold_v"] = kv(1, blocks * P, hkv), kv(1, blocks * P, hkv)
    order = torch.randperm(blocks, generator=g, device=dev).to(torch.int32)
    width = max([1] + page_of)
    table = torch.zeros(c["b"], width, dtype=torch.int32, device=dev)
    at = 0
    for r, n in enumerate(page_of):
        table[r, :n] = order[at:at + n]
        at += n
    s["table"] = table
    if c["fused"]:  # one projection's output: q, k and v of a token side by side
        row = torch.empty(T, (hq + 2 * hkv) * d, dtype=bf, device=dev)
        s["q"], s["k"], s["v"] = (row[:, a * d:b * d].view(T, b - a, d) for a, b in ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv)))
    else:
        s["q"], s["k"], s["v"] = (torch.empty(T, n, d, dtype=bf, device=dev) for n in (hq, hkv, hkv))
    s["q"].copy_(1.5 * torch.randn(T, hq, d, generator=g, device=dev))
    s["k"].copy_(kv(T, hkv))
    s["v"].copy_(kv(T, hkv))
    s["out"] = torch.empty(T, hq, d, dtype=bf, device=dev)
    s["lse"] = torch.empty(T, hq, device=dev)
    if own:
        from paged_kv_cache_pool_gb300 import binding as gk
        h = _Handles(gk, gk.gk_pool_create(1, hq, hkv, d, hot, blocks * P, P, 0, s["hot_k"], s["hot_v"], s["cold_k"], s["cold_v"]))
        for base, lp in zip(s["bases"], prefixes):
            assert gk.gk_prefix_alloc(h.pool, lp) == base
        s["batch"] = gk.PromptBatch(new, [s["bases"][p] if p >= 0 else -1 for p in which], [prefixes[p] if p >= 0 else 0 for p in which],
                                    cold, table, width)
        h.plan = gk.gk_prompt_plan_build(h.pool, s["batch"], torch.cuda.current_stream())
        s["handles"] = h
    return s


def _prepare_tables(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    length, add, leave, free = _rows(c)
    P, R = c["page"], c["rows"]
    held = [-(-n // P) for n in length]
    blocks = sum(held) + free
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    order = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    width = max([1] + [-(-(n + a) // P) for n, a in zip(length, add)])
    s = {"c": c, "R": R, "P": P, "width": width, "blocks": blocks, "slots_n": max(1, sum(add)), "len": ints(length), "add": ints(add),
         "leave": ints(leave), "n_free": ints([free])}
    # the last cells of both are the plain form's bins
    s["cells"], s["free"] = (torch.zeros(n + 1, dtype=torch.int32, device="cuda") for n in (R * width, blocks))
    s["table"] = s["cells"][:-1].view(R, width)
    at = torch.arange(width, device="cuda")[None] < s["len"].add(P - 1).div(P, rounding_mode="floor")[:, None]
    s["table"][at] = order[free:]
    s["free"][:free] = order[:free]
    s["len_out"], s["n_free_out"], s["done"] = torch.empty_like(s["len"]), torch.empty_like(s["n_free"]), torch.empty_like(s["len"])
    s["slots"] = torch.empty(s["slots_n"], dtype=torch.int64, device="cuda")
    if own:
        from paged_kv_cache_pool_gb300 import binding as gk
        # bookkeeping needs no head: the smallest geometry's storage
        s["kv"] = [torch.zeros(max(64, blocks * P) * 64, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
        s["handles"] = _Handles(gk, gk.gk_pool_create(1, 1, 1, 64, 64, blocks * P, P, 0, *s["kv"]))
        s["tables"] = gk.Tables(s["table"], s["free"][:-1], s["len"], s["n_free"], s["len_out"], s["n_free_out"])
    return s


def prepare(case, seed):
    return (_prepare_prompt if case["op"] == "prompt" else _prepare_tables)(case, seed)


def _past(s, r, dtype):
    """K and V of request r's HOT and COLD tokens, [heads][tokens][d]."""
    c, p, n = s["c"], s["which"][r], s["cold"][r]
    hkv, d = GEOMETRY[c["geo"]][1:]
    at = torch.arange(n, device="cuda")
    slot = s["table"][r].long()[at // c["page"]] * c["page"] + at % c["page"]
    lp, base = (s["prefixes"][p], s["bases"][p]) if p >= 0 else (0, 0)
    return [torch.cat([hot[base * hkv:(base + lp) * hkv].view(hkv, lp, d).to(dtype), cold[0, slot].transpose(0, 1).to(dtype)], 1)
            for hot, cold in ((s["hot_k"], s["cold_k"]), (s["hot_v"], s["cold_v"]))]


def _plain_prompt(s):
    hq, hkv, d = GEOMETRY[s["c"]["geo"]]
    t0 = 0
    for r, n in enumerate(s["new"]):
        pk, pv = _past(s, r, torch.float32)
        k = torch.cat([pk, s["k"][t0:t0 + n].transpose(0, 1).float()], 1)
        v = torch.cat([pv, s["v"][t0:t0 + n].transpose(0, 1).float()], 1)
        q = s["q"][t0:t0 + n].float().view(n, hkv, hq // hkv, d).permute(1, 2, 0, 3)
        past, step = pk.shape[1], max(16, (1 << 29) // (hq * k.shape[1]))
        for a in range(0, n, step):  # rows whose scores fit in memory together
            b = min(n, a + step)
            keys = past + b
            score = (q[:, :, a:b].reshape(hkv, -1, d) @ k[:, :keys].transpose(1, 2)).mul_(d ** -0.5).view(hkv, hq // hkv, b - a, keys)
            hidden = torch.arange(keys, device="cuda")[None] > past + torch.arange(a, b, device="cuda")[:, None]
            score.masked_fill_(hidden, float("-inf"))
            top = score.amax(-1, keepdim=True)
            weight = score.sub_(top).exp_()
            total = weight.sum(-1, keepdim=True)
            o = (weight.view(hkv, -1, keys) @ v[:, :keys]).view(hkv, hq // hkv, b - a, d) / total
            s["out"][t0 + a:t0 + b] = o.permute(2, 0, 1, 3).reshape(b - a, hq, d).to(torch.bfloat16)
            s["lse"][t0 + a:t0 + b] = (top + total.log()).permute(2, 0, 1, 3).reshape(b - a, hq)
        t0 += n
    return {"out": s["out"], "lse": s["lse"]}


def _plain_tables(s):
    P, R, table, free, n0 = s["P"], s["R"], s["table"], s["free"], s["n_free"].long()
    up = lambda x: (x + (P - 1)) // P  # noqa: E731
    length, add, leave = s["len"].long(), s["add"].long(), s["leave"] != 0
    col = torch.arange(s["width"], device="cuda")
    # rows that leave: their blocks onto the stack, in row order
    back = (leave[:, None] & (col[None] < up(length)[:, None])).view(-1)
    rank = back.cumsum(0)
    free.scatter_(0, torch.where(back, n0 + rank - 1, s["blocks"]), table.view(-1))
    n1 = n0 + rank[-1:]
    # rows that grow: blocks off the stack, in row order, until it is empty
    length = torch.where(leave, 0, length)
    have = up(length)
    need = up(length + add) - have
    first, begin = need.cumsum(0) - need, add.cumsum(0) - add
    fits = ((have + n1 - first) * P - length).clamp(min=0)
    done = torch.where(first > n1, 0, torch.minimum(add, fits))
    s["done"].copy_(done)
    s["len_out"].copy_(length + done)
    s["n_free_out"].copy_(n1 - (up(length + done) - have).sum())
    t = torch.arange(s["slots_n"], device="cuda")
    row = torch.searchsorted(begin + add, t, right=True).clamp(max=R - 1)
    k = t - begin[row]
    placed = k < done[row]
    pos = torch.where(placed, length[row] + k, 0)
    fresh = placed & (pos // P >= have[row])
    top = torch.where(fresh, n1 - 1 - (first[row] + pos // P - have[row]), 0)
    cell = torch.where(placed, row * s["width"] + pos // P, R * s["width"])
    block = torch.where(fresh, free[top], s["cells"][cell])
    s["cells"].scatter_(0, cell, block)  # tokens of one block write the same id
    s["slots"].copy_(torch.where(placed, block.long() * P + pos % P, -1))
    return _tables_out(s)


def _tables_out(s):
    return {"table": s["table"], "free": s["free"][:-1], "len": s["len_out"], "n_free": s["n_free_out"], "slots": s["slots"],
            "done": s["done"]}


def run(state):
    s = state
    if s["c"]["op"] == "prompt":
        if not own:
            return _plain_prompt(s)
        h = s["handles"]
        s["batch"].set_device(d_q=s["q"], d_k=s["k"], d_v=s["v"], d_out=s["out"], d_lse=s["lse"])
        h.gk.gk_prompt_attn(h.pool, torch.cuda.current_stream(), 0, s["batch"], h.plan)
        return {"out": s["out"], "lse": s["lse"]}
    if not own:
        return _plain_tables(s)
    h = s["handles"]
    h.gk.gk_tables_step(h.pool, torch.cuda.current_stream(), s["tables"], s["add"], s["slots"], s["done"], s["leave"])
    return _tables_out(s)


def exact(case, seed):
    """The attention row by row of its definition, in 64 bits; the tables' outputs are whole numbers."""
    if case["op"] != "prompt":
        return None
    s = _prepare_prompt(case, seed)
    hq, hkv, d = GEOMETRY[case["geo"]]
    T, page = sum(s["new"]), case["page"]
    out = torch.empty(T, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.empty(T, hq, dtype=torch.float64, device="cuda")
    table = s["table"].cpu().numpy()
    start = np.cumsum([0] + s["new"])
    for r, n in enumerate(s["new"]):
        slots = torch.tensor([int(table[r, j // page]) * page + j % page for j in range(s["cold"][r])], dtype=torch.long, device="cuda")
        for head in range(hkv if n else 0):
            keys, values = [], []
            if s["which"][r] >= 0:
                lp = s["prefixes"][s["which"][r]]
                a = s["bases"][s["which"][r]] * hkv + head * lp
                keys.append(s["hot_k"][a:a + lp])
                values.append(s["hot_v"][a:a + lp])
            keys += [s["cold_k"][0, :, head][slots], s["k"][start[r]:start[r + 1], head]]
            values += [s["cold_v"][0, :, head][slots], s["v"][start[r]:start[r + 1], head]]
            K, V = torch.cat(keys).double(), torch.cat(values).double()
            seen = len(K) - n
            for h in range(head * hq // hkv, (head + 1) * hq // hkv):
                for a in range(0, n, 4096):
                    b = min(n, a + 4096)
                    z = (s["q"][start[r] + a:start[r] + b, h].double() / np.sqrt(float(d))) @ K[:seen + b].T
                    z += torch.full_like(z, float("-inf")).triu_(seen + a + 1)
                    at = torch.logsumexp(z, 1)
                    out[start[r] + a:start[r] + b, h] = torch.exp(z - at[:, None]) @ V[:seen + b]
                    lse[start[r] + a:start[r] + b, h] = at
    return {"out": out, "lse": lse}
