"""Cases for what stands between a layer's projections and its attention, and for
the COLD cache held in 4 bits: norms of queries and keys with the rotation of
positions (gk_qk_norm_rope), the same with the append to the paged cache
(gk_append_qkv, bf16 and 4-bit rows), reading tokens back (gk_read_kv) and decode
over 4-bit rows (gk_decode_kv4).

run() computes each in its plain form, elementary torch operations in fp32, or,
where `own` is true, through the library's calls.  Every case is one layer of one
step.  Sizes follow the synthetic workloads of this repository (Llama-3.1-8B: 32
query heads on 8 KV heads of 128; Qwen-2.5-14B: 40 on 8; the tiny workload: 4 on 2
of 64) and a few generic ones.

A 4-bit row (one COLD slot of one layer) holds, for each KV head, the codes of K
then of V (d / 2 bytes each, eight channels a 32-bit word, the lowest nibble first;
word w holds channels 8w .. 8w + 7 at d = 64, and 8 (w / 2) + 64 (w % 2) .. + 7 at
d = 128), then for each KV head the bf16 pairs (lowest value, span) of each 64
channels, K's then V's, and is padded to 16 bytes.  A value is
lowest + code * (span / 15).
"""
import random

import torch

own = False

#: query heads, KV heads, head dim
GEOMETRY = {"tiny": (4, 2, 64), "small": (16, 4, 64), "single": (8, 8, 64), "mqa": (8, 1, 128), "quad": (4, 4, 128),
            "pairs": (16, 8, 128), "llama8b": (32, 8, 128), "qwen14b": (40, 8, 128)}
EPS = 1e-6
#: a span of 64 channels below this is held as none
LEAST = 2.0 ** -100


def _case(name, **c):
    return dict(c, name=name) if name else c


def _rope(name, geo, n, norm=True, rot=None, inter=False, fused=True, far=131072, draw=1):
    return _case(name, op="rope", geo=geo, n=n, norm=norm, rot=GEOMETRY[geo][2] if rot is None else rot, inter=inter, fused=fused,
                 far=far, draw=draw)


def _append(name, geo, b, lo, hi, bits=16, page=16, norm=False, rot=None, inter=False, fused=True, k_out=False, far=131072, draw=1):
    return _case(name, op="append", geo=geo, b=b, lo=lo, hi=hi, bits=bits, page=page, norm=norm,
                 rot=GEOMETRY[geo][2] if rot is None else rot, inter=inter, fused=fused, k_out=k_out, far=far, draw=draw)


def _read(name, geo, n, bits=4, page=16, draw=1):
    return _case(name, op="read", geo=geo, n=n, bits=bits, page=page, draw=draw)


def _decode(name, geo, b, clo, chi, n_prefix=0, plo=0, phi=0, page=1, draw=1):
    return _case(name, op="decode", geo=geo, b=b, clo=clo, chi=chi, n_prefix=n_prefix, plo=plo, phi=phi, page=page, draw=draw)


def listed():
    return [
        # the queries and keys of one decode step of 64 requests, normed head by head (latency)
        _rope("norm_step", "qwen14b", 64),
        # a long prompt's queries and keys, views of one projection's output
        _rope("norm_prompt", "llama8b", 16384),
        # the tiny workload's decode step, half of each head's channels rotate, in neighbouring pairs (latency)
        _append("append_tiny", "tiny", 4, 1, 1, page=1, rot=32, inter=True, fused=False, far=4096),
        # a batch of fresh chat prompts goes into pages of 16, its rotated keys to the prompt attention too
        _append("append_prompts", "llama8b", 24, 64, 1500, norm=True, k_out=True),
        # a decode step of the eight-prefix workload into a 4-bit cache, and what the cache then holds
        _append("append4_step", "qwen14b", 368, 1, 1, bits=4, page=1),
        # a chunk of long prompts into a 4-bit cache, and what the cache then holds
        _append("append4_chunk", "llama8b", 2, 4000, 4096, bits=4, k_out=True),
        # a few tokens of the bf16 cache, to be promoted to a HOT prefix (latency)
        _read("read_few", "llama8b", 130, bits=16, page=1),
        # a 4-bit context that the next chunk of its prompt attends
        _read("read4_context", "llama8b", 12000),
        # the tiny workload's decode over 4-bit rows (latency)
        _decode("decode4_tiny", "tiny", 4, 1, 48, n_prefix=1, plo=64, phi=64),
        # one request far into a long context
        _decode("decode4_long", "llama8b", 1, 131072, 131072, page=16),
        # agents behind one long shared prefix, each with a history of its own
        _decode("decode4_agents", "llama8b", 64, 256, 2048, n_prefix=1, plo=16384, phi=16384),
        # the eight-prefix workload: the largest
        _decode("decode4_mixed", "qwen14b", 368, 128, 4096, n_prefix=8, plo=2048, phi=16384),
    ]


def _log(r, lo, hi):
    return lo if lo >= hi else min(hi, max(lo, round((lo + 1) * ((hi + 1) / (lo + 1)) ** r.random() - 1)))


def draw(rng):
    while True:
        seed, geo = rng.randrange(1 << 30), rng.choice(sorted(GEOMETRY))
        hq, hkv, d = GEOMETRY[geo]
        rot, inter, fused = rng.choice([d, d, d // 2, 16]), rng.random() < 0.3, rng.random() < 0.7
        norm, page, far = rng.random() < 0.5, rng.choice([1, 3, 16, 64]), rng.choice([4096, 40000, 131072])
        op = rng.random()
        if op < 0.2:
            c = _rope(None, geo, _log(rng, 1, 16384), norm, rot, inter, fused, far, seed)
        elif op < 0.55:
            # keys that meet 4 bits are not normed here: a norm's last bit, which sums in other orders give otherwise, can
            # move a value over the border of two codes, a whole step
            bits, hi = rng.choice([4, 16]), _log(rng, 1, 4000)
            c = _append(None, geo, _log(rng, 1, 400), rng.choice([0, hi // 2, hi]), hi, bits, page, norm and bits == 16, rot, inter, fused,
                        rng.random() < 0.5, far, seed)
            if not 1 <= sum(_lengths(c)) <= 16384:
                continue
        elif op < 0.7:
            c = _read(None, geo, _log(rng, 1, 16384), rng.choice([4, 4, 16]), page, seed)
        else:
            chi, phi = _log(rng, 1, 131072), _log(rng, 1, 16384) if rng.random() < 0.5 else 0
            c = _decode(None, geo, _log(rng, 1, 400), rng.choice([0, chi // 8, chi]), chi, rng.randrange(1, 9) if phi else 0, (phi + 1) // 2,
                        phi, page, seed)
            cold, which, prefixes = _contexts(c)
            # the plain form pads every request to the longest
            if c["b"] * max(cold) * hkv * d > 368 * 4096 * 8 * 128 or max(cold) * hq * c["b"] > 368 * 4096 * 40:
                continue
            if work(c)["flops"] > 8e10 or not sum(cold) + sum(prefixes):
                continue
        return c


def _lengths(c):
    """The new tokens of each request of an append."""
    r = random.Random(c["draw"])
    return [_log(r, c["lo"], c["hi"]) for _ in range(c["b"])]


def _contexts(c):
    """COLD tokens and prefix (-1: none) of each request of a decode step; the prefixes' lengths."""
    r = random.Random(c["draw"])
    prefixes = [_log(r, c["plo"], c["phi"]) for _ in range(c["n_prefix"])]
    cold = [_log(r, c["clo"], c["chi"]) for _ in range(c["b"])]
    return cold, [r.randrange(len(prefixes)) if prefixes else -1 for _ in cold], prefixes


def _row_bytes(hkv, d):
    return -(-(hkv * d + hkv * d // 8) // 16) * 16


def work(c):
    hq, hkv, d = GEOMETRY[c["geo"]]
    kv4 = hkv * (d + d // 8)     # codes, lowest values and spans of a token's K and V
    if c["op"] == "rope":
        n = c["n"]
        return {"bytes": n * (4 * (hq + hkv) * d + 4 + 4 * c["rot"]), "flops": n * (hq + hkv) * (3 * c["rot"] + 4 * d * c["norm"])}
    if c["op"] == "append":
        n = sum(_lengths(c))
        bytes_ = n * (4 * hq * d + 4 * hkv * d + (2 * hkv * d if c["k_out"] else 0) + 12 + 4 * c["rot"])
        # 4-bit rows are written, and read back as bf16
        bytes_ += n * (4 * hkv * d if c["bits"] == 16 else 2 * kv4 + 4 * hkv * d)
        return {"bytes": bytes_, "flops": n * ((hq + hkv) * (3 * c["rot"] + 4 * d * c["norm"]) + (12 * hkv * d if c["bits"] == 4 else 0))}
    if c["op"] == "read":
        n = c["n"]
        return {"bytes": n * ((kv4 if c["bits"] == 4 else 4 * hkv * d) + 4 * hkv * d + 8), "flops": n * 4 * hkv * d}
    cold, which, prefixes = _contexts(c)
    used = sum(lp for p, lp in enumerate(prefixes) if p in which)
    seen = sum(cold) + sum(prefixes[p] for p in which if p >= 0)
    return {"bytes": c["b"] * (4 * hq * d + 4 * hq) + 4 * used * hkv * d + sum(cold) * kv4 + sum(-(-n // c["page"]) for n in cold) * 4,
            "flops": 4 * d * hq * seen}


# ---- 4-bit rows -------------------------------------------------------------------------------
def _codes(x):
    """bf16 values [..., d] (as fp32) -> codes, lowest value and span of each 64 channels."""
    x = x.unflatten(-1, (-1, 64))
    lo = x.amin(-1, keepdim=True)
    span = (x.amax(-1, keepdim=True) - lo).to(torch.bfloat16).float()
    span = torch.where(span < LEAST, 0, span)
    code = ((x - lo) * 15 / span).round().clamp(max=15)
    return torch.where(span > 0, code, 0).to(torch.uint8).flatten(-2), lo[..., 0], span[..., 0]


def _pack(k, v):
    """bf16 K, V [n, heads, d] -> rows [n, bytes]."""
    n, heads, d = k.shape
    code, lo, span = _codes(torch.stack([k, v], 2).float())
    word = code.unflatten(-1, (-1, 8, 8)).transpose(-3, -2).flatten(-3).unflatten(-1, (-1, 2))
    data = (word[..., 0] + word[..., 1] * 16).reshape(n, -1)
    scale = torch.stack([lo, span], -1).to(torch.bfloat16).view(torch.uint8).reshape(n, -1)
    rows = torch.zeros(n, _row_bytes(heads, d), dtype=torch.uint8, device=k.device)
    rows[:, :data.shape[1]] = data
    rows[:, data.shape[1]:data.shape[1] + scale.shape[1]] = scale
    return rows


def _unpack(rows, heads, d):
    """rows [..., bytes] -> K, V [..., heads, d] in fp32."""
    data = rows[..., :heads * d].unflatten(-1, (heads, 2, d // 2))
    code = torch.stack([data & 15, data >> 4], -1).flatten(-2).unflatten(-1, (8, d // 64, 8)).transpose(-3, -2).float()
    scale = rows[..., heads * d:heads * d + heads * d // 8].contiguous().view(torch.bfloat16).float()
    scale = scale.unflatten(-1, (heads, 2, d // 64, 1, 1, 2))
    value = code.mul_(scale[..., 1] / 15).add_(scale[..., 0])
    return value.flatten(-3).unbind(-2)


# ---- states -----------------------------------------------------------------------------------
class _Handles:
    """The library's pool (and plan) over a state's storage, for as long as the state lives."""

    def __init__(self, gk, pool):
        self.gk, self.pool, self.plan = gk, pool, None

    def __del__(self):
        if self.plan:
            self.gk.gk_plan_destroy(self.plan)
        self.gk.gk_pool_destroy(self.pool)


def _values(g, *shape):
    """Keys or values: every channel with an offset of its own."""
    x = torch.randn(*shape, generator=g, device="cuda")
    return x.add_(0.4 * torch.randn(shape[-1], generator=g, device="cuda")).to(torch.bfloat16)


def _new_tokens(c, g, n, parts):
    """`parts` heads of n tokens each: rows of one projection's output, or tensors of their own."""
    d = GEOMETRY[c["geo"]][2]
    if c["fused"]:
        row = _values(g, n, sum(parts) * d)
        return [x.view(n, -1, d) for x in row.split([p * d for p in parts], 1)]
    return [_values(g, n, p * d).view(n, p, d) for p in parts]


def _rotation(c, g):
    """cos and sin of every position, and the norms' weights."""
    r, d = c["rot"], GEOMETRY[c["geo"]][2]
    turn = torch.arange(c["far"], dtype=torch.float64, device="cuda")[:, None] * 500000.0 ** (
        -2 * torch.arange(r // 2, dtype=torch.float64, device="cuda") / r)
    weights = [(1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16) if c["norm"] else None for _ in range(2)]
    return torch.cat([turn.cos(), turn.sin()], 1).float(), weights


def _places(lengths, page, g, spare):
    """Slots of packed tokens whose requests fill shuffled pages from their first place on; pages in all; the table."""
    pages = [-(-n // page) for n in lengths]
    blocks = sum(pages) + spare
    width, many = max([1] + pages), len(lengths)
    held = torch.tensor(pages, device="cuda")
    table = torch.zeros(many, width, dtype=torch.int32, device="cuda")
    order = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    table[torch.arange(width, device="cuda")[None] < held[:, None]] = order[:sum(pages)]
    n = torch.tensor(lengths, device="cuda")
    row = torch.repeat_interleave(torch.arange(many, device="cuda"), n)
    at = torch.arange(len(row), device="cuda") - (n.cumsum(0) - n)[row]
    return table[row, at // page].long() * page + at % page, blocks, table, at, row


def _pool(c, s, hot_tokens, blocks):
    """The library's pool over a state's storage."""
    from paged_kv_cache_pool_gb300 import binding as gk
    hq, hkv, d = GEOMETRY[c["geo"]]
    hot = [s.get("hot_k"), s.get("hot_v")]
    if hot[0] is None:
        hot = s["hot"] = [torch.zeros(hot_tokens * hkv * d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    size = (1, hq, hkv, d, hot_tokens, blocks * c["page"], c["page"], 0)
    if "rows" in s:
        return _Handles(gk, gk.gk_pool_create_kv4(*size, *hot, s["rows"]))
    return _Handles(gk, gk.gk_pool_create(*size, *hot, s["cold_k"], s["cold_v"]))


def _prepare_rope(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    hq, hkv, d = GEOMETRY[c["geo"]]
    s = {"c": c}
    s["table"], s["weights"] = _rotation(c, g)
    s["q"], s["k"] = _new_tokens(c, g, c["n"], (hq, hkv))
    # tokens of several requests, one after another: runs of positions
    s["positions"] = torch.randint(0, c["far"], (c["n"],), generator=g, device="cuda", dtype=torch.int32) if c["n"] <= 512 else (
        torch.arange(c["n"], dtype=torch.int32, device="cuda") + c["far"] // 3) % c["far"]
    s["q_out"], s["k_out"] = (torch.empty(c["n"], h, d, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv))
    if own:
        s["cold_k"], s["cold_v"] = (torch.zeros(1, 64, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        s["handles"] = h = _pool(dict(c, page=1), s, 64, 64)
        s["rope"] = h.gk.Rope(s["table"], c["rot"], c["inter"], *s["weights"], EPS)
    return s


def _prepare_append(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    hq, hkv, d = GEOMETRY[c["geo"]]
    lengths = _lengths(c)
    n = sum(lengths)
    s = {"c": c}
    s["table"], s["weights"] = _rotation(c, g)
    s["q"], s["k"], s["v"] = _new_tokens(c, g, n, (hq, hkv, hkv))
    if max(lengths) > 1:
        s["slots"], blocks, _, at, row = _places(lengths, c["page"], g, 3)
        s["positions"] = ((at + 977 * row) % c["far"]).to(torch.int32)
    else:   # a decode step: the token stands anywhere in its page
        blocks = n + 3
        place = torch.randint(0, c["page"], (n,), generator=g, device="cuda")
        s["slots"] = torch.randperm(blocks, generator=g, device="cuda")[:n] * c["page"] + place
        s["positions"] = torch.randint(0, c["far"], (n,), generator=g, device="cuda", dtype=torch.int32)
    s["q_out"], s["k_out"] = (torch.empty(n, h, d, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv))
    if c["bits"] == 4:
        s["rows"] = torch.zeros(1, blocks * c["page"], _row_bytes(hkv, d), dtype=torch.uint8, device="cuda")
        s["read_k"], s["read_v"] = torch.empty_like(s["k_out"]), torch.empty_like(s["k_out"])
    else:
        s["cold_k"], s["cold_v"] = (torch.zeros(1, blocks * c["page"], hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    if own:
        s["handles"] = h = _pool(c, s, 64, blocks)
        s["rope"] = h.gk.Rope(s["table"], c["rot"], c["inter"], *s["weights"], EPS)
    return s


def _prepare_read(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    hq, hkv, d = GEOMETRY[c["geo"]]
    s = {"c": c}
    s["slots"], blocks, _, _, _ = _places([c["n"]], c["page"], g, 5)
    k, v = (_values(g, blocks * c["page"], hkv * d).view(-1, hkv, d) for _ in range(2))
    if c["bits"] == 4:
        s["rows"] = _pack(k, v)[None]
    else:
        s["cold_k"], s["cold_v"] = k[None], v[None]
    s["read_k"], s["read_v"] = (torch.empty(c["n"], hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    if own:
        s["handles"] = _pool(c, s, 64, blocks)
    return s


def _prepare_decode(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    hq, hkv, d = GEOMETRY[c["geo"]]
    cold, which, prefixes = _contexts(c)
    b = c["b"]
    s = {"c": c, "cold": cold, "which": which, "prefixes": prefixes}
    # HOT: prefix p owns rows [base, base + length) of every head, laid out [head][token][d] (one layer)
    s["bases"] = [sum(prefixes[:p]) for p in range(len(prefixes))]
    hot = max(1, sum(prefixes))
    s["hot_k"], s["hot_v"] = _values(g, hot * hkv, d), _values(g, hot * hkv, d)
    _, blocks, s["table"], _, _ = _places(cold, c["page"], g, 7)
    s["rows"] = _pack(*(_values(g, blocks * c["page"], hkv * d).view(-1, hkv, d) for _ in range(2)))[None]
    s["q"] = (1.5 * torch.randn(b, hq, d, generator=g, device="cuda")).to(torch.bfloat16)
    s["out"] = torch.empty(b, hq, d, dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.empty(b, hq, device="cuda")
    s["cold_len"] = torch.tensor(cold, device="cuda")
    if prefixes:
        # the requests of each prefix, padded to the most, and each request's place there
        of = [[r for r in range(b) if which[r] == p] for p in range(len(prefixes))]
        most = max(len(m) for m in of)
        s["members"] = torch.tensor([m + [0] * (most - len(m)) for m in of], device="cuda")
        s["member_of"] = torch.tensor([which[r] * most + of[which[r]].index(r) for r in range(b)], device="cuda")
        s["prefix_base"], s["prefix_len"] = (torch.tensor(x, device="cuda") for x in (s["bases"], prefixes))
    if own:
        s["handles"] = h = _pool(c, s, hot, blocks)
        for base, lp in zip(s["bases"], prefixes):
            assert h.gk.gk_prefix_alloc(h.pool, lp) == base
        s["batch"] = h.gk.Batch([s["bases"][p] if p >= 0 else -1 for p in which], [prefixes[p] if p >= 0 else 0 for p in which], cold,
                                s["table"], s["table"].shape[1])
        h.plan = h.gk.gk_plan_build(h.pool, s["batch"], torch.cuda.current_stream())
    return s


def prepare(case, seed):
    return {"rope": _prepare_rope, "append": _prepare_append, "read": _prepare_read, "decode": _prepare_decode}[case["op"]](case, seed)


# ---- plain forms ------------------------------------------------------------------------------
def _rotated(s, x, weight):
    """Normed (where there is a weight) and rotated heads of bf16 x [n, heads, d], in fp32."""
    c = s["c"]
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    r = c["rot"]
    row = s["table"][s["positions"].long()][:, None]
    cos, sin = row[..., :r // 2], row[..., r // 2:]
    if c["inter"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _plain_append(s):
    c = s["c"]
    s["q_out"].copy_(_rotated(s, s["q"], s["weights"][0]))
    k = _rotated(s, s["k"], s["weights"][1]).to(torch.bfloat16)
    if c["k_out"]:
        s["k_out"].copy_(k)
    if c["bits"] == 4:
        s["rows"][0, s["slots"]] = _pack(k, s["v"])
        return _plain_read(s)
    s["cold_k"][0, s["slots"]] = k
    s["cold_v"][0, s["slots"]] = s["v"]


def _plain_read(s):
    c = s["c"]
    hq, hkv, d = GEOMETRY[c["geo"]]
    k, v = _unpack(s["rows"][0, s["slots"]], hkv, d) if c["bits"] == 4 else (s["cold_k"][0, s["slots"]], s["cold_v"][0, s["slots"]])
    s["read_k"].copy_(k)
    s["read_v"].copy_(v)


def _attend(q, k, v, seen):
    """Partial states of rows q [.., m, d] over k, v [.., n, d], the first `seen` of them: sums, largest scores, totals."""
    score = (q @ k.transpose(-1, -2)).mul_(q.shape[-1] ** -0.5)
    score.masked_fill_(torch.arange(k.shape[-2], device="cuda") >= seen, float("-inf"))
    top = score.amax(-1, keepdim=True)
    weight = score.sub_(top.clamp(min=-1e30)).exp_()
    return weight @ v, top, weight.sum(-1, keepdim=True)


def _plain_decode(s):
    c = s["c"]
    hq, hkv, d = GEOMETRY[c["geo"]]
    b, g = c["b"], hq // hkv
    q = s["q"].float().view(b, hkv, g, d)
    at = torch.arange(max(1, max(s["cold"])), device="cuda")
    slot = s["table"].long()[:, at // c["page"]] * c["page"] + at % c["page"]
    k, v = _unpack(s["rows"][0, slot], hkv, d)
    o, top, total = _attend(q, k.transpose(1, 2), v.transpose(1, 2), s["cold_len"].view(b, 1, 1, 1))
    if s["prefixes"]:
        # every prefix once, for all rows that share it
        lp = s["prefix_len"]
        t = torch.arange(max(s["prefixes"]), device="cuda").minimum(lp[:, None] - 1)[:, None]
        row = s["prefix_base"].view(-1, 1, 1) * hkv + torch.arange(hkv, device="cuda").view(1, -1, 1) * lp.view(-1, 1, 1) + t
        rows = q[s["members"]].transpose(1, 2).flatten(2, 3)
        states = _attend(rows, s["hot_k"][row].float(), s["hot_v"][row].float(), lp.view(-1, 1, 1, 1))
        o2, top2, total2 = (x.unflatten(2, (-1, g)).transpose(1, 2).flatten(0, 1)[s["member_of"]] for x in states)
        both = torch.maximum(top, top2)
        w, w2 = (top - both).exp(), (top2 - both).exp()
        o, top, total = o * w + o2 * w2, both, total * w + total2 * w2
    s["out"].copy_((o / total.where(total > 0, 1)).view(b, hq, d))
    s["lse"].copy_((top + total.log()).view(b, hq))
    return {"out": s["out"], "lse": s["lse"]}


# ---- one pass ---------------------------------------------------------------------------------
def _append_out(s):
    out = {"q": s["q_out"]}
    if s["c"]["k_out"]:
        out["k"] = s["k_out"]
    return {**out, **({"cache_k": s["read_k"], "cache_v": s["read_v"]} if s["c"]["bits"] == 4 else {"cache_k": s["cold_k"], "cache_v": s["cold_v"]})}


def run(state):
    s = state
    op = s["c"]["op"]
    if own:
        h, stream = s["handles"], torch.cuda.current_stream()
        if op == "rope":
            h.gk.gk_qk_norm_rope(h.pool, stream, s["rope"], s["positions"], s["q"], s["k"], s["q_out"], s["k_out"])
        elif op == "append":
            h.gk.gk_append_qkv(h.pool, stream, 0, s["rope"], s["positions"], s["slots"], s["q"], s["k"], s["v"], s["q_out"],
                               s["k_out"] if s["c"]["k_out"] else None)
        elif op == "decode":
            s["batch"].set_device(d_q=s["q"], d_lse=s["lse"])
            h.gk.gk_decode_kv4(h.pool, stream, 0, s["batch"], h.plan, s["out"])
        if op == "read" or op == "append" and s["c"]["bits"] == 4:
            h.gk.gk_read_kv(h.pool, stream, 0, s["slots"], s["read_k"], s["read_v"])
    elif op == "rope":
        s["q_out"].copy_(_rotated(s, s["q"], s["weights"][0]))
        s["k_out"].copy_(_rotated(s, s["k"], s["weights"][1]))
    elif op == "append":
        _plain_append(s)
    elif op == "read":
        _plain_read(s)
    else:
        _plain_decode(s)
    if op == "rope":
        return {"q": s["q_out"], "k": s["k_out"]}
    if op == "append":
        return _append_out(s)
    return {"k": s["read_k"], "v": s["read_v"]} if op == "read" else {"out": s["out"], "lse": s["lse"]}


# ---- in 64 bits -------------------------------------------------------------------------------
def _turned(s, x, weight):
    """One head at a time: the norm, then each pair as a complex number times that of its position."""
    c = s["c"]
    x = x.double().clone()
    if weight is not None:
        x *= weight.double() / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS)
    r = c["rot"]
    row = s["table"].double()[s["positions"].long()]
    by = torch.complex(row[:, :r // 2], row[:, r // 2:])
    first = torch.arange(r // 2, device="cuda") * (2 if c["inter"] else 1)
    second = first + (1 if c["inter"] else r // 2)
    for h in range(x.shape[1]):
        z = torch.complex(x[:, h, first], x[:, h, second]) * by
        x[:, h, first], x[:, h, second] = z.real, z.imag
    return x


def _stored(x):
    """What 4 bits hold of bf16 x [n, heads, d]."""
    x = x.double()
    out = torch.empty_like(x)
    for a in range(0, x.shape[-1], 64):
        part = x[..., a:a + 64]
        low = part.min(-1, keepdim=True).values
        span = (part.max(-1, keepdim=True).values - low).to(torch.bfloat16).double()
        span = torch.where(span < LEAST, torch.inf, span)
        code = torch.round((part - low) * 15 / span).clamp(0, 15)
        out[..., a:a + 64] = low + torch.where(code > 0, code * span / 15, 0)
    return out


def _held(rows, head, d, hkv):
    """K and V of one head from rows [n, bytes], channel by channel of the layout."""
    base = rows[:, head * d:(head + 1) * d].long()
    pairs = rows[:, hkv * d:].contiguous().view(torch.bfloat16).double()
    groups, out = d // 64, []
    for part in range(2):
        x = torch.empty(len(rows), d, dtype=torch.float64, device="cuda")
        for ch in range(d):
            word = ch // 8 if groups == 1 else 2 * (ch % 64 // 8) + ch // 64
            byte = base[:, part * d // 2 + word * 4 + ch % 8 // 2]
            at = ((head * 2 + part) * groups + ch // 64) * 2
            x[:, ch] = pairs[:, at] + (byte // 16 if ch % 2 else byte % 16) * pairs[:, at + 1] / 15
        out.append(x)
    return out


def exact(case, seed):
    """Each operator from its definition, in 64 bits; bf16 and 4-bit storage are part of what a cache holds."""
    c, hkv, d = case, *GEOMETRY[case["geo"]][1:]
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    if c["op"] == "rope":
        return {"q": _turned(s, s["q"], s["weights"][0]), "k": _turned(s, s["k"], s["weights"][1])}
    if c["op"] == "append":
        k = _turned(s, s["k"], s["weights"][1])
        out = {"q": _turned(s, s["q"], s["weights"][0]), **({"k": k} if c["k_out"] else {})}
        if c["bits"] == 4:
            return {**out, "cache_k": _stored(k.to(torch.bfloat16)), "cache_v": _stored(s["v"])}
        for name, x in (("cache_k", k), ("cache_v", s["v"].double())):
            out[name] = s["cold_k"].double()
            out[name][0, s["slots"]] = x
        return out
    if c["op"] == "read":
        if c["bits"] == 16:
            return {"k": s["cold_k"][0, s["slots"]].double(), "v": s["cold_v"][0, s["slots"]].double()}
        heads = [_held(s["rows"][0, s["slots"]], h, d, hkv) for h in range(hkv)]
        return {"k": torch.stack([x[0] for x in heads], 1), "v": torch.stack([x[1] for x in heads], 1)}
    hq, b = s["q"].shape[1], c["b"]
    out = torch.zeros(b, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((b, hq), float("-inf"), dtype=torch.float64, device="cuda")
    slots = [(s["table"][r].long()[:, None] * c["page"] + torch.arange(c["page"], device="cuda")).flatten()[:n] for r, n in enumerate(s["cold"])]
    for head in range(hkv):
        mine = slice(head * hq // hkv, (head + 1) * hq // hkv)
        hot = []
        for base, lp in zip(s["bases"], s["prefixes"]):
            a = base * hkv + head * lp
            hot.append((s["hot_k"][a:a + lp].double(), s["hot_v"][a:a + lp].double()))
        ends = [0]
        for n in s["cold"]:
            ends.append(ends[-1] + n)
        K4, V4 = _held(s["rows"][0, torch.cat(slots)], head, d, hkv)
        for r in range(b):
            keys, values = K4[ends[r]:ends[r + 1]], V4[ends[r]:ends[r + 1]]
            if s["which"][r] >= 0:
                keys, values = (torch.cat(x) for x in zip(hot[s["which"][r]], (keys, values)))
            if len(keys):
                z = s["q"][r, mine].double() @ keys.T / d ** 0.5
                lse[r, mine] = torch.logsumexp(z, 1)
                out[r, mine] = torch.exp(z - lse[r, mine][:, None]) @ values
    return {"out": out, "lse": lse}
