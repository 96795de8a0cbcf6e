"""gk_decode_kv4 against a 64-bit attention over what the rows hold: every geometry, lengths
from none to several pages and CTAs, prefixes, strides, bad blocks, special values, spans far
apart, graphs and streams, and whole steps from the projection on."""
import random

import numpy as np
import pytest

from kv4_ref import attend, bf16_value, check_attention, fields, values

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from paged_kv_cache_pool_gb300 import binding as gk  # noqa: E402
from paged_kv_cache_pool_gb300.engine import Engine  # noqa: E402

GEOMETRIES = [(d, g, hkv) for d, gs in ((64, (1, 2, 4)), (128, (1, 2, 4, 5, 8))) for g in gs for hkv in (1, 2, 3, 5, 8)]
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_pool_gb300 import build
    build.build()


def np64(x):
    return x.double().cpu().numpy()


class Step:
    """Requests with COLD tokens in 4-bit rows of one layer, some behind HOT prefixes; rows that hold no token are NaN."""

    def __init__(self, d, g, hkv, cold, prefixes=(), which=None, page=16, layers=2, layer=1, seed=0, scale=1.5, k=None, v=None, wide=0):
        rng = torch.Generator(device="cuda").manual_seed(seed)
        self.cold, self.layer, self.d, self.hkv, self.hq = list(cold), layer, d, hkv, g * hkv
        self.which = [-1] * len(cold) if which is None else which
        blocks = sum(-(-c // page) for c in cold) + 3
        hot = sum(prefixes) + 5
        self.eng = eng = Engine(layers, self.hq, hkv, d, hot, blocks * page, page, seed=11, kv_bits=4)
        # codes 15, lo and span NaN
        eng.cold.fill_(0xFF)
        eng.hot_k.fill_(float("nan"))
        eng.hot_v.fill_(float("nan"))
        offset = 0.4 * torch.randn(d, generator=rng, device="cuda")

        def rand(n):
            return (torch.randn(n, hkv, d, generator=rng, device="cuda") + offset).to(BF)
        self.bases, self.hot = [], []
        for lp in prefixes:
            self.bases.append(eng.prefix_alloc(lp))
            kv = rand(lp), rand(lp)
            eng.write_prefix(layer, self.bases[-1], lp, 0, *kv)
            self.hot.append(tuple(np64(x) for x in kv))
        self.seqs = [eng.seq_create() for _ in cold]
        slots, _ = eng.append_slots(np.repeat(np.asarray(self.seqs, np.int32), self.cold)) if sum(cold) else (np.zeros(0, np.int64), None)
        self.slots = eng.to_device(slots)
        n = len(slots)
        self.k, self.v = (rand(n) if x is None else x for x in (k, v))
        if n:
            eng.append_kv(layer, self.slots, self.k, self.v)
        width = max([1] + [-(-c // page) for c in cold]) + wide
        self.table = eng.to_device(eng.block_tables(self.seqs, width))
        self.batch = eng.batch([self.bases[w] if w >= 0 else -1 for w in self.which], [prefixes[w] if w >= 0 else 0 for w in self.which],
                               self.cold, self.table, width)
        self.q = (torch.randn(len(cold), self.hq, d, generator=rng, device="cuda") * scale).to(BF)
        self.out = torch.full((len(cold) + 1, self.hq, d), 7.0, dtype=BF, device="cuda")
        self.lse = torch.full((len(cold) + 1, self.hq), 7.0, device="cuda")
        self.plan = eng.plan(self.batch)

    def run(self, stream=None, lse=True):
        self.batch.set_device(d_q=self.q, d_lse=self.lse if lse else None)
        self.eng.decode_kv4(self.layer, self.batch, self.plan, self.out[:-1], stream)

    def want(self, requests=None):
        K, V, size = values(self.eng.cold[self.layer, self.slots].cpu().numpy(), self.hkv, self.d)
        at = np.cumsum([0] + self.cold)
        none = np.zeros((0, self.hkv, self.d))
        got = [attend(np64(self.q[r]), self.hot[self.which[r]] if self.which[r] >= 0 else (none, none),
                      tuple(x[at[r]:at[r + 1]] for x in (K, V, size))) for r in (range(len(self.cold)) if requests is None else requests)]
        return [np.stack(x) for x in zip(*got)]

    def check(self, what="", requests=None):
        torch.cuda.synchronize()
        assert self.eng.device_error() == gk.GK_OK
        assert (self.out[-1] == 7).all() and (self.lse[-1] == 7).all()
        if not self.cold:
            return
        at = slice(0, len(self.cold)) if requests is None else requests
        check_attention(np64(self.out[at]), np64(self.lse[at]), self.want(requests), what)

    def close(self):
        self.eng.close()
        torch.cuda.empty_cache()


@pytest.mark.parametrize("d,g,hkv", GEOMETRIES)
def test_geometries(d, g, hkv):
    """Lengths around a warp's stage and a page, none and one, behind a prefix and not."""
    s = Step(d, g, hkv, [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 0, 257], [70], [-1, -1, 0, -1, 0, -1, 0, -1, 0, -1, 0, -1, 0, -1])
    s.run()
    s.check()
    s.close()


@pytest.mark.parametrize("page", [1, 2, 3, 7, 16, 64])
@pytest.mark.parametrize("d", [64, 128])
def test_pages(d, page):
    s = Step(d, 4, 2, [5, 129, 1, 64, 333, 48], page=page, seed=page)
    s.run()
    s.check()
    s.close()


@pytest.mark.parametrize("cold", [[8000], [4096, 1, 0, 4095], [700] * 9, [64] * 200, [0, 0], [1], []])
def test_lengths(cold):
    """Requests over many CTAs, many over few, none at all."""
    s = Step(128, 4, 8, cold, seed=len(cold))
    s.run()
    s.check()
    s.close()


@pytest.mark.parametrize("d,g,hkv,requests", [(128, 4, 8, 1), (128, 5, 8, 1), (128, 5, 8, 2), (128, 8, 8, 3), (64, 2, 8, 1), (64, 4, 8, 3)])
def test_joins_of_many_states(d, g, hkv, requests):
    """From 16 to 192 rows of a hundred states and more, some behind a prefix: every number of blocks that shares a row's join."""
    s = Step(d, g, hkv, [9000] * requests, [700], [0] + [-1] * (requests - 1), seed=g)
    s.run()
    s.check()
    s.close()


def test_random_steps():
    rnd = random.Random(4)
    for i in range(40):
        d = rnd.choice([64, 128])
        g, hkv = rnd.choice([1, 2, 4] if d == 64 else [1, 2, 4, 5, 8]), rnd.randint(1, 8)
        hi = rnd.choice([3, 40, 300, 1500])
        b = rnd.randint(1, 12)
        prefixes = [rnd.randint(1, 500) for _ in range(rnd.randint(0, 3))]
        s = Step(d, g, hkv, [rnd.randint(0, hi) for _ in range(b)], prefixes, [rnd.randint(-1, len(prefixes) - 1) for _ in range(b)],
                 rnd.choice([1, 3, 16]), seed=i, scale=rnd.choice([0.1, 1.5, 12.0]), wide=rnd.choice([0, 5]))
        s.run()
        s.check(f"step {i}")
        s.close()


def test_many_requests_behind_prefixes():
    """The rows of a prefix stacked over tensor-core items, joined with COLD states."""
    rnd = random.Random(1)
    which = [i % 3 for i in range(90)]
    s = Step(128, 5, 8, [rnd.randint(0, 200) for _ in which], [1000, 130, 2048], which, page=1)
    s.run()
    s.check(requests=[0, 1, 2, 45, 88, 89])
    s.close()


def test_without_lse_and_again():
    """No lse asked for; a second call gives the same bits; a planned update of the same plan serves the next step."""
    s = Step(128, 4, 8, [3000, 5, 0, 64], [200], [0, -1, 0, -1])
    s.run()
    first, lse = s.out.clone(), s.lse.clone()
    s.out[:-1].fill_(3)
    s.lse.fill_(7)
    s.run(lse=False)
    assert torch.equal(s.out, first) and (s.lse == 7).all()
    s.cold = [2999, 4, 0, 64]
    keep = torch.ones(len(s.slots), dtype=torch.bool, device="cuda")
    keep[2999], keep[3004] = False, False
    s.slots = s.slots[keep]
    s.batch = s.eng.batch([s.bases[0], -1, s.bases[0], -1], [200, 0, 200, 0], s.cold, s.table, s.table.shape[1])
    s.eng.plan(s.batch, plan=s.plan)
    s.run()
    s.check()
    assert not torch.equal(s.out, first)
    s.close()


def test_bad_blocks_count_as_zeros():
    """An id outside the pool is reported, and its tokens count as zero K and V."""
    for bad in (-1, 1 << 30, 9):
        s = Step(64, 2, 2, [40, 20], page=16)
        assert s.eng.cold_slots // 16 == 8
        s.run()
        s.check()
        table = s.table.cpu().numpy().copy()
        table[0, 1] = min(bad, 8) if bad == 9 else bad
        s.table.copy_(torch.from_numpy(table))
        s.run()
        torch.cuda.synchronize()
        assert s.eng.device_error() == gk.GK_ERR_DEVICE_BOUNDS and s.eng.device_error() == gk.GK_OK
        K, V, size = (x[:40].copy() for x in values(s.eng.cold[1, s.slots].cpu().numpy(), 2, 64))
        K[16:32], V[16:32], size[16:32] = 0, 0, 0
        none = np.zeros((0, 2, 64))
        O, L, E = attend(np64(s.q[0]), (none, none), (K, V, size))
        check_attention(np64(s.out[0]), np64(s.lse[0]), (O, L, E))
        s.close()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [1, 4, 8, 32])
def test_bad_blocks_in_both_ways_of_copying(d, page):
    """Bad ids among good ones, alone, first and last of a stage, with pages of few tokens and of many."""
    s = Step(d, 2, 3, [70, 33, page], page=page)
    s.run()
    s.check()
    table = s.table.cpu().numpy().copy()
    bad = [(0, 0), (0, (69 // page)), (0, min(33, 69) // page), (1, 32 // page), (2, 0)]
    for r, b in bad:
        table[r, b] = 1 << 30 if b % 2 else -7
    s.table.copy_(torch.from_numpy(table))
    s.run()
    torch.cuda.synchronize()
    assert s.eng.device_error() == gk.GK_ERR_DEVICE_BOUNDS
    K, V, size = (x.copy() for x in values(s.eng.cold[1, s.slots].cpu().numpy(), 3, d))
    at = np.cumsum([0, 70, 33, page])
    for r, b in bad:
        i = slice(at[r] + b * page, min(at[r + 1], at[r] + (b + 1) * page))
        K[i], V[i], size[i] = 0, 0, 0
    none = np.zeros((0, 3, d))
    for r in range(3):
        i = slice(at[r], at[r + 1])
        check_attention(np64(s.out[r]), np64(s.lse[r]), attend(np64(s.q[r]), (none, none), (K[i], V[i], size[i])), f"request {r}")
    s.close()


@pytest.mark.parametrize("hkv", [1, 8])
def test_more_segments_than_a_cta_keeps(hkv):
    """Thousands of requests of a few tokens: a CTA's list of segments is longer than what it keeps of it."""
    rnd = random.Random(3)
    b = 11000 if hkv == 8 else 80000
    s = Step(64, 1, hkv, [rnd.randint(1, 4) for _ in range(b)], page=2, layers=1, layer=0)
    begin, segs = gk.gk_plan_segments(s.plan)
    assert np.diff(begin).max() > 34 and len(segs) == b
    s.run()
    some = sorted(rnd.sample(range(b), 300)) + [b - 1]
    s.check(requests=some)
    s.close()


def test_rows_behind_a_request_do_not_matter():
    """Pages' places past a request's length, and blocks that no table names, hold NaN; block ids past the length are never read."""
    s = Step(128, 4, 2, [17, 33, 1], page=16, wide=3)
    s.table[0, 2:], s.table[1, 3:], s.table[2, 1:] = 1 << 30, -5, 77777
    s.run()
    s.check()
    s.close()


@pytest.mark.parametrize("d", [64, 128])
def test_nan_keys_values_and_queries(d):
    """A key held as NaN makes the rows that attend it NaN, a value its 64 channels, a query its own row."""
    s = Step(d, 4, 2, [70, 70, 70, 70, 70])
    s.run()
    torch.cuda.synchronize()
    out, lse = s.out.clone(), s.lse.clone()
    s.k[70 + 69, 1, 3] = float("inf")            # request 1, KV head 1
    s.v[2 * 70 + 3, 0, d - 1] = float("nan")     # request 2, KV head 0, last group
    s.eng.append_kv(1, s.slots, s.k, s.v)
    s.q[3, 5, 0] = float("nan")
    s.q[4, 0, 1], s.q[4, 7, d - 1] = float("inf"), -float("inf")
    s.run()
    torch.cuda.synchronize()
    nan, nan_l = torch.zeros_like(out, dtype=torch.bool), torch.zeros_like(lse, dtype=torch.bool)
    nan[1, 4:] = nan[3, 5] = nan[4, 0] = nan[4, 7] = True
    nan[2, :4, d - 64:] = True
    nan_l[1, 4:] = nan_l[3, 5] = nan_l[4, 0] = nan_l[4, 7] = True
    assert torch.equal(s.out.isnan(), nan) and torch.equal(s.lse.isnan(), nan_l)
    assert torch.equal(s.out[~nan], out[~nan]) and torch.equal(s.lse[~nan_l], lse[~nan_l])
    s.close()


@pytest.mark.parametrize("d", [64, 128])
def test_nan_in_requests_over_many_ctas(d):
    """A NaN in one of many partial states reaches the joined row."""
    s = Step(d, 4, 2, [5000, 5000], [150], [0, -1])
    s.run()
    s.check()
    for r in (0, 1):
        s.k[5000 * r + 2500, 0, 3] = float("nan")
    s.eng.append_kv(1, s.slots, s.k, s.v)
    s.run()
    torch.cuda.synchronize()
    assert s.out[:2, :4].isnan().all() and s.lse[:2, :4].isnan().all()
    assert s.out[:2, 4:].isfinite().all() and s.lse[:2, 4:].isfinite().all()
    s.close()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("power", [-60, -20, 20, 60])
def test_spans_far_apart(d, power):
    """Values whose size grows, shrinks or jumps by powers of two along a request; keys and queries of any size."""
    n = 400
    rng = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.randn(3 * n, 2, d, generator=rng, device="cuda") for _ in range(2))
    ramp = torch.linspace(0, power, n, device="cuda").round()
    v[:n] *= torch.exp2(ramp)[:, None, None]
    v[n:2 * n] *= torch.exp2(ramp.flip(0))[:, None, None]
    v[2 * n + 137] *= 2.0 ** power
    v[2 * n:, 1] *= 2.0 ** power
    s = Step(d, 2, 2, [n, n, n], k=k.to(BF), v=v.to(BF))
    s.run()
    s.check()
    # queries 2^power long against keys 2^-power: the same scores
    t = Step(d, 2, 2, [n, n, n], k=(k * 2.0 ** -power).to(BF), v=v.to(BF))
    t.q.copy_(s.q.float() * 2.0 ** power)
    t.run()
    t.check()
    s.close()
    t.close()


def test_peaked_and_flat_scores():
    """One key takes all the weight; all keys alike; scores far apart in both signs."""
    rng = torch.Generator(device="cuda").manual_seed(3)
    n, d = 300, 128
    k, v = (torch.randn(3 * n, 1, d, generator=rng, device="cuda").to(BF) for _ in range(2))
    s = Step(d, 8, 1, [n, n, n], k=k, v=v)
    k[n:2 * n] = k[n]
    s.eng.append_kv(1, s.slots, k, v)
    s.q[0] = (8 * k[150]).expand(8, d)
    s.q[2] *= 20
    s.run()
    s.check()
    s.close()


def test_constant_groups_and_zeros():
    """Spans of 0: keys and values that are all lowest value."""
    n, d = 90, 128
    k = torch.ones(2 * n, 2, d, device="cuda") * torch.arange(2 * n, device="cuda")[:, None, None] / 64
    v = torch.zeros(2 * n, 2, d, device="cuda")
    v[n:] = 2.5
    s = Step(d, 2, 2, [n, n], k=k.to(BF), v=v.to(BF))
    s.run()
    s.check()
    assert (s.out[0] == 0).all() and (s.out[1] == 2.5).all()
    s.close()


def test_offsets_past_32_bits():
    """A request whose pages lie behind 2^32 bytes of rows, second layer."""
    eng = Engine(2, 32, 8, 128, 64, 1 << 21, 16, kv_bits=4)
    filler = eng.seq_create()
    eng.append_slots(np.full((1 << 21) - 320, filler, np.int32))
    seq = eng.seq_create()
    slots, _ = eng.append_slots(np.full(300, seq, np.int32))
    assert slots.min() * 1152 > 1 << 31
    rng = torch.Generator(device="cuda").manual_seed(5)
    k, v = (torch.randn(300, 8, 128, generator=rng, device="cuda").to(BF) for _ in range(2))
    eng.append_kv(1, eng.to_device(slots), k, v)
    q = torch.randn(1, 32, 128, generator=rng, device="cuda").to(BF)
    table = eng.to_device(eng.block_tables([seq]))
    batch = eng.batch([-1], [0], [300], table, table.shape[1])
    out, lse = torch.empty(1, 32, 128, dtype=BF, device="cuda"), torch.empty(1, 32, device="cuda")
    batch.set_device(d_q=q, d_lse=lse)
    eng.decode_kv4(1, batch, eng.plan(batch), out)
    K, V, size = values(eng.cold[1, eng.to_device(slots)].cpu().numpy(), 8, 128)
    none = np.zeros((0, 8, 128))
    check_attention(np64(out[0]), np64(lse[0]), attend(np64(q[0]), (none, none), (K, V, size)))
    assert eng.device_error() == gk.GK_OK
    eng.close()
    torch.cuda.empty_cache()


def test_captured_and_on_another_stream():
    """One plan in two captured graphs, replayed on new queries and keys; an eager call on a side stream."""
    s = Step(128, 4, 8, [900, 33, 0, 700], [300], [0, -1, 0, -1])
    s.run()
    s.check()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s.run(torch.cuda.current_stream())
        graphs.append(graph)
    for i, graph in enumerate((graphs[0], graphs[1], graphs[0])):
        s.q.mul_(-1)
        s.k.copy_(s.k.roll(1, 0))
        s.eng.append_kv(1, s.slots, s.k, s.v)
        s.out[:-1].fill_(3)
        graph.replay()
        s.check(f"replay {i}")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s.out[:-1].fill_(3)
    side.wait_stream(torch.cuda.current_stream())
    s.run(side)
    side.synchronize()
    s.check("side stream")
    s.close()


def test_two_pools_at_once():
    """Two pools' steps on two streams."""
    a, b = Step(128, 4, 8, [5000, 100], seed=1), Step(64, 4, 2, [3000, 7], [500], [0, -1], seed=2)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, st in zip((a, b), streams):
            s.run(st)
    torch.cuda.synchronize()
    a.check("first")
    b.check("second")
    a.close()
    b.close()


def test_pools_of_more_and_fewer_kv_heads():
    """Pools whose heads share a kernel but whose CTAs take different shared memory, in turn."""
    steps = [Step(128, 4, hkv, [300, 40], seed=hkv) for hkv in (8, 1, 5)]
    for s in steps + steps:
        s.out[:-1].fill_(3)
        s.run()
        s.check(f"{s.hkv} KV heads")
    for s in steps:
        s.close()


def test_steps_from_the_projection_on():
    """Prompts and decode steps over a 4-bit cache as an engine runs them: slots, norm + rotation + append, prompt attention over the
    bf16 keys, then steps of decode with a forked request, each against 64 bits."""
    d, hq, hkv, layers, page = 128, 8, 2, 2, 4
    eng = Engine(layers, hq, hkv, d, 512, 200 * page, page, seed=3, kv_bits=4)
    rng = torch.Generator(device="cuda").manual_seed(9)
    table = eng.rope_table(4096)
    ropes = [eng.rope(table, False, *[(1 + 0.2 * torch.randn(d, generator=rng, device="cuda")).to(BF) for _ in range(2)]) for _ in range(layers)]
    lens = [50, 7, 129]
    seqs = [eng.seq_create() for _ in lens]
    slots, _ = eng.append_slots(np.repeat(np.asarray(seqs, np.int32), lens))
    d_slots, T = eng.to_device(slots), sum(lens)
    pos = torch.cat([torch.arange(n, dtype=torch.int32, device="cuda") for n in lens])

    def qkv(n):
        row = torch.randn(n, (hq + 2 * hkv) * d, generator=rng, device="cuda").to(BF)
        return [x.unflatten(1, (-1, d)) for x in row.split([hq * d, hkv * d, hkv * d], 1)]
    batch = eng.prompt_batch(lens)
    plan = eng.prompt_plan(batch)
    for layer in range(layers):
        q, k, v = qkv(T)
        k_out, out = torch.empty(T, hkv, d, dtype=BF, device="cuda"), torch.empty(T, hq, d, dtype=BF, device="cuda")
        eng.append_qkv(layer, ropes[layer], pos, d_slots, q, k, v, k_out=k_out)      # queries in place
        eng.prompt(layer, batch, plan, q, k_out, v, out)
        torch.cuda.synchronize()
        t0 = 0
        for n in lens:
            s = torch.einsum("ihd,jhd->hij", q[t0:t0 + n].double(), k_out[t0:t0 + n].double().repeat_interleave(hq // hkv, 1)) / d ** 0.5
            s += torch.full_like(s, float("-inf")).triu_(1)
            want = torch.einsum("hij,jhd->ihd", s.softmax(-1), v[t0:t0 + n].double().repeat_interleave(hq // hkv, 1))
            assert (out[t0:t0 + n].double() - want).abs().max() < 2e-2
            t0 += n
    # a prompt's context moves to a HOT prefix as bf16, and the next chunk attends it there
    base = eng.prefix_alloc(lens[2])
    for layer in range(layers):
        ck, cv = eng.read_kv(layer, d_slots[-lens[2]:])
        eng.write_prefix(layer, base, lens[2], 0, ck, cv)
    chunk = eng.prompt_batch([40], [base], [lens[2]])
    chunk_plan = eng.prompt_plan(chunk)
    q, k, v = qkv(40)
    out = torch.empty(40, hq, d, dtype=BF, device="cuda")
    eng.qk_norm_rope(ropes[1], torch.arange(lens[2], lens[2] + 40, dtype=torch.int32, device="cuda"), q, k)
    eng.prompt(1, chunk, chunk_plan, q, k, v, out)
    K, V = (torch.cat([a, b]).double().repeat_interleave(hq // hkv, 1) for a, b in ((ck, k), (cv, v)))
    s = torch.einsum("ihd,jhd->hij", q.double(), K) / d ** 0.5
    s += torch.full_like(s, float("-inf")).triu_(lens[2] + 1)
    assert (out.double() - torch.einsum("hij,jhd->ihd", s.softmax(-1), V)).abs().max() < 2e-2
    # decode: the first request is forked, so that its partial page is copied before the step writes into it
    seqs.append(eng.seq_fork(seqs[0]))
    lens.append(lens[0])
    none = np.zeros((0, hkv, d))
    plan = None
    for step in range(6):
        new, cow = eng.append_slots(seqs)
        assert (len(cow) > 0) == (step == 0)
        pos = eng.to_device(np.asarray(lens, np.int32))
        lens = [n + 1 for n in lens]
        tab = eng.block_tables(seqs)
        d_tab = eng.to_device(tab)
        b = eng.batch([-1] * 4, [0] * 4, lens, d_tab, tab.shape[1])
        plan = eng.plan(b, plan=plan)
        for layer in range(layers):
            q, k, v = qkv(4)
            out, lse = torch.empty(4, hq, d, dtype=BF, device="cuda"), torch.empty(4, hq, device="cuda")
            eng.append_qkv(layer, ropes[layer], pos, eng.to_device(new), q, k, v, d_cow=eng.to_device(cow.reshape(-1)) if len(cow) else None)
            qc = q.contiguous()
            b.set_device(d_q=qc, d_lse=lse)
            eng.decode_kv4(layer, b, plan, out)
            torch.cuda.synchronize()
            for r in range(4):
                at = torch.tensor([int(tab[r][t // page]) * page + t % page for t in range(lens[r])], device="cuda")
                K, V, size = values(eng.cold[layer, at].cpu().numpy(), hkv, d)
                check_attention(np64(out[r]), np64(lse[r]), attend(np64(qc[r]), (none, none), (K, V, size)), f"step {step} request {r}")
    # the fork and its parent hold the same first tokens and different last ones
    assert eng.device_error() == gk.GK_OK
    eng.close()


def test_refusals_with_storage():
    """What a pool with storage refuses before any launch."""
    s = Step(64, 2, 2, [40], page=1)

    def status(**change):
        b = gk.gk_batch.from_buffer_copy(s.batch.c)
        out = s.out.data_ptr()
        for k, v in change.items():
            if k == "out":
                out = v
            else:
                setattr(b, k, v)
        import ctypes
        return gk.lib().gk_decode_kv4(s.eng.pool, None, 1, ctypes.byref(b), s.plan, out)
    s.run()
    assert status() == gk.GK_OK
    p = s.q.data_ptr()
    for change in (dict(num_requests=2), dict(d_q=None), dict(out=None), dict(d_block_table=None), dict(max_blocks=39), dict(d_q=p + 2),
                   dict(out=p + 8), dict(d_lse=p + 2), dict(d_block_table=p + 1)):
        assert status(**change) == gk.GK_ERR_INVALID, change
    for change in (dict(d_new_k=p), dict(d_new_v=p)):
        assert status(**change) == gk.GK_ERR_UNSUPPORTED
    s.run()
    s.check()
    s.close()


@pytest.mark.parametrize("d,g", [(64, 1), (64, 2), (64, 4), (128, 1), (128, 4), (128, 5), (128, 8)])
@pytest.mark.parametrize("page,length", [(1, 70), (4, 70), (1, 33), (16, 37), (64, 31), (1, 17)])
def test_bad_last_block_of_a_request(d, g, page, length):
    """A request whose last token is in a bad block, in a stage that it does not fill, while the pool's first rows hold NaN: its
    places past the end must not bring any of them in."""
    s = Step(d, g, 2, [length] * 3, page=page, seed=page)
    table = s.table.cpu().numpy().copy()
    K, V, size = (x.copy() for x in values(s.eng.cold[1, s.slots].cpu().numpy(), 2, d))
    last = (length - 1) // page
    free = [r for r in range(3) if 0 not in table[r, :last]]
    assert len(free) >= 2
    table[:, last] = -3
    s.table.copy_(torch.from_numpy(table))
    s.eng.cold[1, :page].fill_(0xFF)
    s.run()
    torch.cuda.synchronize()
    assert s.eng.device_error() == gk.GK_ERR_DEVICE_BOUNDS
    none = np.zeros((0, 2, d))
    for r in free:
        i, bad = slice(r * length, (r + 1) * length), slice(r * length + last * page, (r + 1) * length)
        K[bad], V[bad], size[bad] = 0, 0, 0
        check_attention(np64(s.out[r]), np64(s.lse[r]), attend(np64(s.q[r]), (none, none), (K[i], V[i], size[i])), f"request {r}")
    s.close()


def check_weighted(s, what=""):
    """Outputs against 64 bits, in the values that carry weight.  As attend() counts them, but for the products of weight and span:
    those are scaled so that a largest one, over the queries of a KV head, lies between 2^10 and 2^11, and one below fp16's normal
    range is off by half a step of 2^-24, 2^-35 of it.  Weights are relative to a score that the largest passes by 2^4 at most and
    that was a row's largest once, so that they add up to 1 or more.  With W = max e^(s_j - max s) (|lo| + span) of a KV head:
      |O - O*| <= 2^-8 |O*| + (2^-11 + 2^-12) C + n 2^-31 W."""
    torch.cuda.synchronize()
    assert s.eng.device_error() == gk.GK_OK
    K, V, size = values(s.eng.cold[s.layer, s.slots].cpu().numpy(), s.hkv, s.d)
    at, g = np.cumsum([0] + s.cold), s.hq // s.hkv
    for r, n in enumerate(s.cold):
        i = slice(at[r], at[r + 1])
        for h in range(s.hkv):
            q, out, lse = (np64(x)[r, h * g:(h + 1) * g] for x in (s.q, s.out, s.lse))
            z = q @ K[i, h].T / np.sqrt(s.d)
            m = z.max(1, keepdims=True)
            p = np.exp(z - m)
            total = p.sum(1, keepdims=True)
            assert np.abs(lse - (m + np.log(total))[:, 0]).max() <= 2e-4, f"{what}: lse of request {r}"
            O, C = p @ V[i, h] / total, p @ size[i, h] / total
            W = (p[:, :, None] * size[i, h][None]).max()
            over = np.abs(out - O) - (2.0 ** -8 * np.abs(O) + (2.0 ** -11 + 2.0 ** -12) * C + n * 2.0 ** -31 * W)
            assert over.max() <= 0, f"{what}: request {r}, KV head {h} off by {over.max():.3g} over its bound"


@pytest.mark.parametrize("d,g", [(64, 1), (64, 4), (128, 2), (128, 4), (128, 5), (128, 8)])
@pytest.mark.parametrize("power,others,query", [(40, 0, 64), (90, 0, 64), (110, -25, 128)])
def test_wide_values_of_little_weight(d, g, power, others, query):
    """A token whose values are far larger than the others' and whose weight is far smaller (or 0) takes nothing from the tokens that
    carry the weight: at the first place, at a stage's ends, at the last, and where it had the weight until larger scores came."""
    n, places = 200, [0, 31, 32, 100, 199]
    rng = torch.Generator(device="cuda").manual_seed(power)
    requests = len(places) + 2
    k, v = (torch.randn(requests, n, 2, d, generator=rng, device="cuda") for _ in range(2))
    k *= 0.25
    k[..., 0] = 0
    wide = 2.0 ** power                   # times the values' own scale, so that it is a number of fp32
    for r, t in enumerate(places):
        k[r, t, :, 0] = -12
        v[r, t] *= wide
    k[-2, :32, :, 0] = -12                # a stage of small scores, the wide token among them
    v[-2, 3] *= wide
    k[-1, :, :, 0] = torch.linspace(-12, 0, n, device="cuda")[:, None]     # scores that rise all the way
    v[-1, 3] *= wide
    v[-1, 70, 1] *= wide
    v[v.abs() < 2.0 ** 20] *= 2.0 ** others
    s = Step(d, g, 2, [n] * requests, k=k.flatten(0, 1).to(BF), v=v.flatten(0, 1).to(BF), scale=0.25)
    s.q[..., 0] = query
    s.run()
    check_weighted(s)
    s.close()


@pytest.mark.parametrize("d,g", [(64, 4), (128, 2), (128, 4), (128, 5)])
@pytest.mark.parametrize("scale", [40, 400])
def test_lse_of_large_scores(d, g, scale):
    """Scores of hundreds and thousands, whose parts from lo and from codes cancel.  Of the sum S = sum |q| (|lo| + span) / sqrt(d):
    sum(q) in at most 11 fp32 sums and a product, 12 roundings of 2^-24, three bf16 terms to 2^-27; each tensor-core product adds 8 or 16
    exact terms and what was there, counted as 2^-21 of their absolute sum, once for the part of lo and at most four times for that
    of codes; four roundings of 2^-24 scale and add the parts: below 2^-18 S.  lse by as much as the worst key, and 2e-4 as ever."""
    s = Step(d, g, 2, [300, 70, 1000, 1], scale=scale, seed=scale)
    s.run()
    torch.cuda.synchronize()
    rows = s.eng.cold[1, s.slots].cpu().numpy()
    K = values(rows, 2, d)[0]
    lo, span = (np.repeat(np.abs(bf16_value(x).astype(np.float64)), 64, -1)[:, :, 0] for x in fields(rows, 2, d)[1:])
    at = np.cumsum([0] + s.cold)
    for r in range(4):
        i = slice(at[r], at[r + 1])
        for h in range(2):
            q = np64(s.q[r, h * g:(h + 1) * g])
            z = q @ K[i, h].T / np.sqrt(d)
            m = z.max(1)
            want = m + np.log(np.exp(z - m[:, None]).sum(1))
            S = (np.abs(q) @ (lo + span)[i, h].T / np.sqrt(d)).max(1)
            off = np.abs(np64(s.lse[r, h * g:(h + 1) * g]) - want)
            assert (off <= 2.0 ** -18 * S + 2e-4).all(), (r, h, off.max(), S.max())
    s.close()
