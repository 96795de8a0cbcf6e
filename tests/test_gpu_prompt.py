"""gk_prompt_attn against a plain fp64 attention: every geometry, ragged lengths
from none to several tiles, each source of keys alone and together, strides,
hidden infinities and NaN, bad block ids, captured graphs, other streams, and a
whole step (slots, K/V writes, prompt attention, then decode over what it wrote)."""
import random

import numpy as np
import pytest

from prompt_ref import check, expected

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from paged_kv_cache_pool_gb300 import binding as gk  # noqa: E402

GEOMETRIES = [(d, g) for d, gs in ((64, (1, 2, 4)), (128, (1, 2, 4, 5, 8))) for g in gs]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_pool_gb300 import build
    build.build()


class Prompts:
    """A pool with HOT prefixes and COLD contexts, and the packed new tokens of one step."""

    def __init__(self, d, g, hkv, new, prefixes=(), which=None, cold=None, page=16, layers=2, layer=1, seed=0, scale=1.0,
                 fused=False, spare_nan=True, spare_blocks=3, hot_skip=0):
        rng = torch.Generator(device="cuda").manual_seed(seed)
        bf = torch.bfloat16
        self.new, self.layer, self.d, self.hkv, self.hq, self.page = list(new), layer, d, hkv, hkv * g, page
        which = [-1] * len(new) if which is None else which
        cold = [0] * len(new) if cold is None else cold

        def rand(*shape):
            return torch.randn(*shape, generator=rng, device="cuda").to(bf)
        hot = max(1, sum(prefixes)) + 5 + hot_skip
        blocks = [-(-c // page) for c in cold]
        slots = (sum(blocks) + spare_blocks) * page
        # everything that no key lives in holds NaN
        junk = float("nan") if spare_nan else 0.0
        self.hot = [torch.full((hot * layers * hkv * d,), junk, dtype=bf, device="cuda") for _ in range(2)]
        self.cold = [torch.full((layers, slots, hkv, d), junk, dtype=bf, device="cuda") for _ in range(2)]
        self.pool = gk.gk_pool_create(layers, self.hq, hkv, d, hot, slots, page, 11, *self.hot, *self.cold)
        bases, pre = [], []
        if hot_skip:
            gk.gk_prefix_alloc(self.pool, hot_skip)      # the prefixes come behind it
        for lp in prefixes:
            bases.append(gk.gk_prefix_alloc(self.pool, lp))
            k, v = rand(lp, hkv, d), rand(lp, hkv, d)
            gk.gk_write_prefix_kv(self.pool, None, layer, bases[-1], lp, 0, k, v)
            pre.append((k, v))
        seqs, order = [], []
        for c in cold:
            seqs.append(gk.gk_seq_create(self.pool))
            order += [seqs[-1]] * c
        sl, _ = gk.gk_seq_append_slots(self.pool, order)
        ck, cv = rand(len(order), hkv, d), rand(len(order), hkv, d)
        if order:
            gk.gk_append_kv(self.pool, None, layer, torch.from_numpy(sl).cuda(), ck, cv)
        width = max([1] + blocks)
        self.table = torch.from_numpy(gk.gk_seq_tables(self.pool, seqs, width)[0]).cuda()
        T = sum(new)
        self.T = T
        if fused:
            row = torch.full((T, (self.hq + 2 * hkv) * d + 16), junk, dtype=bf, device="cuda")
            ends = np.cumsum([0, self.hq, hkv, hkv]) * d + 8
            self.q, self.k, self.v = (row[:, a:b].view(T, -1, d) if T else row[:, a:b].reshape(0, (b - a) // d, d)
                                      for a, b in zip(ends, ends[1:]))
        else:
            self.q, self.k, self.v = (torch.empty(T, h, d, dtype=bf, device="cuda") for h in (self.hq, hkv, hkv))
        self.q.copy_(torch.randn(T, self.hq, d, generator=rng, device="cuda") * scale)
        self.k.copy_(rand(T, hkv, d))
        self.v.copy_(rand(T, hkv, d))
        self.batch = gk.PromptBatch(new, [bases[w] if w >= 0 else -1 for w in which],
                                    [prefixes[w] if w >= 0 else 0 for w in which], cold, self.table, width)
        at = np.cumsum([0] + list(cold))
        empty = torch.empty(0, hkv, d, dtype=bf, device="cuda")
        self.past = [[torch.cat([pre[w][i] if w >= 0 else empty, (ck, cv)[i][a:b]]) for i in range(2)]
                     for w, a, b in zip(which, at, at[1:])]
        self.out = torch.full((T, self.hq, d), 7.0, dtype=bf, device="cuda")
        self.lse = torch.full((T, self.hq), 7.0, device="cuda")
        self.plan = None

    def run(self, stream=None, lse=True):
        if self.plan is None:
            self.plan = gk.gk_prompt_plan_build(self.pool, self.batch, stream)
        self.batch.set_device(self.q, self.k, self.v, self.out, self.lse if lse else None)
        gk.gk_prompt_attn(self.pool, stream, self.layer, self.batch, self.plan)
        return self

    def host(self, x):
        return x.double().cpu().numpy()

    def want(self):
        return expected(self.host(self.q), self.host(self.k), self.host(self.v), self.new,
                        [[self.host(x) for x in kv] for kv in self.past])

    def verify(self, what="", error=gk.GK_OK):
        torch.cuda.synchronize()
        assert gk.gk_device_error(self.pool) == error
        check(self.host(self.out), self.host(self.lse), self.want(), what)

    def info(self):
        return gk.gk_prompt_plan_info(self.plan)

    def close(self):
        if self.plan:
            gk.gk_prompt_plan_destroy(self.plan)
        gk.gk_pool_destroy(self.pool)


def prompts(*a, **k):
    p = Prompts(*a, **k)
    try:
        p.run().verify(str((a, k)))
        return p.info()
    finally:
        p.close()


@pytest.mark.parametrize("d,g", GEOMETRIES)
def test_fresh_prompts(d, g):
    prompts(d, g, 2, [1, 0, 129, 31, 300, 2], fused=True)


@pytest.mark.parametrize("d,g", GEOMETRIES)
def test_prefix_and_context(d, g):
    prompts(d, g, 2, [5, 140, 0, 33, 1], prefixes=[200, 128], which=[0, 1, 0, 0, -1], cold=[37, 0, 9, 260, 130], page=16)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 700])
@pytest.mark.parametrize("d,g", [(128, 4), (64, 1), (128, 5)])
def test_one_prompt_of_every_edge(d, g, n):
    prompts(d, g, 1, [n])


@pytest.mark.parametrize("past", [1, 2, 127, 128, 129, 255, 256, 383, 900])
@pytest.mark.parametrize("kind", ["hot", "cold"])
def test_one_source_of_every_edge(kind, past):
    prompts(128, 4, 2, [3, 70], prefixes=[past] if kind == "hot" else (), which=[0, 0] if kind == "hot" else None,
            cold=[past, past] if kind == "cold" else None, page=1 if past % 2 else 16)


@pytest.mark.parametrize("page", [1, 3, 4, 16, 128, 200])
def test_page_sizes(page):
    prompts(128, 5, 2, [40, 7], cold=[333, 201], page=page)


def test_long_keys_of_few_rows_are_split_and_joined():
    for new, kw in (([3], dict(cold=[5000])), ([1], dict(prefixes=[6001], which=[0])), ([600], {})):
        info = prompts(128, 4, 2, new, **kw)
        # at most five tiles of keys (the last case) may stay whole: the join's launch costs about as much
        assert not kw or info["max_pieces"] > 1 and info["partials"] > 0


def test_stacked_requests_of_one_prefix():
    info = prompts(128, 4, 2, [4, 1, 16, 0, 9, 70, 2, 30] * 3, prefixes=[4000, 300], which=[0] * 20 + [1] * 4,
                   cold=[5, 0, 130, 3, 0, 60, 1, 0] * 3, page=1)
    assert info["stacked_requests"] > 0


@pytest.mark.parametrize("scale", [0.0, 8.0, 64.0])
def test_flat_and_peaked_scores(scale):
    prompts(128, 4, 2, [300, 20], prefixes=[150], which=[0, -1], cold=[0, 140], scale=scale)


def test_many_items_per_cta():
    # several items on each SM: the ring, the barriers and tensor memory carry over
    prompts(64, 2, 8, [200 + 37 * i for i in range(12)], prefixes=[500], which=[0, -1] * 6, cold=[0, 150, 0, 0, 3, 300] * 2)


def test_no_lse():
    p = Prompts(128, 4, 2, [50])
    p.run(lse=False)
    torch.cuda.synchronize()
    assert (p.lse == 7).all()
    p.run().verify()
    p.close()


def test_rows_behind_the_last_request_stay():
    p = Prompts(128, 4, 2, [33, 5])
    out = torch.full((100, p.hq, p.d), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((100, p.hq), 3.0, device="cuda")
    p.out, p.lse = out[:38], lse[:38]
    p.run().verify()
    assert (out[38:] == 3).all() and (lse[38:] == 3).all()
    p.close()


def test_no_tokens():
    for new in ([], [0, 0]):
        p = Prompts(128, 4, 2, new)
        p.run().verify()
        p.close()


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_hidden_infinities_and_nan(bad):
    """What later tokens of a request, or another request's tokens, hold reaches no row that does not see them."""
    p = Prompts(128, 4, 2, [150, 40, 200], cold=[0, 20, 300])
    p.v[100, 1, 5] = bad              # seen by rows 100.. of request 0
    p.v[155, 0, :] = bad              # request 1, token 5
    p.k[350, :, 3] = bad              # request 2, token 160: its scores, from there on, hold no finite sum
    p.run()
    torch.cuda.synchronize()
    O, A, L = p.want()
    out, lse = p.host(p.out), p.host(p.lse)
    clean = np.isfinite(O) & np.isfinite(L)[..., None]
    assert np.isfinite(out[clean]).all()
    assert (np.abs(out - O)[clean] <= (2 ** -7 + 2 ** -12) * A[clean]).all()
    # request 0: only channel 5 of KV head 1 and only from token 100 on
    assert np.isfinite(out[:100]).all() and not np.isfinite(out[100:150, 4:, 5]).any()
    assert np.isfinite(out[:150, :4]).all() and np.isfinite(np.delete(out[:150, 4:], 5, axis=2)).all()
    assert np.isfinite(lse[:190]).all()
    assert np.isfinite(out[150:155]).all() and not np.isfinite(out[155:190, :4]).any()
    assert np.isfinite(out[190:350]).all()
    p.close()


def test_bad_block_ids_are_reported_and_read_nothing():
    p = Prompts(128, 4, 2, [20], cold=[100], page=16, spare_nan=False)
    for v in (-1, 10 ** 9, 2 ** 31 - 1):
        p.table[0, 3] = v
        p.run()
        torch.cuda.synchronize()
        assert gk.gk_device_error(p.pool) == gk.GK_ERR_DEVICE_BOUNDS
        # tokens 48..63 count as zero keys and values
        q, k, w = p.host(p.q), p.host(p.k), p.host(p.v)
        pk, pv = (p.host(x) for x in p.past[0])
        pk[48:64] = 0
        pv[48:64] = 0
        check(p.host(p.out), p.host(p.lse), expected(q, k, w, p.new, [(pk, pv)]), "bad block")
    p.close()


def test_captured_replayed_and_on_another_stream():
    p = Prompts(128, 4, 2, [300, 9, 40], prefixes=[260], which=[0, 0, -1], cold=[10, 700, 0])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        p.run(side)
        side.synchronize()
        p.verify("side stream")
        first = p.out.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            p.run(side)
            p.run(side)
    p.out.fill_(0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(p.out, first)
    # new values in the same buffers
    p.q.copy_(torch.randn_like(p.q))
    graph.replay()
    p.verify("replayed")
    p.close()


def test_the_same_inputs_give_the_same_bits():
    p = Prompts(128, 5, 2, [300, 9, 40], prefixes=[2600], which=[0, 0, 0], cold=[10, 700, 0])
    p.run()
    a, b = p.out.clone(), p.lse.clone()
    for _ in range(5):
        p.run()
        torch.cuda.synchronize()
        assert torch.equal(a, p.out) and torch.equal(b, p.lse)
    p.close()


def test_two_plans_of_one_pool_on_two_streams():
    a = Prompts(128, 4, 2, [300, 9, 40], prefixes=[900], which=[0, 0, -1], cold=[10, 700, 0])
    other = gk.PromptBatch([40, 309], None, None, None)
    out, lse = torch.empty_like(a.out), torch.empty_like(a.lse)
    other.set_device(a.q, a.k, a.v, out, lse)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    plan = gk.gk_prompt_plan_build(a.pool, other, s2)
    for _ in range(10):
        a.run(s1)
        gk.gk_prompt_attn(a.pool, s2, a.layer, other, plan)
    a.verify("first")
    e = [np.zeros((0, 2, 128))] * 2
    check(a.host(out), a.host(lse), expected(a.host(a.q), a.host(a.k), a.host(a.v), [40, 309], [e, e]), "second")
    gk.gk_prompt_plan_destroy(plan)
    a.close()


def test_plan_update_reuses_a_plan():
    p = Prompts(128, 4, 2, [30, 9], cold=[10, 700])
    p.run().verify()
    big = gk.PromptBatch([39], None, None, None)
    for batch, new, past in ((big, [39], [(p.past[0][0][:0], p.past[0][1][:0])]), (p.batch, p.new, p.past)):
        gk.gk_prompt_plan_update(p.pool, p.plan, batch)
        p.batch, p.new, p.past, keep = batch, new, past, (p.batch, p.new, p.past)
        p.run().verify("updated")
        p.batch, p.new, p.past = keep
    p.close()


def test_chunks_of_a_prompt_equal_the_whole():
    """A prompt's second chunk over the pages its first chunk was written to, then decode over both."""
    from paged_kv_cache_pool_gb300.engine import Engine
    L, hq, hkv, d, n = 1, 8, 2, 128, 700
    eng = Engine(L, hq, hkv, d, 16, 1024, 16, seed=5)
    rng = torch.Generator(device="cuda").manual_seed(9)
    q, k, v = (torch.randn(n, h, d, generator=rng, device="cuda").to(torch.bfloat16) for h in (hq, hkv, hkv))
    seq = eng.seq_create()
    out, lse = torch.empty_like(q), torch.empty(n, hq, device="cuda")
    done = 0
    for size in (333, 1, 366):
        table = eng.to_device(eng.block_tables([seq], 64))
        slots, _ = eng.append_slots([seq] * size)
        part = slice(done, done + size)
        eng.append_kv(0, eng.to_device(slots), k[part], v[part])
        batch = eng.prompt_batch([size], None, None, [done], table, 64)
        eng.prompt(0, batch, eng.prompt_plan(batch), q[part], k[part], v[part], out[part], lse[part])
        torch.cuda.synchronize()
        done += size
    assert eng.device_error() == gk.GK_OK
    host = lambda x: x.double().cpu().numpy()  # noqa: E731
    e = np.zeros((0, hkv, d))
    check(host(out), host(lse), expected(host(q), host(k), host(v), [n], [(e, e)]), "chunks")
    # a decode step whose query is the last token's gives the last row
    table = eng.to_device(eng.block_tables([seq], 64))
    b = eng.batch([-1], [0], [n], table, 64)
    o1, l1 = torch.empty(1, hq, d, device="cuda"), torch.empty(1, hq, device="cuda")
    b.set_device(d_q=q[-1:], d_out=o1, d_lse=l1)
    for backend in (gk.GK_BACKEND_DENSE, gk.GK_BACKEND_CASCADE):
        eng.decode(0, b, eng.plan(b), backend)
        torch.cuda.synchronize()
        assert (l1[0] - lse[-1]).abs().max() < 1e-3 and (o1[0] - out[-1].float()).abs().max() < 2e-2
    eng.close()


def test_strided_output():
    """Rows of out inside a wider tensor, whose other columns stay."""
    p = Prompts(128, 4, 2, [70, 3, 200], prefixes=[130], which=[0, -1, -1], cold=[0, 900, 0], fused=True)
    wide = torch.full((p.T, p.hq * p.d + 24), 5.0, dtype=torch.bfloat16, device="cuda")
    p.out = wide[:, 8:8 + p.hq * p.d].view(p.T, p.hq, p.d)
    p.run().verify("strided out")
    assert (wide[:, :8] == 5).all() and (wide[:, 8 + p.hq * p.d:] == 5).all()
    p.close()


@pytest.mark.parametrize("seed", range(24))
def test_random_steps(seed):
    r = random.Random(seed)
    d, g = r.choice(GEOMETRIES)
    page, b = r.choice([1, 3, 16, 64]), r.choice([1, 2, 5, 12, 30])
    most = r.choice([3, 40, 300, 900]) if b < 12 else r.choice([1, 8, 60])
    prefixes = [r.randint(1, 1500) for _ in range(r.randint(1, 3))]
    prompts(d, g, r.choice([1, 2, 3]), [r.randint(0, most) for _ in range(b)], prefixes=prefixes,
            which=[r.randint(-1, len(prefixes) - 1) for _ in range(b)], cold=[r.choice([0, r.randint(0, 700)]) for _ in range(b)],
            page=page, seed=seed, fused=r.random() < 0.5, scale=r.choice([1.0, 1.0, 6.0]))


def test_many_small_requests():
    r = random.Random(5)
    prompts(128, 4, 2, [r.randint(0, 9) for _ in range(400)], prefixes=[700, 129, 1], which=[min(3, i // 120) - 1 for i in range(400)],
            cold=[r.choice([0, 1, 17, 150]) for _ in range(400)], page=4)


@pytest.mark.parametrize("d,g", [(64, 4), (128, 5)])
def test_one_long_prompt(d, g):
    prompts(d, g, 1, [4500], cold=[1000])


@pytest.mark.parametrize("bad", [-float("inf"), -1e30])
def test_keys_that_score_the_lowest(bad):
    """Visible keys whose scores are minus infinity, or far below every other, weigh nothing; also as a row's first keys."""
    p = Prompts(128, 4, 2, [200, 40], cold=[0, 150])
    p.q[:, :, 0] = p.q[:, :, 0].abs() + 0.5
    p.k[0:70, :, 0] = bad            # hides the first keys of request 0; its own rows 70.. see others
    p.k[130:141, :, 0] = bad
    p.k[230:235, :, 0] = bad
    p.run()
    torch.cuda.synchronize()
    O, A, L = p.want()
    seen = np.isfinite(L).all(1) & (L > -1e20).all(1)
    assert seen.sum() == 240 - 70
    check(p.host(p.out)[seen], p.host(p.lse)[seen], (O[seen], A[seen], L[seen]), f"lowest {bad}")
    p.close()


@pytest.mark.parametrize("where", ["cold", "hot"])
def test_caches_past_32_bit_offsets(where):
    """K and V of the pool lie more than 2^31 elements behind its first."""
    if where == "cold":
        p = Prompts(128, 4, 8, [100], cold=[400], page=16, spare_blocks=140000)
        at = p.cold[0].numel()
    else:
        p = Prompts(128, 4, 8, [100], prefixes=[333], which=[0], hot_skip=1100000)
        at = p.hot[0].numel()
    assert at > 2 ** 31
    p.run().verify(where)
    p.close()


def test_plans_are_not_built_or_updated_while_capturing():
    p = Prompts(128, 4, 2, [30, 2], cold=[0, 300])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        p.run(side)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            with pytest.raises(gk.GkError) as e:
                gk.gk_prompt_plan_build(p.pool, p.batch, side)
            assert e.value.status == gk.GK_ERR_UNSUPPORTED
            with pytest.raises(gk.GkError) as e:
                gk.gk_prompt_plan_update(p.pool, p.plan, p.batch, side)
            assert e.value.status == gk.GK_ERR_UNSUPPORTED
            p.run(side)              # the plan is as it was
    p.out.fill_(0)
    graph.replay()
    p.verify("after refusals")
    p.close()


def test_two_graphs_of_one_plan_replayed_in_turn():
    """They share the plan's partial states; on one stream each replay ends before the next begins."""
    p = Prompts(128, 4, 2, [6], cold=[3000])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs, graphs = [], []
    with torch.cuda.stream(side):
        p.run(side)
        side.synchronize()
        assert p.info()["partials"] > 0
        q2 = (p.q * -0.5).contiguous()
        for q in (p.q, q2):
            out = torch.zeros_like(p.out)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                p.batch.set_device(q, p.k, p.v, out, p.lse)
                gk.gk_prompt_attn(p.pool, side, p.layer, p.batch, p.plan)
            outs.append(out)
            graphs.append(graph)
        for i in range(20):
            graphs[i & 1].replay()
    torch.cuda.synchronize()
    p.out = outs[1]
    p.q.copy_(q2)
    p.verify("second graph")
    p.q.copy_(q2 * -2)
    p.run()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], p.out)
    p.close()
