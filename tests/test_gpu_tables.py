"""gk_tables_step against the host block manager's own calls (gk_seq_release and
gk_seq_append_slots), bit for bit: random streams of steps with rows that leave,
grow and run out of blocks; bad inputs; captured graphs; and a whole step from
lengths to decode with nothing on the host but the lengths."""
import random

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from paged_kv_cache_pool_gb300 import binding as gk  # noqa: E402
from paged_kv_cache_pool_gb300.engine import Engine  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_pool_gb300 import build
    build.build()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Host:
    """The same rows as sequences of a host-only pool of the same blocks."""

    def __init__(self, rows, n_blocks, page, seed):
        self.pool = gk.gk_pool_create(1, 1, 1, 64, 0, n_blocks * page, page, seed)
        self.seqs = [gk.gk_seq_create(self.pool) for _ in range(rows)]

    def step(self, release, add):
        for r, x in enumerate(release):
            if x:
                gk.gk_seq_release(self.pool, self.seqs[r])
                self.seqs[r] = None
        for r, s in enumerate(self.seqs):
            if s is None:
                self.seqs[r] = gk.gk_seq_create(self.pool)
        order = [self.seqs[r] for r, n in enumerate(add) for _ in range(n)]
        try:
            slots = gk.gk_seq_append_slots(self.pool, order)[0] if order else np.zeros(0, np.int64)
        except gk.GkError as e:
            assert e.status == gk.GK_ERR_OOM
            slots = e.slots
        return slots

    def table(self, r):
        return gk.gk_seq_table(self.pool, self.seqs[r])

    def close(self):
        gk.gk_pool_destroy(self.pool)


def _engine(n_blocks, page, seed):
    return Engine(1, 1, 1, 64, 1, n_blocks * page, page, seed=seed)


@pytest.mark.parametrize("seed", range(16))
def test_random_steps_match_the_host_manager(seed):
    rnd = random.Random(seed)
    page = rnd.choice([1, 1, 4, 16, 16, 48])
    rows = rnd.choice([1, 2, 7, 33, 300, 1024, 1025, 2500])
    n_blocks = max(4, int(rows * rnd.choice([1, 3, 9])))
    hi = rnd.choice([1, 3, 40, 700]) if rows < 400 else rnd.choice([1, 3, 30])
    eng, host = _engine(n_blocks, page, seed), Host(rows, n_blocks, page, seed)
    # rows that can hold every block and what a step asks beyond them: only the stack runs out
    tables, held = eng.device_tables(rows, n_blocks + hi, n_blocks)
    for step in range(12):
        release = [int(rnd.random() < 0.2) if rnd.random() < 0.7 else 0 for _ in range(rows)]
        add = [rnd.choice([0, 1, rnd.randint(0, hi)]) for _ in range(rows)]
        want = host.step(release, add)
        total = sum(add)
        spare = rnd.choice([0, 0, 5])
        use = ints(release) if any(release) or rnd.random() < 0.5 else None
        slots, done = eng.tables_step(tables, ints(add), total + spare, use)
        assert eng.device_error() == gk.GK_OK
        slots, done = slots.cpu().numpy(), done.cpu().numpy()
        assert slots[:len(want)].tolist() == want.tolist() and (slots[len(want):] == -1).all()
        assert int(done.sum()) == len(want)
        length, table = tables.length.cpu().numpy(), tables.table.cpu().numpy()
        for r in rnd.sample(range(rows), min(rows, 60)) + [0, rows - 1]:
            ids, n = host.table(r)
            assert length[r] == n and table[r, :len(ids)].tolist() == ids.tolist()
        assert int(tables.num_free) == gk.gk_cold_stats(host.pool)[0]
    host.close()
    eng.seq_release(held)
    assert gk.gk_cold_stats(eng.pool) == (n_blocks, n_blocks)
    eng.close()


def test_long_rows_and_an_empty_stack():
    eng, host = _engine(40000, 1, 3), Host(3, 40000, 1, 3)
    tables, _ = eng.device_tables(3, 40000, 40000)
    for release, add in (([0, 0, 0], [30000, 0, 9000]), ([0, 1, 1], [1, 5000, 20000]), ([0, 0, 0], [1, 1, 1]),
                         ([1, 0, 0], [0, 7, 0])):
        want = host.step(release, add)
        slots, done = eng.tables_step(tables, ints(add), sum(add), ints(release))
        assert slots.cpu().tolist() == want.tolist() + [-1] * (sum(add) - len(want)) and int(done.sum()) == len(want)
        assert int(tables.num_free) == gk.gk_cold_stats(host.pool)[0]
    assert eng.device_error() == gk.GK_OK
    host.close()
    eng.close()


def _tables(page=4, lens=(5, 0, 9), free=(3, 7, 1, 2), held=((0, 4), (), (5, 6, 8)), width=4, **out):
    table = np.full((3, width), 77, np.int32)
    for r, h in enumerate(held):
        table[r, :len(h)] = h
    eng = _engine(10, page, 0)
    return eng, gk.Tables(ints(table.tolist()), ints(list(free)), ints(list(lens)), ints([len(free)]), **out)


def _step(eng, t, add, n_slots, release=None, n_free=None):
    if n_free is not None:
        t.num_free.fill_(n_free)
    slots, done = eng.tables_step(t, ints(add), n_slots, None if release is None else ints(release))
    return slots.cpu().tolist(), done.cpu().tolist(), eng.device_error()


def test_a_step_by_hand():
    eng, t = _tables()
    slots, done, err = _step(eng, t, [4, 2, 3], 10)
    # row 0: 5..7 in block 4, 8 in the first free block, 2; row 1 in block 1; row 2: 9..11 in its own block 8
    assert slots == [17, 18, 19, 8, 4, 5, 33, 34, 35, -1] and done == [4, 2, 3] and err == gk.GK_OK
    assert t.length.cpu().tolist() == [9, 2, 12] and int(t.num_free) == 2
    assert t.table.cpu().tolist() == [[0, 4, 2, 77], [1, 77, 77, 77], [5, 6, 8, 77]]
    # rows 0 and 2 leave and row 0 starts again: its blocks 0 4 2, then 5 6 8, are pushed; 8 and 6 come off first
    t2 = gk.Tables(t.table, torch.cat([t.free, ints([0] * 6)]), t.length, t.num_free)
    slots, done, err = _step(eng, t2, [5, 0, 0], 5, [1, 0, 1])
    assert slots == [32, 33, 34, 35, 24] and err == gk.GK_OK
    assert t2.length.cpu().tolist() == [5, 2, 0] and int(t2.num_free) == 6
    assert t2.free.cpu().tolist()[:8] == [3, 7, 0, 4, 2, 5, 6, 8]
    eng.close()


def test_separate_outputs_leave_the_inputs():
    lo, nf = ints([9, 9, 9]), ints([9])
    eng, t = _tables(length_out=lo, num_free_out=nf)
    for _ in range(2):
        slots, _, err = _step(eng, t, [4, 2, 3], 9)
        assert slots == [17, 18, 19, 8, 4, 5, 33, 34, 35] and err == gk.GK_OK
        assert t.length.cpu().tolist() == [5, 0, 9] and int(t.num_free) == 4
        assert lo.cpu().tolist() == [9, 2, 12] and nf.cpu().tolist() == [2]
    eng.close()


@pytest.mark.parametrize("change,add,n_slots,release,want_done", [
    (dict(lens=(-1, 0, 9)), [1, 1, 1], 3, None, [0, 1, 1]),              # a negative length
    (dict(lens=(5, 0, 17)), [1, 1, 1], 3, None, [1, 1, 0]),              # a length past its row
    (dict(), [1, -3, 1], 2, None, [1, 0, 1]),                            # a negative add
    (dict(), [12, 1, 1], 14, None, [0, 1, 1]),                           # a table longer than its row
    (dict(), [1, 2147483647, 1], 8, None, [1, 0, 0]),                    # tokens that no slot map holds
    (dict(), [1, 1, 3], 4, None, [1, 1, 0]),                             # a slot map too short for the last row
    (dict(free=(3, 7, 1, 99)), [4, 1, 0], 5, None, [4, 1, 0]),           # an id that is no block: its slots are -1
    (dict(free=(3, 7, 1, -1)), [4, 1, 0], 5, None, [4, 1, 0]),
    (dict(), [0, 0, 0], 1, [1, 0, 1], [0, 0, 0]),                        # five blocks back onto a full stack of four
])
def test_bad_inputs_are_reported(change, add, n_slots, release, want_done):
    eng, t = _tables(**change)
    slots, done, err = _step(eng, t, add, n_slots, release)
    assert err == gk.GK_ERR_DEVICE_BOUNDS and done == want_done
    assert all(-1 <= s < 40 for s in slots)
    if release:
        assert t.length.cpu().tolist() == [5, 0, 9] and int(t.num_free) == 4
    eng.close()


@pytest.mark.parametrize("count", [-1, 5, 2 ** 31 - 1, -2 ** 31])
def test_a_bad_count_is_an_empty_stack(count):
    eng, t = _tables()
    slots, done, err = _step(eng, t, [4, 2, 3], 9, None, count)
    assert err == gk.GK_ERR_DEVICE_BOUNDS and done == [3, 0, 0] and slots == [17, 18, 19] + [-1] * 6
    eng.close()


def test_no_rows_no_slots():
    eng, t = _tables()
    assert _step(eng, t, [0, 0, 0], 0) == ([], [0, 0, 0], gk.GK_OK)
    none = gk.Tables(ints([[]]).view(0, 1)[:, :0], t.free, ints([]), t.num_free)
    slots = ints([5]).long()
    gk.gk_tables_step(eng.pool, None, none, ints([]), slots, ints([]))
    torch.cuda.synchronize()
    assert slots.tolist() == [5] and int(t.num_free) == 4
    eng.close()


def test_captured_and_replayed_on_a_side_stream():
    """A graph of two steps: each replay goes on from the state the last one left."""
    page, rows, n = 4, 50, 4000
    eng, host = _engine(n, page, 8), Host(rows, n, page, 8)
    t, _ = eng.device_tables(rows, 400, n)
    add, release = ints([1] * rows), ints([int(r % 7 == 3) for r in range(rows)])
    many = ints([r % 5 for r in range(rows)])
    slots = [torch.empty(rows * 5, dtype=torch.int64, device="cuda") for _ in range(2)]
    done = torch.empty(rows, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        gk.gk_tables_step(eng.pool, side, t, add, slots[0], done)   # first use outside the capture
        side.synchronize()
        host.step([0] * rows, [1] * rows)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            gk.gk_tables_step(eng.pool, side, t, add, slots[0], done)
            gk.gk_tables_step(eng.pool, side, t, many, slots[1], done, release)
    for _ in range(5):
        graph.replay()
        torch.cuda.synchronize()
        want = host.step([0] * rows, [1] * rows)
        assert slots[0][:rows].cpu().tolist() == want.tolist()
        want = host.step(release.cpu().tolist(), many.cpu().tolist())
        assert slots[1][:len(want)].cpu().tolist() == want.tolist() and (slots[1][len(want):] == -1).all()
    assert eng.device_error() == gk.GK_OK
    host.close()
    eng.close()


def test_from_lengths_to_decode():
    """Slots and tables from the device, K/V through them, prompt attention behind them, then a decode step."""
    from prompt_ref import check, expected
    hq, hkv, d, page = 8, 2, 128, 16
    eng = Engine(1, hq, hkv, d, 300, 4096, page, seed=2)
    rng = torch.Generator(device="cuda").manual_seed(4)

    def rand(n, h):
        return torch.randn(n, h, d, generator=rng, device="cuda").to(torch.bfloat16)
    host = lambda x: x.double().cpu().numpy()  # noqa: E731
    base = eng.prefix_alloc(200)
    pk, pv = rand(200, hkv), rand(200, hkv)
    eng.write_prefix(0, base, 200, 0, pk, pv)
    t, held = eng.device_tables(4, 64, 200)
    which = [base, base, -1, base]
    lps = [200 if b >= 0 else 0 for b in which]
    past = [[host(pk), host(pv)] if b >= 0 else [np.zeros((0, hkv, d))] * 2 for b in which]
    length = [0, 0, 0, 0]
    # prompts, then turns; row 2 leaves before the second step and its slot starts another prompt
    for new, leave in (([130, 40, 300, 0], None), ([7, 90, 33, 260], [0, 0, 1, 0]), ([1, 1, 1, 1], None)):
        if leave:
            past[2], length[2] = [np.zeros((0, hkv, d))] * 2, 0
        T = sum(new)
        slots, _ = eng.tables_step(t, ints(new), T, None if leave is None else ints(leave))
        q, k, v = rand(T, hq), rand(T, hkv), rand(T, hkv)
        out, lse = torch.empty_like(q), torch.empty(T, hq, device="cuda")
        batch = eng.prompt_batch(new, which, lps, length, t.table, 64)
        eng.prompt(0, batch, eng.prompt_plan(batch), q, k, v, out, lse)
        eng.append_kv(0, slots, k, v)
        torch.cuda.synchronize()
        assert eng.device_error() == gk.GK_OK
        check(host(out), host(lse), expected(host(q), host(k), host(v), new, past), str(new))
        t0 = 0
        for r, n in enumerate(new):
            past[r] = [np.concatenate([a, host(x[t0:t0 + n])]) for a, x in zip(past[r], (k, v))]
            length[r] += n
            t0 += n
    assert t.length.cpu().tolist() == length
    # the last prompt step was one token a row: decode over the same tables gives the same rows
    b = eng.batch(which, lps, length, t.table, 64)
    o, l1 = torch.empty(4, hq, d, device="cuda"), torch.empty(4, hq, device="cuda")
    b.set_device(d_q=q, d_out=o, d_lse=l1)
    eng.decode(0, b, eng.plan(b), gk.GK_BACKEND_CASCADE)
    torch.cuda.synchronize()
    assert (l1 - lse).abs().max() < 1e-3 and (o - out.float()).abs().max() < 2e-2
    eng.seq_release(held)
    eng.close()
