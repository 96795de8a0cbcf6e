"""The barriers' model is the kernel's, and would notice (CPU).

The counts, arrivals and ring depths that test_prompt_barriers_host.Model repeats are
read from the kernel's source here, so a change there fails until the model follows.
And each fault that the protocol has had, or that a wait or an arrival of it keeps
out, is put into a copy of the model: it has to be rejected."""
import inspect
import os
import re
import textwrap

import pytest

import test_prompt_barriers_host as model

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_pool_gb300", "csrc", "prompt_attn.cu")

#: the model's name of each barrier of the kernel; an arrival of each thread of a warp is one arrival there
NAMES = {"B_QFULL": "QFULL0", "B_QEMPTY": "QEMPTY0", "B_SFULL": "S0", "B_PFULL": "P0", "B_OFULL": "O0", "B_RFULL": "F0", "B_REMPTY": "E0",
         "B_RSCAN": "C0", "B_ROUT": "W0"}


@pytest.fixture(scope="module")
def source():
    return re.sub(r"//[^\n]*", "", open(SOURCE).read())


def test_counts_are_the_kernels(source):
    counts = {name: int(n) for name, n in re.findall(r"mbar_init\(bar\((B_\w+)[^)]*\), (\d+)\)", source)}
    assert counts.pop("B_FINAL") == 1
    assert set(counts) == set(NAMES)
    bars = model.Model(0, 5).bars
    for name, n in counts.items():
        threads, single = divmod(n, 32) if n >= 32 else (0, n)     # whole warps, and arrivals of one thread
        assert bars[NAMES[name]].count == threads + single, name


def test_arrivals_are_the_kernels(source):
    """How often each role arrives: as the model's, 32 for each of its arrivals of a warp's threads."""
    many = sorted((re.sub(r"[\s()]", "", b), int(n)) for b, n in re.findall(r"mbar_arrive_n\((bar\(B_\w+[^;]*?\)|b), (\d+)\);", source))
    assert many == sorted([
        ("barB_RFULL+st", 128),        # a staging element: no load fills it (model: 4)
        ("b", 127),                    # beside expect_tx's own (model: 3 and the load's)
        ("barB_RFULL+st", 32),         # a gather warp that scanned (model: 1 of 4)
        ("barB_REMPTY+ring.st", 7),    # the relay (model: 7)
        ("barB_REMPTY+st", 8),         # the output warp (model: 8)
        ("barB_REMPTY+ring.st", 2),    # a softmax warp of a partial state (model: 2 of 8)
    ])
    text = inspect.getsource(model.Model)
    for line in ('self.arrive("F%d" % st, 4)', 'self.arrive("F%d" % st, 3)', 'self.arrive("E%d" % ring.st, 7)', 'self.arrive("E%d" % st, 8)',
                 'self.arrive("E%d" % ring.st, 2)'):
        assert line in text


def test_ring_depths_are_the_kernels(source):
    deep, flat = re.search(r"NST = D == 128 \? (\d+) : (\d+);", source).groups()
    assert model.STAGES == {128: int(deep), 64: int(flat)}


def _mutant(*changes):
    """The model with texts of its methods replaced: (method, old, new)."""
    body = {}
    for method, old, new in changes:
        src = body.get(method) or textwrap.dedent(inspect.getsource(getattr(model.Model, method)))
        assert src.count(old) == 1, (method, old, src.count(old))
        body[method] = src.replace(old, new)
    made = {}
    for src in body.values():
        exec(src, vars(model), made)
    return type("Mutant", (model.Model,), made)


WAIT_E = 'yield from self.wait("E%d" % st, ph ^ 1)'
FAULTS = {
    "the load role does not wait for the stages that are gathered": [
        ("producer", WAIT_E, "if j >= 2 * nt or kinds[j // 2] != 'c':\n                    " + WAIT_E)],
    "gather warps wait for free stages themselves": [
        ("producer", 'self.arrive("C%d" % st)\n            else', "pass\n            else"),
        ("gather", 'yield from self.wait("C%d" % st, ph[st])\n            ph[st] ^= 1',
         'yield from self.wait(*(("E%d" % st, at ^ 1) if cold else ("C%d" % st, ph[st])))\n            ph[st] ^= not cold'),
        ("gather", "st = ring.st\n", "st, at = ring.st, ring.ph\n")],
    "a staging element gets two phases' arrivals": [
        ("softmax", 'self.arrive("W%d" % ring.st)', 'self.arrive("W%d" % ring.st)\n                self.arrive("E%d" % ring.st, 2)')],
    "a Q tile without key tiles takes part in the staging": [
        ("staging", "return (cnt[0] > 0) + (cnt[1] > 0)", "return 2"),
        ("softmax", "mine = int(i == 1 and cnt[0] > 0)", "mine = int(i == 1)"),
        ("softmax", """if cnt[i] > 0:
            yield from self.wait("O%d" % i, on & 1)
            on += 1
            assert self.pv[i] == (n, cnt[i] - 1), "O read early"
""", """if cnt[i] > 0:
            yield from self.wait("O%d" % i, on & 1)
            on += 1
            assert self.pv[i] == (n, cnt[i] - 1), "O read early"
        if True:
"""),
        ("writer", "if cnt[i] == 0:\n                continue\n", "pass\n")],
    "the relay arrives for a probability tile before the last one's phase is over": [
        ("relay", "if pn[i] > 0:", "if False:")],
    "the relay does not wait for the value tile": [
        ("relay", "yield from full((n, 2 * j + 1))\n", "self.arrive('E%d' % ring.st, 7); ring.next()\n")],
    "the load role loads a Q tile over one in use": [
        ("producer", 'yield from self.wait("QEMPTY%d" % i, (qn[i] & 1) ^ 1)', "pass")],
    "S is issued over a tile that softmax has not read": [
        ("issuer", 'yield from self.wait("P%d" % i, pn[i] & 1)', "yield None")],
    "the output warp gives its stage back too early": [
        ("writer", 'yield from self.wait("W%d" % st, ph[st])', "yield None")],
    "a softmax warp stages its output before the element is there": [
        ("softmax", 'yield from self.wait("F%d" % ring.st, ring.ph)', "yield None")],
}


def test_a_copy_without_a_fault_passes():
    same = _mutant(("relay", "if pn[i] > 0:", "if pn[i] != 0:"))
    for seed in range(40):
        same(seed, model.STAGES[128]).run()


@pytest.mark.parametrize("fault", sorted(FAULTS))
@pytest.mark.parametrize("d", [128, 64])
def test_faults_are_rejected(fault, d):
    wrong = _mutant(*FAULTS[fault])
    for seed in range(150):
        try:
            wrong(seed, model.STAGES[d]).run()
        except AssertionError:
            return
    raise AssertionError("150 schedules passed with it")
