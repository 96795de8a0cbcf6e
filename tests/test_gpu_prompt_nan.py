"""Rows of gk_prompt_attn whose own query, or whose visible keys, hold an infinity or
NaN: they come out NaN as by the definition, whole or cut into pieces, stacked over a
prefix or not, and no other row notices.  Pieces whose keys all score minus infinity
weigh nothing."""
import numpy as np
import pytest

from prompt_ref import check
from test_gpu_prompt import Prompts

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_pool_gb300 import build
    build.build()


#: name -> new lengths, prefixes, which, cold, and whether rows of partial states come out of it
STEPS = {"whole": ([64], (), None, None, False), "pieces": ([6], (), None, [3000], True),
         "sixteen pieces": ([1, 3], (), None, [40000, 0], True),
         "stacked": ([4, 1, 16, 9] * 4, [4000], [0] * 16, [5, 0, 130, 3] * 4, True)}


def _verify(p, nan, what):
    """Rows of `nan` [T, Hq] are NaN throughout, every other row is within the counted tolerance."""
    torch.cuda.synchronize()
    out, lse = p.host(p.out), p.host(p.lse)
    assert np.isnan(out[nan]).all() and np.isnan(lse[nan]).all(), f"{what}: NaN rows came out as numbers"
    check(out[~nan], lse[~nan], [x[~nan] for x in p.want()], what)


@pytest.mark.parametrize("name", sorted(STEPS))
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_queries_that_are_no_numbers(name, bad):
    new, prefixes, which, cold, parts = STEPS[name]
    p = Prompts(128, 4, 2, new, prefixes=prefixes, which=which, cold=cold)
    nan = np.zeros((p.T, p.hq), bool)
    for row, head in ((0, 0), (0, 7), (p.T - 1, 3), (p.T // 2, 5)):
        p.q[row, head] = bad
        nan[row, head] = True
    p.run()
    assert (p.info()["partials"] > 0) == parts
    with np.errstate(invalid="ignore"):
        _verify(p, nan, f"{name} {bad}")
    p.close()


@pytest.mark.parametrize("d,g", [(64, 1), (64, 4), (128, 5)])
def test_one_channel_is_enough(d, g):
    p = Prompts(d, g, 2, [6, 2], prefixes=[2000], which=[0, 0], cold=[1500, 0])
    p.q[1, 1, 3] = float("nan")
    p.run()
    assert p.info()["partials"] > 0
    nan = np.zeros((p.T, p.hq), bool)
    nan[1, 1] = True
    with np.errstate(invalid="ignore"):
        _verify(p, nan, "one channel")
    p.close()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_keys_that_are_no_numbers_reach_every_row_that_sees_them(bad):
    """A new key of a step in pieces: its own row and the later ones."""
    p = Prompts(128, 4, 2, [9], cold=[3000])
    p.q[:, :, 3] = p.q[:, :, 3].abs() + 0.5     # an infinity in K then scores +infinity, which has no softmax
    p.k[5, 1, 3] = bad
    p.run()
    assert p.info()["partials"] > 0
    nan = np.zeros((p.T, p.hq), bool)
    nan[5:, 4:] = True
    with np.errstate(invalid="ignore"):
        _verify(p, nan, f"key {bad}")
    p.close()


def test_pieces_of_keys_that_score_minus_infinity_weigh_nothing():
    p = Prompts(128, 4, 2, [6], cold=[3000])
    p.q[:, :, 0] = p.q[:, :, 0].abs() + 0.5
    # the first 1500 COLD tokens, whole pieces among them, in the pool and in what the check reads
    tokens = np.arange(1500)
    slots = p.table[0].cpu().numpy()[tokens // p.page].astype(np.int64) * p.page + tokens % p.page
    p.cold[0][p.layer, torch.from_numpy(slots).cuda(), :, 0] = float("-inf")
    p.past[0][0][:1500, :, 0] = float("-inf")
    p.run()
    assert p.info()["max_pieces"] > 4
    with np.errstate(invalid="ignore"):
        _verify(p, np.zeros((p.T, p.hq), bool), "minus infinity")
    p.close()


@pytest.mark.parametrize("name", sorted(STEPS))
def test_rows_whose_every_score_is_minus_infinity(name):
    """out = 0 and lse = -inf, whole, in pieces and stacked."""
    new, prefixes, which, cold, parts = STEPS[name]
    p = Prompts(128, 4, 2, new, prefixes=prefixes, which=which, cold=cold, spare_nan=False)
    p.q[:, :, 0] = p.q[:, :, 0].abs() + 0.5
    p.q[:, 1, 0] = -p.q[:, 1, 0]        # ... but of head 1 plus infinity, which has no softmax
    for x in (p.hot[0].view(-1, p.d), p.cold[0], p.k):
        x[..., 0] = float("-inf")
    p.run()
    torch.cuda.synchronize()
    assert (p.info()["partials"] > 0) == parts
    out, lse = p.host(p.out), p.host(p.lse)
    assert np.isnan(out[:, 1]).all() and np.isnan(lse[:, 1]).all()
    rest = [h for h in range(p.hq) if h != 1]
    assert (out[:, rest] == 0).all() and (lse[:, rest] == -np.inf).all()
    p.close()


@pytest.mark.parametrize("scale", [1.0, 8.0, 64.0])
def test_large_finite_values(scale):
    """V up to 2^62, over scores that rise far above a row's first keys: nothing overflows before the division by Z."""
    p = Prompts(128, 4, 2, [300, 20], cold=[0, 2000], scale=scale)
    p.v.mul_(2.0 ** 60).clamp_(-2.0 ** 62, 2.0 ** 62)
    p.run().verify(f"large values, queries by {scale}")
    p.close()
