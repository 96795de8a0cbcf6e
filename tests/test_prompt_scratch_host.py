"""Device memory that a prompt plan asks for (no GPU): a partial state takes as many rows as
its block of tokens has, however many short requests are stacked over a prefix."""
import pytest

from test_prompt_host import gk  # noqa: F401  (the fixture)


def _plan(gk, pool, *step):
    plan = gk.gk_prompt_plan_build(pool, gk.PromptBatch(*step, None, 1 << 20))
    try:
        return gk.gk_prompt_plan_info(plan), gk.gk_prompt_plan_items(plan)[1]
    finally:
        gk.gk_prompt_plan_destroy(plan)


@pytest.mark.parametrize("g,d", [(4, 128), (5, 128), (1, 64), (8, 128)])
@pytest.mark.parametrize("requests", [64, 512, 2048])
def test_stacked_turns_of_a_few_tokens(gk, requests, g, d):  # noqa: F811
    hkv = 8 if g < 8 else 1
    pool = gk.gk_pool_create(1, g * hkv, hkv, d, 20000, 1600, 16)
    try:
        base = gk.gk_prefix_alloc(pool, 16384)
        new = [1 + r % 3 for r in range(requests)]
        info, items = _plan(gk, pool, new, [base] * requests, [16384] * requests, [64] * requests)
    finally:
        gk.gk_pool_destroy(pool)
    assert info["stacked_requests"] == requests and info["partials"] > 0
    # a row of a state: d outputs and an LSE, in fp32
    rows = [min(2 * (128 // g), (run or new[req]) - tok0) * g for req, run, head, tok0, t, nt, entry, hot in items if entry >= 0]
    assert len(rows) == info["partials"]
    assert info["scratch_bytes"] == sum(rows) * (d + 1) * 4
    # no row has more than a state of its own and 16 of the prefix
    assert info["scratch_bytes"] <= 17 * sum(new) * g * hkv * (d + 1) * 4


def test_a_step_without_partial_states_asks_for_none(gk):  # noqa: F811
    pool = gk.gk_pool_create(1, 32, 8, 128, 20000, 1600, 16)
    try:
        info, _ = _plan(gk, pool, [300, 5], None, None, None)
        assert info["partials"] == 0 and info["scratch_bytes"] == 0
    finally:
        gk.gk_pool_destroy(pool)
