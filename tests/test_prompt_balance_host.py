"""The prompt planner where one context is far longer than the others (no GPU): however
many short requests stand beside it, no SM is left with the whole of it."""
import time

import pytest

from test_prompt_host import _check_plan, gk  # noqa: F401  (the fixture)


@pytest.mark.parametrize("requests", [40, 450, 456, 700, 2500])
@pytest.mark.parametrize("hkv", [2, 8])
def test_one_long_context_among_many_short_turns(gk, requests, hkv):  # noqa: F811
    pool = gk.gk_pool_create(1, 4 * hkv, hkv, 128, 0, 1600, 16)
    try:
        ctx = [16] * requests
        ctx[requests // 3] = 131072
        step = [1] * requests, [-1] * requests, [0] * requests, ctx
        info = _check_plan(gk, pool, 4, hkv, *step)
        plan = gk.gk_prompt_plan_build(pool, gk.PromptBatch(step[0], None, None, ctx, None, 1 << 20))
        begin, items = gk.gk_prompt_plan_items(plan)
        gk.gk_prompt_plan_destroy(plan)
    finally:
        gk.gk_pool_destroy(pool)
    # what an SM is expected to take: an item of one Q tile costs about as much as 2.6 of its key tiles besides them
    cost = [sum(2.6 + it[5] for it in items[a:b]) for a, b in zip(begin, begin[1:])]
    assert info["max_pieces"] > 1
    assert max(cost) <= 1.25 * sum(cost) / 152 + 1025 / 16, (info, max(cost), sum(cost) / 152)


def test_many_even_requests_stay_whole(gk):  # noqa: F811
    """... and are planned without a search for pieces."""
    pool = gk.gk_pool_create(1, 32, 8, 128, 0, 1600, 16)
    try:
        batch = gk.PromptBatch([200] * 1500, None, None, [500] * 1500, None, 1 << 20)
        best = 1e9
        for _ in range(5):
            t0 = time.perf_counter()
            plan = gk.gk_prompt_plan_build(pool, batch)
            best = min(best, time.perf_counter() - t0)
            info = gk.gk_prompt_plan_info(plan)
            gk.gk_prompt_plan_destroy(plan)
        assert info["items"] == 1500 * 4 * 8 and info["max_pieces"] == 1 and info["partials"] == 0
        print(f"{info['items']} items in {best * 1e3:.1f} ms")
    finally:
        gk.gk_pool_destroy(pool)
