"""The prompt planner and the refusals of gk_prompt_* on the host (no GPU): every
row meets every key tile it sees exactly once, whatever is split or stacked."""
import random

import numpy as np
import pytest


@pytest.fixture(scope="module")
def gk():
    from paged_kv_cache_pool_gb300 import build
    build.build()
    from paged_kv_cache_pool_gb300 import binding
    return binding


def _up(n):
    return -(-n // 128)


def _check_plan(gk, pool, g, hkv, new, bases, lps, ctx):
    """Items against a row-by-row count; returns the summary."""
    batch = gk.PromptBatch(new, bases, lps, ctx, None, 1 << 20)
    plan = gk.gk_prompt_plan_build(pool, batch)
    try:
        info = gk.gk_prompt_plan_info(plan)
        begin, items = gk.gk_prompt_plan_items(plan)
    finally:
        gk.gk_prompt_plan_destroy(plan)
    tpt = 128 // g
    start = np.cumsum([0] + list(new))
    T = int(start[-1])
    assert info["tokens"] == T and info["items"] == len(items) == begin[-1] and (np.diff(begin) > 0).all()
    assert info["ctas"] == len(begin) - 1 <= 152
    past = [lp + c for lp, c in zip(lps, ctx)]
    assert info["flops"] == 4 * 128 * g * hkv * sum(n * p + n * (n + 1) // 2 for n, p in zip(new, past))
    seen = np.zeros((hkv, T, max([0] + [_up(lp) + _up(c) + _up(n) for n, lp, c in zip(new, lps, ctx)])), np.int32)
    entries = []
    for req, run, head, tok0, tile0, ntile, entry, nt_hot in items:
        assert ntile > 0 and tok0 % (2 * tpt) == 0 and 0 <= head < hkv
        n = run if run else new[req]
        a, b = start[req] + tok0, start[req] + min(n, tok0 + 2 * tpt)
        assert a < b
        if run:
            assert tile0 + ntile <= nt_hot and entry >= 0
            assert len({bases[r] for r in range(len(new)) if start[r + 1] > a and start[r] < b and new[r]}) == 1
        seen[head, a:b, tile0:tile0 + ntile] += 1
        if entry >= 0:
            entries.append(entry)
    assert len(set(entries)) == len(entries) and (not entries or max(entries) < info["partials"])
    for r, n in enumerate(new):
        for i in range(n):
            t = _up(lps[r]) + _up(ctx[r]) + i // 128 + 1
            row = seen[:, start[r] + i]
            assert (row[:, :t] == 1).all(), (r, i)
            assert (row <= 1).all()
    return info


@pytest.mark.parametrize("seed", range(30))
def test_every_row_meets_its_key_tiles_once(gk, seed):
    rnd = random.Random(seed)
    g, hkv = rnd.choice([1, 2, 4, 5, 8]), rnd.choice([1, 2, 8])
    pool = gk.gk_pool_create(1, g * hkv, hkv, 128, 40000, 1600, 16)
    try:
        lp = [rnd.choice([1, 127, 128, 129, 3000, 9000]) for _ in range(2)]
        base = [gk.gk_prefix_alloc(pool, x) for x in lp]
        n = rnd.randint(1, 24)
        hi = rnd.choice([3, 40, 400])
        new = [rnd.choice([0, 1, rnd.randint(0, hi), hi]) for _ in range(n)]
        which = [rnd.choice([-1, 0, 0, 0, 1]) for _ in range(n)]
        if rnd.random() < 0.5:
            which.sort()
        ctx = [rnd.choice([0, 0, 1, 128, rnd.randint(0, 2000)]) for _ in range(n)]
        _check_plan(gk, pool, g, hkv, new, [base[w] if w >= 0 else -1 for w in which],
                    [lp[w] if w >= 0 else 0 for w in which], ctx)
    finally:
        gk.gk_pool_destroy(pool)


def test_few_rows_over_many_keys_are_split_and_neighbours_stacked(gk):
    pool = gk.gk_pool_create(1, 32, 8, 128, 20000, 1600, 16)
    try:
        base = gk.gk_prefix_alloc(pool, 16384)
        assert _check_plan(gk, pool, 4, 8, [3], [-1], [0], [9000])["max_pieces"] > 4
        info = _check_plan(gk, pool, 4, 8, [5] * 40, [base] * 40, [16384] * 40, [100] * 40)
        assert info["stacked_requests"] == 40
        # long turns fill their own tiles: nothing to gain
        assert _check_plan(gk, pool, 4, 8, [640] * 4, [base] * 4, [16384] * 4, [0] * 4)["stacked_requests"] == 0
        assert _check_plan(gk, pool, 4, 8, [], [], [], [])["items"] == 0
        assert _check_plan(gk, pool, 4, 8, [0, 0], [-1, base], [0, 16384], [5, 0])["ctas"] == 0
    finally:
        gk.gk_pool_destroy(pool)


def test_plan_refusals(gk):
    pool = gk.gk_pool_create(1, 8, 2, 128, 1000, 160, 16)
    try:
        base = gk.gk_prefix_alloc(pool, 300)

        def refused(text, *a, **k):
            with pytest.raises(gk.GkError, match=text) as e:
                gk.gk_prompt_plan_build(pool, gk.PromptBatch(*a, **k))
            assert e.value.status == gk.GK_ERR_INVALID
        refused("negative", [3, -1])
        refused("negative", [3], None, None, [-1])
        refused("go together", [3], [base], None)
        refused("go together", [3], None, [300])
        refused("not live", [3], [base], [299])
        refused("not live", [3], [base + 1], [300])
        refused("must be 0", [3], [-1], [300])
        refused("block-table row", [3], None, None, [33], None, 2)
        refused("2\\^31", [2 ** 30, 2 ** 30, 5])
        with pytest.raises(ValueError):
            gk.PromptBatch([3, 4], [base], [300])
        lib = gk.lib()
        assert lib.gk_prompt_plan_build(None, None, None, None) == gk.GK_ERR_INVALID
        assert lib.gk_prompt_plan_update(None, None, None) == gk.GK_ERR_INVALID
        assert lib.gk_prompt_plan_info(None, None) == gk.GK_ERR_INVALID
        assert lib.gk_prompt_plan_items(None, None, None, None, None) == gk.GK_ERR_INVALID
        assert lib.gk_prompt_attn(None, None, 0, None, None) == gk.GK_ERR_INVALID
        lib.gk_prompt_plan_destroy(None)
    finally:
        gk.gk_pool_destroy(pool)


def test_launch_refusals(gk):
    torch = pytest.importorskip("torch")
    pool, other = (gk.gk_pool_create(2, 8, 2, 128, 1000, 160, 16) for _ in range(2))
    batch = gk.PromptBatch([3, 4], None, None, [0, 20], None, 2)
    plan = gk.gk_prompt_plan_build(pool, batch)
    try:
        def refused(text, layer=0, at=pool):
            with pytest.raises(gk.GkError, match=text) as e:
                gk.gk_prompt_attn(at, None, layer, batch, plan)
            assert e.value.status == gk.GK_ERR_INVALID
        refused("layer", 2)
        refused("layer", -1)
        refused("another pool", at=other)
        refused("pointers missing")
        batch.set_device(4096, 4096, 4096, 0)
        refused("pointers missing")
        batch.set_device(4096, 4096, 4096, 4096)
        refused("block table missing")
        batch.set_device(4096, 4096, 4096, 4096, None, 4096, 1)
        refused("row shorter")
        batch.set_device(4096, 4096 + 8, 4096, 4096, None, 4096, 2)
        refused("aligned")
        batch.set_device(4096, 4096, 4096, 4096)
        for field, bad in (("d_lse", 4098), ("d_block_table", 4097)):
            was = getattr(batch.c, field)
            setattr(batch.c, field, bad)
            refused("4-byte aligned")
            setattr(batch.c, field, was)
        for field, bad in (("q_stride", 1016), ("q_stride", 1028), ("k_stride", 248), ("v_stride", -256), ("out_stride", 2 ** 39)):
            setattr(batch.c, field, bad)
            refused("stride")
            setattr(batch.c, field, 0)
        refused("no device tables")
        x = torch.zeros(7, 8, 128, dtype=torch.bfloat16)
        for bad in (x[:6], x.float(), x.transpose(1, 2), x[:, :, ::2]):
            with pytest.raises(ValueError):
                batch.set_device(bad, x, x, x)
    finally:
        gk.gk_prompt_plan_destroy(plan)
        gk.gk_pool_destroy(pool)
        gk.gk_pool_destroy(other)


def test_a_refused_update_leaves_a_plan_that_does_not_run(gk):
    pool = gk.gk_pool_create(1, 8, 2, 128, 1000, 160, 16)
    batch = gk.PromptBatch([3])
    plan = gk.gk_prompt_plan_build(pool, batch)
    try:
        with pytest.raises(gk.GkError):
            gk.gk_prompt_plan_update(pool, plan, gk.PromptBatch([-3]))
        batch.set_device(4096, 4096, 4096, 4096)
        with pytest.raises(gk.GkError, match="no device tables"):
            gk.gk_prompt_attn(pool, None, 0, batch, plan)
        gk.gk_prompt_plan_update(pool, plan, batch)
        assert gk.gk_prompt_plan_info(plan)["tokens"] == 3
    finally:
        gk.gk_prompt_plan_destroy(plan)
        gk.gk_pool_destroy(pool)
