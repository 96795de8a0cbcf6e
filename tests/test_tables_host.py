"""Refusals of gk_tables_step (no GPU): every one of them comes before any device work."""
import pytest


@pytest.fixture(scope="module")
def gk():
    from paged_kv_cache_pool_gb300 import build
    build.build()
    from paged_kv_cache_pool_gb300 import binding
    return binding


def test_refusals(gk):
    torch = pytest.importorskip("torch")
    ints = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    pool = gk.gk_pool_create(1, 8, 2, 128, 0, 160, 16)
    try:
        add, done, slots = ints(4), ints(4), torch.zeros(9, dtype=torch.int64)

        def refused(text, add=add, slots=slots, done=done, n_slots=None, **change):
            t = gk.Tables(ints(4, 3), ints(10), ints(4), ints(1))
            for k, v in change.items():
                setattr(t.c, k, v)
            with pytest.raises(gk.GkError, match=text) as e:
                gk.gk_tables_step(pool, None, t, add, slots, done, None, n_slots)
            assert e.value.status == gk.GK_ERR_INVALID
        for field in ("num_rows", "max_blocks", "capacity"):
            refused("negative", **{field: -1})
        refused("negative", n_slots=-1)
        refused("2\\^20", num_rows=(1 << 20) + 1)
        for field in ("d_table", "d_free", "d_len", "d_len_out", "d_num_free", "d_num_free_out", "d_work"):
            refused("null", **{field: None})
        refused("null", add=None)
        refused("null", done=None)
        refused("null", slots=None, n_slots=3)
        refused("aligned", d_work=4096 + 8)
        for field in ("d_table", "d_free", "d_len", "d_len_out", "d_num_free", "d_num_free_out"):
            refused("4-byte aligned", **{field: 4096 + 2})
        refused("8-byte aligned", slots=4096 + 4, n_slots=3)
        refused("no device storage")
        assert gk.lib().gk_tables_step(None, None, None, None, None, 0, None, None) == gk.GK_ERR_INVALID
        for bad in (dict(table=ints(4, 3).float()), dict(length=ints(3)), dict(num_free=ints(2)), dict(table=ints(3, 4).t()),
                    dict(length_out=ints(5))):
            with pytest.raises(ValueError):
                gk.Tables(**{**dict(table=ints(4, 3), free=ints(10), length=ints(4), num_free=ints(1)), **bad})
    finally:
        gk.gk_pool_destroy(pool)
