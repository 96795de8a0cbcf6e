"""What gk_tables_step takes as tensors (no GPU): flags of another type and arrays too
short are refused before the kernel reads or writes past their ends."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def gk():
    from paged_kv_cache_pool_gb300 import build
    build.build()
    from paged_kv_cache_pool_gb300 import binding
    return binding


def ints(*n):
    return torch.zeros(*n, dtype=torch.int32)


def test_row_arrays_and_the_slot_mapping(gk):
    pool = gk.gk_pool_create(1, 8, 2, 128, 0, 160, 16)
    good = dict(d_add=ints(4), d_slot_mapping=torch.zeros(9, dtype=torch.int64), d_done=ints(4), d_release=ints(4))
    tables = gk.Tables(ints(4, 3), ints(10), ints(4), ints(1))
    wide = dict(d_add=ints(6), d_done=ints(2, 2), n_slots=9)       # longer ones, and [2, 2] for four rows, hold the rows
    addresses = dict(d_add=4096, d_done=4096, d_slot_mapping=4096, d_release=4096, n_slots=9)
    try:
        for ok in ({}, wide, addresses, dict(d_release=None), dict(n_slots=0), dict(n_slots=8)):
            with pytest.raises(gk.GkError, match="no device storage"):    # every check passed
                gk.gk_tables_step(pool, None, tables, **{**good, **ok})
        row_like = [torch.zeros(4, dtype=torch.bool), torch.zeros(4, dtype=torch.int64), torch.zeros(4), ints(3), ints(8)[::2],
                    ints(1).expand(4), torch.zeros(4, dtype=torch.int8)]
        bad = [(k, x) for k in ("d_add", "d_done", "d_release") for x in row_like]
        long = torch.zeros(9, dtype=torch.int64)
        bad += [("d_slot_mapping", x) for x in (long.int(), long.double(), torch.zeros(18, dtype=torch.int64)[::2])]
        bad += [("n_slots", 10)]
        for name, x in bad:
            with pytest.raises(ValueError):
                gk.gk_tables_step(pool, None, tables, **{**good, name: x})
    finally:
        gk.gk_pool_destroy(pool)


def test_tables_are_int32(gk):
    for other in (torch.zeros(4, 3, dtype=torch.uint32), torch.zeros(4, 3), torch.zeros(4, 3, dtype=torch.int64)):
        with pytest.raises(ValueError):
            gk.Tables(other, ints(10), ints(4), ints(1))
