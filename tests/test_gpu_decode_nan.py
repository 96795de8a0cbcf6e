"""Decode rows whose query holds NaN: NaN from both backends and every arrangement, split
over CTAs or not, and no other row's bits change."""
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


ARRANGEMENTS = [("dense", None, None), *((f"{m}-{k}", mode, kind) for m, mode in (("split", gk.GK_CASCADE_SPLIT), ("sequential", gk.GK_CASCADE_SEQUENTIAL))
                                         for k, kind in (("tensor", gk.GK_PREFIX_TENSOR), ("warp", gk.GK_PREFIX_WARP)))]


@pytest.mark.parametrize("name,mode,kind", ARRANGEMENTS, ids=[a[0] for a in ARRANGEMENTS])
@pytest.mark.parametrize("suffix", [[700, 3, 0, 40], [0, 0, 0, 0], [20000, 1, 5, 0]], ids=["suffixes", "prefix only", "one long"])
def test_nan_queries(name, mode, kind, suffix):
    hq, hkv, d, lp = 8, 2, 128, 1000
    eng = Engine(1, hq, hkv, d, lp, 21504, 16, seed=3)
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    base = eng.prefix_alloc(lp)
    eng.write_prefix(0, base, lp, 0, rand(lp, hkv, d), rand(lp, hkv, d))
    seqs = [eng.seq_create() for _ in suffix]
    order = [s for s, n in zip(seqs, suffix) for _ in range(n)]
    if order:
        slots, _ = eng.append_slots(order)
        eng.append_kv(0, eng.to_device(slots), rand(len(order), hkv, d), rand(len(order), hkv, d))
    table = eng.to_device(eng.block_tables(seqs, 1250))
    # the last request has no prefix, and where its suffix is empty too, no key at all
    batch = eng.batch([base] * 3 + [-1], [lp] * 3 + [0], suffix, table, 1250)
    if mode is not None:
        gk.gk_pool_set_cascade_mode(eng.pool, mode, 2 if mode == gk.GK_CASCADE_SPLIT else 0)
        gk.gk_pool_set_prefix_kernel(eng.pool, kind)
    plan = eng.plan(batch)
    q = rand(4, hq, d)
    bad = q.clone()
    rows = [(0, 0), (0, 5), (1, 7), (2, 3)] + ([(3, 1)] if suffix[3] else [])
    for r, h in rows:
        bad[r, h, 9] = float("nan")
    got = []
    for x in (q, bad):
        out, lse = torch.full((4, hq, d), 5.0, device="cuda"), torch.full((4, hq), 5.0, device="cuda")
        batch.set_device(d_q=x, d_out=out, d_lse=lse)
        eng.decode(0, batch, plan, gk.GK_BACKEND_DENSE if mode is None else gk.GK_BACKEND_CASCADE)
        torch.cuda.synchronize()
        got.append((out.cpu().numpy(), lse.cpu().numpy()))
    assert eng.device_error() == gk.GK_OK
    eng.close()
    nan = np.zeros((4, hq), bool)
    for r, h in rows:
        nan[r, h] = True
    (o0, l0), (o1, l1) = got
    assert np.isfinite(o0).all() and not np.isnan(l0).any()
    assert np.isnan(o1[nan]).all() and np.isnan(l1[nan]).all(), [(r, h, o1[r, h, :3], l1[r, h]) for r, h in rows]
    assert np.array_equal(o0[~nan], o1[~nan]) and np.array_equal(l0[~nan], l1[~nan])
