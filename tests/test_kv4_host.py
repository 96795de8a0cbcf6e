"""4-bit pools and the calls on q, k, v rows without a GPU: sizes, plans and refusals."""
import ctypes
import random
import threading

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_prompt_tensors_host import OnGpu, bf16  # noqa: E402


@pytest.fixture(scope="module")
def gk():
    from paged_kv_cache_pool_gb300 import build
    build.build()
    from paged_kv_cache_pool_gb300 import binding
    return binding


@pytest.fixture
def pool(gk):
    p = gk.gk_pool_create_kv4(2, 8, 2, 128, 1000, 64 * 16, 16, 0)
    yield p
    gk.gk_pool_destroy(p)


def refused(gk, status, call, *args, **kw):
    with pytest.raises(gk.GkError) as e:
        call(*args, **kw)
    assert e.value.status == status, e.value
    return str(e.value)


@pytest.mark.parametrize("hkv,d,want", [(1, 64, 80), (2, 64, 144), (3, 64, 224), (8, 64, 576), (1, 128, 144), (5, 128, 720), (8, 128, 1152),
                                        (0, 64, 0), (9, 128, 0), (8, 96, 0), (-1, 64, 0)])
def test_row_bytes(gk, hkv, d, want):
    assert gk.gk_kv4_row_bytes(hkv, d) == want


def test_pool_needs_one_store(gk):
    """A 4-bit pool has one COLD store: cold_v must be NULL; a bf16 pool still needs both."""
    def create(fn, hot_k, hot_v, cold_k, cold_v):
        cfg = gk.gk_pool_config(1, 4, 2, 64, 64, 64, 1, 0, 0, hot_k, hot_v, cold_k, cold_v)
        out = ctypes.c_void_p()
        st = fn(ctypes.byref(cfg), ctypes.byref(out))
        if st == gk.GK_OK:
            gk.gk_pool_destroy(out.value)
        return st
    kv4, both = gk.lib().gk_pool_create_kv4, gk.lib().gk_pool_create
    assert create(kv4, 4096, 8192, 12288, None) == gk.GK_OK
    assert create(kv4, None, None, None, None) == gk.GK_OK          # bookkeeping only
    assert create(kv4, 4096, 8192, 12288, 16384) == gk.GK_ERR_INVALID
    assert create(kv4, 4096, 8192, None, None) == gk.GK_ERR_INVALID
    assert create(kv4, None, None, 12288, None) == gk.GK_ERR_INVALID
    assert create(kv4, 4096, 8192, 12288 + 16, None) == gk.GK_ERR_INVALID
    assert create(both, 4096, 8192, 12288, 16384) == gk.GK_OK
    assert create(both, 4096, 8192, 12288, None) == gk.GK_ERR_INVALID
    with pytest.raises(ValueError, match="rows of 144 bytes"):
        gk.gk_pool_create_kv4(1, 4, 2, 64, 64, 64, 1, 0, 4096, 8192, torch.zeros(64 * 144 - 1, dtype=torch.uint8))
    assert gk.lib().gk_pool_create_kv4(None, None) == gk.GK_ERR_INVALID


def test_block_manager_is_the_same(gk, pool):
    other = gk.gk_pool_create(2, 8, 2, 128, 1000, 64 * 16, 16, 0)
    try:
        seqs = [[gk.gk_seq_create(p) for _ in range(3)] for p in (pool, other)]
        for p, s in zip((pool, other), seqs):
            s.append(gk.gk_seq_fork(p, s[0]))
        got = [gk.gk_seq_append_slots(p, [s[0]] * 20 + [s[1]] * 7) for p, s in zip((pool, other), seqs)]
        assert got[0][0].tolist() == got[1][0].tolist() and got[0][1].tolist() == got[1][1].tolist()
        assert gk.gk_cold_stats(pool) == gk.gk_cold_stats(other)
        assert gk.gk_prefix_alloc(pool, 100) == gk.gk_prefix_alloc(other, 100)
    finally:
        gk.gk_pool_destroy(other)


def test_plans(gk, pool):
    """Sequential plans; a request that one segment covers, and no prefix, needs no partial state; bytes are those of 4-bit rows."""
    base = gk.gk_prefix_alloc(pool, 300)
    for mode in (gk.GK_CASCADE_AUTO, gk.GK_CASCADE_SPLIT):
        gk.gk_pool_set_cascade_mode(pool, mode)
        plan = gk.gk_plan_build(pool, gk.Batch([-1, base, -1], [0, 300, 0], [40, 500, 0], None, 64))
        info = gk.gk_plan_info(plan)
        assert info["cascade_split"] == 0 and info["suffix_bytes"] == 540 * 2 * 144 and info["prefix_bytes"] == 300 * 2 * 128 * 4
        assert info["dense_bytes"] == info["suffix_bytes"] + info["prefix_bytes"]
        begin, segs = gk.gk_plan_segments(plan)
        whole = [s.tolist() for s in segs if s[0] == 0]
        assert whole == [[0, 0, 40, -1]]
        entries = sorted(int(s[3]) for s in segs if s[0] == 1)
        assert len(entries) == len(set(entries)) and sum(int(s[2] - s[1]) for s in segs if s[0] == 1) == 500
        assert info["num_partials"] > max(entries)
        assert all(b > a for a, b in zip(begin, begin[1:]))
        gk.gk_plan_destroy(plan)


@pytest.mark.parametrize("d,hkv", [(128, 8), (64, 1), (128, 3), (64, 8)])
def test_work_covers_every_token_once(gk, d, hkv):
    """The gather's pieces: every token once and in order, as many CTAs as run at a time, pieces of at least 64 tokens but at ends,
    partial states one run a request, whole requests alone where they fit."""
    rnd = random.Random(d + hkv)
    p = gk.gk_pool_create_kv4(1, hkv, hkv, d, 5000, 1 << 22, 1, 0)
    base = gk.gk_prefix_alloc(p, 1000)
    try:
        for lens in ([1], [0, 0], [131072], [700] * 9, [20] * 400, [64] * 304, [65] * 305, [4096, 1, 0, 4095], [2] * 5000,
                     [rnd.randint(1, 4096) for _ in range(368)], [rnd.randint(0, 70) for _ in range(900)], [100000] + [5] * 600):
            for hot in (False, True):
                n = len(lens)
                b = gk.Batch([base if hot else -1] * n, [1000 if hot else 0] * n, lens, None, 131072)
                plan = gk.gk_plan_build(p, b)
                begin, segs = gk.gk_plan_segments(plan)
                info = gk.gk_plan_info(plan)
                got = {}
                for r, t0, t1, _ in segs.tolist():
                    assert t0 == got.get(r, 0) and t1 > t0
                    got[r] = t1
                assert all(got.get(r, 0) == x for r, x in enumerate(lens))
                assert begin[0] == 0 and begin[-1] == len(segs) and (np.diff(begin) > 0).all()
                assert len(begin) - 1 == info["suffix_ctas"] <= 152 * 16
                pieces = np.bincount(segs[:, 0], minlength=n) if len(segs) else np.zeros(n, int)
                assert pieces.max(initial=0) <= 513
                for r, t0, t1, _ in segs.tolist():
                    assert t1 - t0 >= 64 or t1 == lens[r] and (t0 == 0 or t1 - t0 >= 1)
                entries = {}
                for r, _, _, e in segs.tolist():
                    if not hot and pieces[r] == 1:
                        assert e == -1
                    else:
                        entries.setdefault(r, []).append(e)
                every = [e for v in entries.values() for e in v]
                assert len(set(every)) == len(every) and all(v == list(range(v[0], v[0] + len(v))) for v in entries.values())
                assert not every or max(every) < info["num_partials"]
                gk.gk_plan_destroy(plan)
    finally:
        gk.gk_pool_destroy(p)


def test_calls_of_bf16_pools_refuse(gk, pool):
    b = gk.Batch([-1], [0], [40], 4096, 64, 4096, 4096, 4096)
    plan = gk.gk_plan_build(pool, b)
    for call in (gk.gk_decode_dense, gk.gk_decode_cascade, gk.gk_cascade_levels, gk.gk_cascade_prefix, gk.gk_cascade_suffix,
                 gk.gk_cascade_merge):
        assert "gk_decode_kv4" in refused(gk, gk.GK_ERR_UNSUPPORTED, call, pool, None, 0, b, plan)
    refused(gk, gk.GK_ERR_UNSUPPORTED, gk.gk_decode_dense_static, pool, None, 0, b)
    refused(gk, gk.GK_ERR_UNSUPPORTED, gk.gk_sm_speeds_measure, pool, None, 0, b, plan)
    refused(gk, gk.GK_ERR_UNSUPPORTED, gk.gk_calibrate, pool)
    refused(gk, gk.GK_ERR_UNSUPPORTED, gk.gk_dispatch, pool, plan)
    gk.gk_plan_destroy(plan)
    refused(gk, gk.GK_ERR_UNSUPPORTED, gk.gk_prompt_plan_build, pool, gk.PromptBatch([5, 5], None, None, [0, 3], 4096, 64))
    gk.gk_prompt_plan_destroy(gk.gk_prompt_plan_build(pool, gk.PromptBatch([5, 5], None, None, [0, 0], 4096, 64)))


def test_decode_refuses(gk, pool):
    def batch(**kw):
        b = gk.Batch([-1], [0], [40], 4096, 64, 4096, None, 4096)
        for k, v in kw.items():
            setattr(b.c, k, v)
        return b
    plan = gk.gk_plan_build(pool, batch())
    bf16_pool = gk.gk_pool_create(2, 8, 2, 128, 1000, 64 * 16, 16, 0)
    try:
        other = gk.gk_plan_build(bf16_pool, batch())
        refused(gk, gk.GK_ERR_UNSUPPORTED, gk.gk_decode_kv4, bf16_pool, None, 0, batch(), other, 4096)
        assert "another pool" in refused(gk, gk.GK_ERR_INVALID, gk.gk_decode_kv4, pool, None, 0, batch(), other, 4096)
        gk.gk_plan_destroy(other)
    finally:
        gk.gk_pool_destroy(bf16_pool)
    for layer in (-1, 2):
        assert "layer" in refused(gk, gk.GK_ERR_INVALID, gk.gk_decode_kv4, pool, None, layer, batch(), plan, 4096)
    # a pool without storage has no device tables
    assert "device" in refused(gk, gk.GK_ERR_INVALID, gk.gk_decode_kv4, pool, None, 0, batch(), plan, 4096)
    for bad in (None, None, None):
        assert gk.lib().gk_decode_kv4(bad, None, 0, None, None, None) == gk.GK_ERR_INVALID
    for y in (torch.zeros(1, 8, 128), torch.zeros(2, 8, 128, dtype=torch.bfloat16), torch.zeros(1, 4, 128, dtype=torch.bfloat16),
              torch.zeros(1, 128, 8, dtype=torch.bfloat16).transpose(1, 2)):
        with pytest.raises(ValueError, match="out must be"):
            gk.gk_decode_kv4(pool, None, 0, batch(), plan, OnGpu(y))
    with pytest.raises(ValueError, match="on the GPU"):
        gk.gk_decode_kv4(pool, None, 0, batch(), plan, torch.zeros(1, 8, 128, dtype=torch.bfloat16))
    gk.gk_plan_destroy(plan)


GOOD = dict(num_tokens=7, rot_dim=64, interleaved=0, eps=1e-6, num_positions=100, d_cos_sin=4096, d_positions=4100, d_q_weight=4096,
            d_k_weight=4096, d_q=4096, d_k=4096, d_v=4096, d_q_out=8192, d_k_out=8192)
INVALID = [dict(num_tokens=-1), dict(num_tokens=(1 << 27) + 1), dict(interleaved=2), dict(eps=-1.0), dict(eps=float("nan")),
           dict(num_positions=-1), dict(d_cos_sin=None), dict(d_positions=None), dict(d_q_out=None), dict(d_q=None), dict(d_q=4098),
           dict(d_k=4104), dict(d_q_out=8200), dict(d_k_out=8208 + 2), dict(d_q_weight=4104), dict(d_k_weight=4098), dict(d_cos_sin=4104),
           dict(d_positions=4102), dict(q_stride=8 * 128 - 8), dict(q_stride=8 * 128 + 4), dict(k_stride=128), dict(k_stride=-256),
           dict(q_out_stride=1), dict(k_out_stride=(1 << 38) + 8)]


@pytest.mark.parametrize("change", INVALID, ids=lambda c: "-".join(f"{k}={v}" for k, v in c.items()))
def test_rows_that_are_refused(gk, pool, change):
    x = gk.gk_qkv(**{**GOOD, **change})
    assert gk.lib().gk_qk_norm_rope(pool, None, ctypes.byref(x)) == gk.GK_ERR_INVALID
    assert "storage" not in gk.gk_last_error(pool)
    assert gk.lib().gk_append_qkv(pool, None, 0, ctypes.byref(x), 4096, 0, None) == gk.GK_ERR_INVALID
    assert "storage" not in gk.gk_last_error(pool)


def test_rows_good_and_bad_for_one_call(gk, pool):
    def rope(**change):
        st = gk.lib().gk_qk_norm_rope(pool, None, ctypes.byref(gk.gk_qkv(**{**GOOD, **change})))
        return st, gk.gk_last_error(pool)

    def append(layer=0, slots=4096, n_cow=0, cow=None, **change):
        st = gk.lib().gk_append_qkv(pool, None, layer, ctypes.byref(gk.gk_qkv(**{**GOOD, **change})), slots, n_cow, cow)
        return st, gk.gk_last_error(pool)
    # everything in order: what is missing is the pool's storage
    for st, text in (rope(), rope(d_v=None), rope(d_q=None, d_q_out=None), rope(d_k=None, d_k_out=None), rope(rot_dim=0, d_cos_sin=None),
                     append(), append(d_k_out=None), append(d_q=None, d_q_out=None), append(n_cow=2, cow=4096), rope(num_tokens=0, d_q=None),
                     append(num_tokens=0, slots=None), rope(d_v=4098)):
        assert st == gk.GK_ERR_INVALID and "storage" in text, text
    for r in (8, 24, 144, -16, 130):
        assert rope(rot_dim=r)[0] == append(rot_dim=r)[0] == gk.GK_ERR_UNSUPPORTED
    for st, text in (rope(d_k_out=None), append(d_k=None), append(d_v=None), append(d_v=4104), append(v_stride=128), append(layer=2),
                     append(layer=-1), append(slots=None), append(slots=4100), append(n_cow=1), append(n_cow=-1), append(n_cow=1, cow=4098)):
        assert st == gk.GK_ERR_INVALID and "storage" not in text, text
    assert gk.lib().gk_qk_norm_rope(None, None, None) == gk.GK_ERR_INVALID
    assert gk.lib().gk_append_qkv(pool, None, 0, None, None, 0, None) == gk.GK_ERR_INVALID


def test_append_of_misaligned_rows_refuses(gk, pool):
    append = lambda layer=0, n=3, s=4096, k=4096, v=4096, n_cow=0, cow=None: (  # noqa: E731
        gk.lib().gk_append_kv(pool, None, layer, n, s, k, v, n_cow, cow), gk.gk_last_error(pool))
    assert "storage" in append()[1] and "storage" in append(n=0, s=None, k=None, v=None, n_cow=1, cow=4100)[1]
    for st, text in (append(k=4104), append(v=4098), append(s=4100), append(n_cow=1, cow=4098), append(k=None), append(layer=2)):
        assert st == gk.GK_ERR_INVALID and "storage" not in text, text


def test_read_refuses(gk, pool):
    read = lambda layer=0, n=3, s=4096, k=4096, v=4096, ks=0, vs=0: (  # noqa: E731
        gk.lib().gk_read_kv(pool, None, layer, n, s, k, v, ks, vs), gk.gk_last_error(pool))
    assert "storage" in read()[1] and "storage" in read(ks=264, vs=256)[1]
    for st, text in (read(layer=2), read(layer=-1), read(n=-1), read(n=(1 << 27) + 1), read(s=None), read(k=None), read(v=None),
                     read(k=4104), read(v=4098), read(s=4100), read(ks=248), read(vs=260), read(ks=-256)):
        assert st == gk.GK_ERR_INVALID and "storage" not in text, text
    assert gk.lib().gk_read_kv(None, None, 0, 0, None, None, None, 0, 0) == gk.GK_ERR_INVALID


def rows(gk, **change):
    t = dict(q=bf16(7, 8, 128), k=bf16(7, 2, 128), v=bf16(7, 2, 128), q_out=bf16(7, 8, 128), k_out=bf16(7, 2, 128),
             positions=OnGpu(torch.zeros(7, dtype=torch.int32)))
    return {**t, **change}


def test_tensors_of_rows(gk, pool):
    table = OnGpu(torch.zeros(100, 64))
    rope = gk.Rope(table, None, True, bf16(128), None)
    rope.set(pool, n=7, **rows(gk))
    assert (rope.c.rot_dim, rope.c.interleaved, rope.c.num_positions, rope.c.num_tokens) == (64, 1, 100, 7)
    assert (rope.c.q_stride, rope.c.k_stride, rope.c.v_stride) == (1024, 256, 256) and rope.c.d_k_weight is None
    fused = torch.zeros(7, 12 * 128 + 8, dtype=torch.bfloat16)
    q, k, v = (OnGpu(fused[:, a:b].view(7, -1, 128)) for a, b in ((0, 1024), (1024, 1280), (1280, 1536)))
    rope.set(pool, n=7, **rows(gk, q=q, k=k, v=v))
    assert rope.c.q_stride == rope.c.k_stride == rope.c.v_stride == 1544
    for change in (dict(q=bf16(7, 4, 128)), dict(k=bf16(7, 8, 128)), dict(q=bf16(6, 8, 128)), dict(q=bf16(7, 8, 64)),
                   dict(v=OnGpu(torch.zeros(7, 2, 128))), dict(q_out=OnGpu(torch.zeros(7, 8, 256, dtype=torch.bfloat16)[..., ::2])),
                   dict(k=OnGpu(torch.zeros(1, 2, 128, dtype=torch.bfloat16).expand(7, 2, 128))),
                   dict(k=torch.zeros(7, 2, 128, dtype=torch.bfloat16)), dict(positions=None),
                   dict(positions=OnGpu(torch.zeros(7, dtype=torch.int64))), dict(positions=OnGpu(torch.zeros(6, dtype=torch.int32))),
                   dict(positions=OnGpu(torch.zeros(14, dtype=torch.int32)[::2])), dict(positions=torch.zeros(7, dtype=torch.int32))):
        with pytest.raises(ValueError):
            rope.set(pool, n=7, **rows(gk, **change))
    # the same layouts for another pool: its geometry counts
    other = gk.gk_pool_create(1, 16, 2, 128, 64, 64, 1)
    with pytest.raises(ValueError, match="heads"):
        rope.set(other, n=7, **rows(gk))
    gk.gk_pool_destroy(other)
    with pytest.raises(ValueError, match="weights"):
        gk.Rope(None, None, False, bf16(64)).set(pool, n=7, **rows(gk))
    for bad in (torch.zeros(100, 64, dtype=torch.float64), torch.zeros(64), torch.zeros(64, 100).t()):
        with pytest.raises(ValueError, match="cos_sin"):
            gk.Rope(OnGpu(bad))
    with pytest.raises(ValueError, match="rot_dim"):
        gk.Rope(table, 128)
    with pytest.raises(ValueError, match="cos_sin"):
        gk.Rope(None, 64)
    with pytest.raises(ValueError, match="cos_sin"):
        gk.Rope(torch.zeros(100, 64))
    for w in (OnGpu(torch.zeros(128)), bf16(1, 128), torch.zeros(128, dtype=torch.bfloat16)):
        with pytest.raises(ValueError, match="weight"):
            gk.Rope(None, None, False, None, w)


def test_slots_of_tensors(gk, pool):
    rope = gk.Rope()
    t = rows(gk)
    with pytest.raises(ValueError, match="on the GPU"):
        gk.gk_append_qkv(pool, None, 0, rope, None, torch.zeros(7, dtype=torch.int64), t["q"], t["k"], t["v"])
    for slots in (torch.zeros(7, dtype=torch.int32), torch.zeros(6, dtype=torch.int64), torch.zeros(14, dtype=torch.int64)[::2]):
        with pytest.raises(ValueError, match="slot"):
            gk.gk_append_qkv(pool, None, 0, rope, None, OnGpu(slots), t["q"], t["k"], t["v"])
        with pytest.raises(ValueError, match="slot"):
            gk.gk_read_kv(pool, None, 0, OnGpu(slots), t["k"], t["v"], n=7)
    with pytest.raises(ValueError, match="heads"):
        gk.gk_read_kv(pool, None, 0, OnGpu(torch.zeros(7, dtype=torch.int64)), t["q"], t["v"])
    with pytest.raises(ValueError, match="copy-on-write"):
        gk.gk_append_qkv(pool, None, 0, rope, None, OnGpu(torch.zeros(7, dtype=torch.int64)), t["q"], t["k"], t["v"],
                         d_cow_pairs=OnGpu(torch.zeros(4, dtype=torch.int64)))


class Library:
    """Stands in for libgk: a call on rows says what it was given once the other thread's call is under way too."""

    def __init__(self, calls):
        self.together, self.got = threading.Barrier(calls), {}

    def gk_qk_norm_rope(self, pool, stream, ref):
        self.together.wait(20)
        c = ref._obj
        self.got[stream] = {f: getattr(c, f) for f, _ in c._fields_}
        return 0

    def gk_append_qkv(self, pool, stream, layer, ref, slots, n_cow, cow):
        return self.gk_qk_norm_rope(pool, stream, ref)


@pytest.mark.parametrize("append", [False, True])
def test_threads_that_share_a_rope(gk, monkeypatch, append):
    """Two threads, each with a pool and rows of its own, in a call at once: either's rows are its own."""
    monkeypatch.setattr(gk, "_lib", Library(2))
    monkeypatch.setattr(gk, "_geometry", {1: (8, 2, 128), 2: (4, 4, 64)})
    rope = gk.Rope(OnGpu(torch.zeros(100, 64)), None, True)
    failed = []

    def run(pool, n):
        try:
            for _ in range(20):
                at = [pool * 1000000 + 4096 * i for i in range(7)]
                if append:
                    gk.gk_append_qkv(pool, pool, 0, rope, at[0], at[1], at[2], at[3], at[4], at[5], at[6], n=n)
                else:
                    gk.gk_qk_norm_rope(pool, pool, rope, at[0], at[2], at[3], at[5], at[6], n=n)
                got = gk._lib.got[pool]
                want = dict(num_tokens=n, rot_dim=64, interleaved=1, num_positions=100, d_cos_sin=4096, d_positions=at[0], d_q=at[2],
                            d_k=at[3], d_v=at[4] if append else None, d_q_out=at[5], d_k_out=at[6])
                assert {f: got[f] for f in want} == want
        except Exception as e:
            failed.append(e)
    threads = [threading.Thread(target=run, args=x) for x in ((1, 7), (2, 300))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


def test_layouts_are_checked_by_each_thread(gk, pool, monkeypatch):
    """A layout that one thread has seen is another's to check, strides and all."""
    rope = gk.Rope(OnGpu(torch.zeros(100, 64)))
    fused = torch.zeros(7, 12 * 128, dtype=torch.bfloat16)
    q, k, v = (OnGpu(fused[:, a:b].view(7, -1, 128)) for a, b in ((0, 1024), (1024, 1280), (1280, 1536)))
    rope.set(pool, n=7, **rows(gk, q=q, k=k, v=v))
    seen = []

    def other():
        rope.set(pool, n=7, **rows(gk))
        seen.append((rope.c.num_tokens, rope.c.q_stride))
        try:
            rope.set(pool, n=7, **rows(gk, q=bf16(7, 4, 128)))
        except ValueError:
            rope.set(pool, n=7, **rows(gk, q=q, k=k, v=v))
            seen.append((rope.c.num_tokens, rope.c.q_stride, rope.c.rot_dim))
    t = threading.Thread(target=other)
    t.start()
    t.join()
    assert seen == [(7, 1024), (7, 1536, 64)] and rope.c.q_stride == 1536


def test_queries_of_a_decode_are_packed(gk, pool, monkeypatch):
    """Views of a fused projection, which append_qkv rotates in place, are refused where the rows are read as packed ones; so are
    queries and an lse of too few rows, of another type, or on the host."""
    fused = OnGpu(torch.zeros(3, 12 * 128, dtype=torch.bfloat16)[:, :1024].view(3, 8, 128))
    batch = gk.Batch([-1] * 3, [0] * 3, [40] * 3, 4096, 64, 8192, None, 12288)
    plan = gk.gk_plan_build(pool, batch)
    with pytest.raises(ValueError, match="q must be contiguous"):
        batch.set_device(d_q=fused, d_lse=16384)
    with pytest.raises(ValueError, match="lse must be contiguous"):
        batch.set_device(d_q=bf16(3, 8, 128), d_lse=OnGpu(torch.zeros(3, 16)[:, ::2]))
    assert (batch.c.d_q, batch.c.d_lse) == (8192, 12288)
    with pytest.raises(ValueError, match="q must be contiguous"):
        gk.Batch([-1] * 3, [0] * 3, [40] * 3, 4096, 64, fused)
    called = []
    monkeypatch.setattr(gk, "_lib", type("Lib", (), {"gk_decode_kv4": lambda self, *a: called.append(a) or 0})())
    out = bf16(3, 8, 128)
    good = [8192, bf16(3, 8, 128), bf16(4, 8, 128), bf16(3, 1024), OnGpu(fused.x[:, :, :].contiguous()),
            OnGpu(torch.zeros(1, 12 * 128, dtype=torch.bfloat16)[:, :1024].view(1, 8, 128).expand(1, 8, 128))]
    for q in good[:-1]:
        gk.gk_decode_kv4(pool, None, 0, batch.set_device(d_q=q, d_lse=OnGpu(torch.zeros(3, 8))), plan, out)
    assert len(called) == 5
    # one request's row is packed however its projection strides
    one = gk.Batch([-1], [0], [40], 4096, 64).set_device(d_q=good[-1])
    gk.gk_decode_kv4(pool, None, 0, one, plan, bf16(1, 8, 128))
    for q in (bf16(2, 8, 128), bf16(3, 8, 64), OnGpu(torch.zeros(3, 8, 128)), torch.zeros(3, 8, 128, dtype=torch.bfloat16)):
        with pytest.raises(ValueError, match="q must be bf16"):
            gk.gk_decode_kv4(pool, None, 0, batch.set_device(d_q=q), plan, out)
    batch.set_device(d_q=8192)
    for lse in (OnGpu(torch.zeros(2, 8)), OnGpu(torch.zeros(3, 8, dtype=torch.bfloat16)), torch.zeros(3, 8)):
        with pytest.raises(ValueError, match="lse must be fp32"):
            gk.gk_decode_kv4(pool, None, 0, batch.set_device(d_lse=lse), plan, out)
    gk.gk_decode_kv4(pool, None, 0, batch.set_device(), plan, out)
    assert len(called) == 7
    monkeypatch.undo()
    gk.gk_plan_destroy(plan)


@pytest.mark.parametrize("d,hkv", [(64, 1), (128, 1), (64, 2)])
def test_pieces_of_a_request_are_at_most_512(gk, d, hkv):
    """Lengths that leave a remainder, alone and behind requests that fill a part of a CTA."""
    rnd = random.Random(hkv)
    p = gk.gk_pool_create_kv4(1, hkv, hkv, d, 64, 1 << 24, 1, 0)
    try:
        for n in [33279, 131583, 512 * 64 + 511, 512 * 64 + 1, 511 * 64 + 65, 511 * 96 + 1, 1 << 20, (1 << 22) - 1] + [
                rnd.randint(20000, 300000) for _ in range(40)]:
            for ahead in ([], [70], [5] * 31, [rnd.randint(1, 500) for _ in range(rnd.randint(1, 40))]):
                lens = ahead + [n] + ahead
                plan = gk.gk_plan_build(p, gk.Batch([-1] * len(lens), [0] * len(lens), lens, None, n))
                begin, segs = gk.gk_plan_segments(plan)
                gk.gk_plan_destroy(plan)
                pieces = np.bincount(segs[:, 0], minlength=len(lens))
                assert pieces.max() <= 512, (lens, pieces.max())
                at = segs[segs[:, 0] == len(ahead)]
                assert at[0, 1] == 0 and at[-1, 2] == n and (at[1:, 1] == at[:-1, 2]).all() and len(begin) - 1 <= 152 * 16
    finally:
        gk.gk_pool_destroy(p)
