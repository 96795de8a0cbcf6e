"""gk_qk_norm_rope, gk_append_qkv and gk_read_kv against 64-bit forms: every geometry,
rotations of the whole head, of a part and of neighbouring pairs, strides, in place, both
kinds of cache, copy-on-write, bad slots and positions, special values, graphs and streams."""
import numpy as np
import pytest

from kv4_ref import bf16_bits, bf16_value, check_rotated, encode, fields, rotated

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from paged_kv_cache_pool_gb300 import binding as gk  # noqa: E402
from paged_kv_cache_pool_gb300.engine import Engine  # noqa: E402

GEOMETRIES = [(d, g, hkv) for d, gs in ((64, (1, 2, 4)), (128, (1, 2, 4, 5, 8))) for g, hkv in zip(gs, (3, 8, 1, 5, 2))]
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_pool_gb300 import build
    build.build()


def np64(x):
    return x.double().cpu().numpy()


class Rows:
    """q, k, v of n tokens, views of one projection's output or tensors of their own."""

    def __init__(self, n, hq, hkv, d, seed=0, fused=True, far=5000):
        g = torch.Generator(device="cuda").manual_seed(seed)
        parts = (hq, hkv, hkv)
        if fused:
            row = torch.randn(n, sum(parts) * d + 8, generator=g, device="cuda").to(BF)
            ends = np.cumsum([0, *parts]) * d
            self.q, self.k, self.v = (row[:, a:b].unflatten(1, (-1, d)) for a, b in zip(ends, ends[1:]))
        else:
            self.q, self.k, self.v = (torch.randn(n, p, d, generator=g, device="cuda").to(BF) for p in parts)
        self.pos = torch.randint(0, far, (n,), generator=g, device="cuda", dtype=torch.int32)
        self.weights = [(1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(BF) for _ in range(2)]


@pytest.mark.parametrize("d,g,hkv", GEOMETRIES)
@pytest.mark.parametrize("rot,inter,norm", [(None, False, True), (None, True, False), (16, False, True), (48, True, True), (32, False, False),
                                            (48, False, False), (0, False, True), (0, False, False)])
def test_norm_and_rotation(d, g, hkv, rot, inter, norm):
    rot = d if rot is None else rot
    eng = Engine(1, g * hkv, hkv, d, 64, 64, 1)
    for n, fused in ((1, True), (37, True), (150, False)):
        x = Rows(n, g * hkv, hkv, d, n, fused)
        table = eng.rope_table(5000, rot) if rot else None
        wq, wk = x.weights if norm else (None, None)
        rope = eng.rope(table, inter, wq, wk, 1e-5)
        q_out, k_out = (torch.full((n + 1, h, d), 9.0, dtype=BF, device="cuda") for h in (g * hkv, hkv))
        eng.qk_norm_rope(rope, x.pos, x.q, x.k, q_out[:n], k_out[:n])
        host = None if table is None else table.cpu().numpy()
        for got, src, w, what in ((q_out, x.q, wq, "q"), (k_out, x.k, wk, "k")):
            want = rotated(np64(src), x.pos.cpu().numpy(), host, rot, inter, None if w is None else np64(w), 1e-5)
            check_rotated(np64(got[:n]), want, what)
            assert (got[n:] == 9).all()
        # in place, keys alone, queries alone: the same bits
        q, k = x.q.clone(), x.k.clone()
        eng.qk_norm_rope(rope, x.pos, q, None)
        eng.qk_norm_rope(rope, x.pos, None, k)
        assert torch.equal(q, q_out[:n]) and torch.equal(k, k_out[:n])
        eng.qk_norm_rope(rope, x.pos, x.q, x.k)
        assert torch.equal(x.q, q_out[:n]) and torch.equal(x.k, k_out[:n])
    assert eng.device_error() == gk.GK_OK
    eng.close()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("part", [1, 2, 4])
@pytest.mark.parametrize("inter", [False, True])
def test_rotation_rounds_like_elementary_operations(d, part, inter):
    """Without a norm: fp32 products and sums, each rounded by itself, then bf16, bit for bit (of 4 million values a contracted sum
    would move about 80)."""
    n, rot = 4000, d // part
    eng = Engine(1, 8, 2, d, 64, 64, 1)
    x = Rows(n, 8, 2, d, 6)
    table = eng.rope_table(5000, rot)
    q, k = torch.empty(n, 8, d, dtype=BF, device="cuda"), torch.empty(n, 2, d, dtype=BF, device="cuda")
    eng.qk_norm_rope(eng.rope(table, inter), x.pos, x.q, x.k, q, k)
    c, s = (t[:, None] for t in table[x.pos.long()].split(rot // 2, 1))
    for got, x in ((q, x.q), (k, x.k)):
        want = x.float()
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
        ya, yb = want[..., a] * c - want[..., b] * s, want[..., b] * c + want[..., a] * s
        want[..., a], want[..., b] = ya, yb
        assert torch.equal(got, want.to(BF))
    eng.close()


def test_far_positions_and_growth():
    """A rotation keeps each pair's length, and turns by the table's angle at the last position of a long table."""
    d, far = 128, 1 << 20
    eng = Engine(1, 4, 4, d, 64, 64, 1)
    table = eng.rope_table(far, base=500000.0)
    x = Rows(3, 4, 4, d, 1, False)
    x.pos.copy_(torch.tensor([far - 1, 0, 524287]))
    q, k = torch.empty_like(x.q), torch.empty_like(x.k)
    eng.qk_norm_rope(eng.rope(table), x.pos, x.q, x.k, q, k)
    turn = np.arange(64)[None] * 0 + 500000.0 ** (-2 * np.arange(64) / 128)
    angle = x.pos.cpu().numpy().astype(np.float64)[:, None] * turn
    a, b = np64(x.q)[..., :64], np64(x.q)[..., 64:]
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    want = np.concatenate([a * c - b * s, b * c + a * s], -1)
    size = np.concatenate([np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)], -1)
    # the angle itself in 64 bits: up to 2^20 with 2^-52, below 2^-31; the table's rounding adds 2^-24 of each term
    assert (np.abs(np64(q) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * size).all()
    assert torch.equal(q[1], x.q[1])
    eng.close()


def place(eng, lens):
    """Slots of packed tokens of new sequences, and the sequences."""
    seqs = [eng.seq_create() for _ in lens]
    slots, cow = eng.append_slots(np.repeat(np.asarray(seqs, np.int32), lens))
    assert len(cow) == 0
    return eng.to_device(slots), seqs


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("d,g,hkv", GEOMETRIES)
@pytest.mark.parametrize("page", [1, 3, 16])
def test_append(d, g, hkv, page, bits):
    """The cache holds what gk_append_kv stores of the normed and rotated rows, every other byte stays."""
    eng = Engine(2, g * hkv, hkv, d, 64, 99 * page, page, seed=5, kv_bits=bits)
    store = [eng.cold] if bits == 4 else [eng.cold_k, eng.cold_v]
    x = Rows(61, g * hkv, hkv, d, 3)
    rope = eng.rope(eng.rope_table(5000), False, *x.weights)
    slots, _ = place(eng, [1, 0, 33, 27])
    q, k = torch.empty(61, g * hkv, d, dtype=BF, device="cuda"), torch.empty(61, hkv, d, dtype=BF, device="cuda")
    eng.qk_norm_rope(rope, x.pos, x.q, x.k, q, k)
    for s in store:
        s.view(torch.uint8).fill_(0x5A)
    eng.append_kv(1, slots, k, x.v.contiguous())
    want = [s.clone() for s in store]
    for s in store:
        s.view(torch.uint8).fill_(0x5A)
    q2, k2 = torch.empty_like(q), torch.empty_like(k)
    eng.append_qkv(1, rope, x.pos, slots, x.q, x.k, x.v, q2, k2)
    assert torch.equal(q, q2) and torch.equal(k, k2)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(store, want))
    # without k_out and without queries
    for s in store:
        s.view(torch.uint8).fill_(0x5A)
    eng.append_qkv(1, rope, x.pos, slots, None, x.k, x.v)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(store, want))
    if bits == 16:
        assert torch.equal(eng.cold_k[1, slots], k) and torch.equal(eng.cold_v[1, slots], x.v)
    assert (store[0][0].view(torch.uint8) == 0x5A).all()
    rk, rv = eng.read_kv(1, slots)
    if bits == 16:
        assert torch.equal(rk, k) and torch.equal(rv, x.v)
    else:
        check_codes(eng.cold[1, slots].cpu().numpy(), k, x.v, rk, rv)
    assert eng.device_error() == gk.GK_OK
    eng.close()


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("d,rot", [(64, 16), (64, 32), (64, 48), (128, 16), (128, 48), (128, 64), (128, 80), (128, 112)])
def test_append_of_heads_that_rotate_in_part(d, rot, bits):
    """What the cache holds, and a group of NaN in it, is what gk_append_kv stores of rows that were rotated before."""
    eng = Engine(1, 8, 4, d, 64, 512, 1, kv_bits=bits)
    x = Rows(300, 8, 4, d, 8)
    x.v[7, 1, d - 1] = float("nan")
    x.v[9, 2, 0] = float("inf")
    rope = eng.rope(eng.rope_table(5000, rot), False, *x.weights)
    slots = torch.randperm(512, device="cuda")[:300]
    q, k, q2, k2 = (torch.empty(300, h, d, dtype=BF, device="cuda") for h in (8, 4, 8, 4))
    eng.qk_norm_rope(rope, x.pos, x.q, x.k, q, k)
    store = [eng.cold] if bits == 4 else [eng.cold_k, eng.cold_v]
    for s in store:
        s.view(torch.uint8).fill_(0x5A)
    eng.append_kv(0, slots, k, x.v.contiguous())
    want = [s.clone() for s in store]
    for s in store:
        s.view(torch.uint8).fill_(0x5A)
    eng.append_qkv(0, rope, x.pos, slots, x.q, x.k, x.v, q2, k2)
    assert torch.equal(q, q2) and torch.equal(k, k2)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(store, want))
    eng.close()


def check_codes(rows, k, v, rk, rv):
    """Rows hold the documented codes of k and v in the documented places, and read back as what they stand for."""
    n, hkv, d = k.shape
    codes, lo, span = fields(rows, hkv, d)
    for part, (x, r) in enumerate(((k, rk), (v, rv))):
        want, wlo, wspan, border = encode(np64(x))
        assert (bf16_value(lo[:, :, part]) == wlo).all() and (bf16_value(span[:, :, part]) == wspan).all()
        # 15 (x - lo) / span in fp32: three roundings of 2^-24 on at most 15, below 2^-18
        off = codes[:, :, part] != want
        assert (np.abs(codes[:, :, part] - want)[off] == 1).all() and (border[off] < 2.0 ** -18).all()
        step = bf16_value(span[:, :, part]) / np.float32(15)
        val = np.repeat(bf16_value(lo[:, :, part]), 64, -1) + codes[:, :, part].astype(np.float32) * np.repeat(step, 64, -1)
        assert (bf16_bits(val) == bf16_bits(r.float().cpu().numpy())).all()
    # the padding of a row is not written
    used = hkv * d + hkv * d // 8
    assert (rows[:, used:] == 0x5A).all()


def test_values_at_the_border_of_codes():
    """Ties go to even, ends to codes 0 and 15, constant groups come back as they were, tiny spans as their least value."""
    eng = Engine(1, 2, 2, 64, 64, 64, 1, kv_bits=4)
    v = torch.zeros(6, 2, 64, device="cuda")
    v[0, 0] = torch.arange(64, device="cuda") % 31 * 0.5          # span 15: x = code + 0 or 0.5
    v[0, 1] = -v[0, 0]
    v[1] = 3.140625
    v[2] = -0.0
    v[3, 0, 0], v[3, 1] = 2.0 ** -101, 2.0 ** -99
    v[3, 1, 5] = 2.0 ** -98
    v[4, 0, 7], v[4, 1, 63] = 2.0 ** 119, -2.0 ** 119             # span 2^119
    v[5, :, 1], v[5, :, 2] = 2.0 ** -60, 1.0
    v = v.to(BF)
    slots = torch.arange(6, device="cuda")
    eng.append_kv(0, slots, v, v)
    k2, v2 = eng.read_kv(0, slots)
    assert torch.equal(k2, v2)
    codes = fields(eng.cold[0, :6].cpu().numpy(), 2, 64)[0]
    x = np.arange(64) % 31 * 0.5
    assert (codes[0, 0, 0] == np.rint(x)).all() and (codes[0, 1, 1] == np.rint(15 - x)).all()
    assert torch.equal(v2[1], v[1]) and (v2[2] == 0).all() and (v2[3, 0] == 0).all()
    assert v2[3, 1, 5] == 2.0 ** -98 and v2[3, 1, 6] == 2.0 ** -99
    assert v2[4, 0, 7] == 2.0 ** 119 and (v2[4, 0, :7] == 0).all() and v2[4, 1, 63] == -2.0 ** 119 and (v2[4, 1, :63] == 0).all()
    assert v2[5, 0, 2] == 1 and (v2[5, 0, :2] == 0).all()
    eng.close()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 2.0 ** 127])
def test_groups_that_hold_no_number(d, bad):
    """An infinity, a NaN or a span past 2^120 makes its group of 64 read as NaN, and no other."""
    eng = Engine(1, 2, 2, d, 64, 64, 1, kv_bits=4)
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randn(5, 2, d, generator=g, device="cuda").to(BF)
    v = torch.randn(5, 2, d, generator=g, device="cuda").to(BF)
    slots = torch.arange(5, device="cuda")
    eng.append_kv(0, slots, k, v)
    k0, v0 = eng.read_kv(0, slots)
    k[1, 1, d - 1] = bad
    v[3, 0, 5] = bad
    eng.append_kv(0, slots, k, v)
    k1, v1 = eng.read_kv(0, slots)
    nan_k, nan_v = torch.zeros_like(k, dtype=torch.bool), torch.zeros_like(k, dtype=torch.bool)
    nan_k[1, 1, d - 64:] = True
    nan_v[3, 0, :64] = True
    assert torch.equal(k1.isnan(), nan_k) and torch.equal(v1.isnan(), nan_v)
    assert torch.equal(k1[~nan_k], k0[~nan_k]) and torch.equal(v1[~nan_v], v0[~nan_v])
    eng.close()


@pytest.mark.parametrize("bits", [16, 4])
def test_slots_and_positions_outside(bits):
    """A token with a bad slot keeps its rotated rows; one with a bad position leaves everything as it was; both are reported."""
    eng = Engine(1, 8, 2, 64, 64, 64, 1, kv_bits=bits)
    store = eng.cold if bits == 4 else eng.cold_k
    x = Rows(9, 8, 2, 64, 2, far=100)
    rope = eng.rope(eng.rope_table(100))
    slots = torch.arange(9, device="cuda") + 10
    q, k = (torch.full((9, h, 64), 9.0, dtype=BF, device="cuda") for h in (8, 2))
    q0, k0 = torch.empty_like(q), torch.empty_like(k)
    eng.qk_norm_rope(rope, x.pos, x.q, x.k, q0, k0)
    for bad in (-1, 64, 1 << 40, -(1 << 40)):
        s = slots.clone()
        s[4] = bad
        store.view(torch.uint8).fill_(0x5A)
        eng.append_qkv(0, rope, x.pos, s, x.q, x.k, x.v, q, k)
        assert eng.device_error() == gk.GK_ERR_DEVICE_BOUNDS and eng.device_error() == gk.GK_OK
        assert torch.equal(q, q0) and torch.equal(k, k0)
        changed = (store.view(torch.uint8) != 0x5A).flatten(2).any(2)[0].nonzero().flatten().tolist()
        assert changed == [10, 11, 12, 13, 15, 16, 17, 18]
        rk, rv = eng.read_kv(0, s)
        assert eng.device_error() == gk.GK_ERR_DEVICE_BOUNDS
        assert (rk[4] == 0).all() and (rv[4] == 0).all() and (rv[5] != 0).any()
    for bad in (-1, 100, -(1 << 31), (1 << 31) - 1):
        pos = x.pos.clone()
        pos[7] = bad
        store.view(torch.uint8).fill_(0x5A)
        q.fill_(9)
        k.fill_(9)
        eng.append_qkv(0, rope, pos, slots, x.q, x.k, x.v, q, k)
        assert eng.device_error() == gk.GK_ERR_DEVICE_BOUNDS
        assert (q[7] == 9).all() and (k[7] == 9).all() and torch.equal(q[:7], q0[:7]) and torch.equal(k[8], k0[8])
        assert (store[0, 17].view(torch.uint8) == 0x5A).all() and (store[0, 18].view(torch.uint8) != 0x5A).any()
        q.fill_(9)
        eng.qk_norm_rope(rope, pos, x.q, x.k, q, k)
        assert eng.device_error() == gk.GK_ERR_DEVICE_BOUNDS and (q[7] == 9).all()
    eng.close()


@pytest.mark.parametrize("bits", [16, 4])
def test_copy_on_write_before_the_append(bits):
    """A forked sequence's partial block is copied, then both write behind it; a bad pair is reported and copies nothing."""
    eng = Engine(2, 8, 2, 64, 64, 16 * 8, 8, kv_bits=bits)
    x = Rows(13, 8, 2, 64, 2)
    rope = eng.rope(eng.rope_table(5000))
    slots, (a,) = place(eng, [11])
    eng.append_qkv(1, rope, x.pos[:11], slots, None, x.k[:11], x.v[:11])
    b = eng.seq_fork(a)
    new, cow = eng.append_slots([a, b])
    assert len(cow) == 1
    eng.append_qkv(1, rope, x.pos[11:], eng.to_device(new), None, x.k[11:], x.v[11:], d_cow=eng.to_device(cow.reshape(-1)))
    k, _ = torch.empty_like(x.k), None
    eng.qk_norm_rope(rope, x.pos, None, x.k, None, k)
    for seq, last in ((a, 11), (b, 12)):
        table = eng.block_tables([seq])[0]
        at = torch.tensor([int(table[t // 8]) * 8 + t % 8 for t in range(12)], device="cuda")
        rk, rv = eng.read_kv(1, at)
        want_k, want_v = (torch.cat([y[:11], y[last:last + 1]]) for y in (k, x.v))
        if bits == 16:
            assert torch.equal(rk, want_k) and torch.equal(rv, want_v)
        else:
            direct = Engine(1, 8, 2, 64, 64, 64, 1, kv_bits=4)
            order = torch.arange(12, device="cuda")
            direct.append_kv(0, order, want_k, want_v.contiguous())
            dk, dv = direct.read_kv(0, order)
            assert torch.equal(rk, dk) and torch.equal(rv, dv)
            direct.close()
    assert eng.device_error() == gk.GK_OK
    store = eng.cold if bits == 4 else eng.cold_k
    before = store.clone()
    for pair in ([-1, 0], [0, 16], [1 << 30, 1]):
        eng.append_qkv(1, rope, x.pos[:0], eng.to_device(np.zeros(0, np.int64)), None, x.k[:0], x.v[:0],
                       d_cow=eng.to_device(np.asarray(pair, np.int32)))
        assert eng.device_error() == gk.GK_ERR_DEVICE_BOUNDS and torch.equal(store.view(torch.uint8), before.view(torch.uint8))
    eng.close()


def test_reading_back_strides_repeats_and_counts():
    for bits in (16, 4):
        eng = Engine(2, 10, 5, 128, 64, 256, 1, kv_bits=bits)
        x = Rows(200, 10, 5, 128, 4)
        slots = torch.randperm(256, device="cuda")[:200]
        eng.append_kv(1, slots, x.k.contiguous(), x.v.contiguous())
        k, v = eng.read_kv(1, slots)
        pick = torch.tensor([3, 3, 199, 0, 3], device="cuda")
        wide = torch.full((5, 12, 128), 9.0, dtype=BF, device="cuda")
        eng.read_kv(1, slots[pick], wide[:, 1:6], wide[:, 6:11])
        assert torch.equal(wide[:, 1:6], k[pick]) and torch.equal(wide[:, 6:11], v[pick])
        assert (wide[:, 0] == 9).all() and (wide[:, 11] == 9).all()
        eng.read_kv(1, slots[:0])
        assert eng.device_error() == gk.GK_OK
        eng.close()


def test_offsets_past_32_bits():
    """The last slots of a cache of more than 2^32 bytes, second layer."""
    slots_n = 1 << 21
    for bits in (16, 4):
        eng = Engine(2, 8, 8, 128, 64, slots_n, 16, kv_bits=bits)
        x = Rows(20, 8, 8, 128, 6)
        rope = eng.rope(eng.rope_table(5000))
        slots = torch.arange(slots_n - 20, slots_n, device="cuda").flip(0)
        eng.append_qkv(1, rope, x.pos, slots, x.q, x.k, x.v, torch.empty_like(x.q))
        small = Engine(1, 8, 8, 128, 64, 64, 16, kv_bits=bits)
        at = torch.arange(20, device="cuda")
        small.append_qkv(0, rope, x.pos, at, x.q, x.k, x.v, torch.empty_like(x.q))
        for a, b in zip(eng.read_kv(1, slots), small.read_kv(0, at)):
            assert torch.equal(a, b)
        assert eng.device_error() == gk.GK_OK
        eng.close()
        small.close()
        torch.cuda.empty_cache()


def test_captured_and_on_another_stream():
    """A captured append and read replays on new inputs; calls on a side stream order with it."""
    eng = Engine(1, 32, 8, 128, 64, 512, 1, kv_bits=4)
    x, y = Rows(64, 32, 8, 128, 7), Rows(64, 32, 8, 128, 8)
    rope = eng.rope(eng.rope_table(5000), False, *x.weights)
    slots = torch.randperm(512, device="cuda")[:64]
    q, k = torch.empty_like(x.q), torch.empty_like(x.k)
    want = []
    for z in (x, y):
        eng.append_qkv(0, rope, z.pos, slots, z.q, z.k, z.v, q, k)
        want.append([t.clone() for t in (q, k, *eng.read_kv(0, slots))])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    rk, rv = torch.empty_like(k), torch.empty_like(k)
    row = torch.empty(64, 48 * 128, dtype=BF, device="cuda")
    parts = [t.unflatten(1, (-1, 128)) for t in row.split([32 * 128, 8 * 128, 8 * 128], 1)]
    pos = torch.zeros(64, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        eng.append_qkv(0, rope, pos, slots, *parts, q, k, stream=torch.cuda.current_stream())
        gk.gk_read_kv(eng.pool, torch.cuda.current_stream(), 0, slots, rk, rv)
    for z, w in ((x, want[0]), (y, want[1]), (x, want[0])):
        for a, b in zip(parts, (z.q, z.k, z.v)):
            a.copy_(b)
        pos.copy_(z.pos)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((q, k, rk, rv), w))
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        eng.append_qkv(0, rope, y.pos, slots, y.q, y.k, y.v, q, k, stream=side)
        gk.gk_read_kv(eng.pool, side, 0, slots, rk, rv)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((q, k, rk, rv), want[1]))
    assert eng.device_error() == gk.GK_OK
    eng.close()


def test_special_values_of_rows():
    """A NaN or infinity in a head stays in its head's norm and its pair's rotation."""
    eng = Engine(1, 4, 2, 64, 64, 64, 1)
    x = Rows(6, 4, 2, 64, 9, False)
    rope_plain, rope_norm = eng.rope(eng.rope_table(5000)), eng.rope(eng.rope_table(5000), False, *x.weights)
    clean = [t.clone() for t in (x.q, x.k)]
    eng.qk_norm_rope(rope_plain, x.pos, *clean)
    normed = [t.clone() for t in (x.q, x.k)]
    eng.qk_norm_rope(rope_norm, x.pos, *normed)
    x.q[2, 1, 5] = float("nan")
    q = x.q.clone()
    eng.qk_norm_rope(rope_plain, x.pos, q, None)
    bad = torch.zeros_like(q, dtype=torch.bool)
    bad[2, 1, 5] = bad[2, 1, 37] = True
    assert torch.equal(q.isnan(), bad) and torch.equal(q[~bad], clean[0][~bad])
    q = x.q.clone()
    eng.qk_norm_rope(rope_norm, x.pos, q, None)
    bad[2, 1] = True
    assert torch.equal(q.isnan(), bad) and torch.equal(q[~bad], normed[0][~bad])
    # rows of zeros have no length: eps keeps them zeros
    z = torch.zeros_like(x.q)
    eng.qk_norm_rope(rope_norm, x.pos, z, None)
    assert (z == 0).all()
    eng.close()


def busy():
    """Tens of milliseconds of work on the current stream."""
    a = torch.randn(8192, 8192, device="cuda").to(BF)
    for _ in range(40):
        a = a @ a


def stored_rows(n=20000):
    eng = Engine(1, 8, 8, 128, 64, n, 1, kv_bits=4)
    slots = torch.arange(n, device="cuda")
    k, v = (torch.randn(n, 8, 128, device="cuda").to(BF) for _ in range(2))
    eng.append_kv(0, slots, k, v)
    want = [x.clone() for x in eng.read_kv(0, slots)]
    torch.cuda.synchronize()
    return eng, slots, want


def test_rows_read_on_a_side_stream_are_of_that_stream():
    """What read_kv allocates is not memory that the current stream still uses, and what is dropped is not handed to the current
    stream while the side stream still uses it."""
    eng, slots, want = stored_rows()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        used = [torch.empty_like(x) for x in want]
        torch.cuda.synchronize()
        busy()
        for x in used:
            x.fill_(7)
        del used, x                                     # free for the current stream, whose fills are still to come
        got = eng.read_kv(0, slots, stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    copies = [torch.empty_like(x) for x in want]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        busy()
        got = eng.read_kv(0, slots, stream=side)
        for a, b in zip(copies, got):
            a.copy_(b)
    del got, a, b
    other = [torch.full_like(x, 7) for x in want]        # on the current stream, at once
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(copies, want)) and all((x == 7).all() for x in other)
    eng.close()


def test_rows_read_without_a_stream_of_their_own():
    """On the default stream while another one is current: refused unless both outputs are given; in a capture, its stream is named."""
    eng, slots, want = stored_rows(300)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        with pytest.raises(ValueError, match="stream"):
            eng.read_kv(0, slots)
        side.synchronize()
    k, v = (torch.empty_like(x) for x in want)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        eng.read_kv(0, slots, k, v)
    torch.cuda.synchronize()
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = eng.read_kv(0, slots, stream=torch.cuda.current_stream())
    for x in got:
        x.fill_(7)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    eng.close()
