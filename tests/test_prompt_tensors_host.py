"""What PromptBatch takes as tensors (no GPU): those that the kernel would read as
something else, or past their end, are refused before any launch."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def gk():
    from paged_kv_cache_pool_gb300 import build
    build.build()
    from paged_kv_cache_pool_gb300 import binding
    return binding


class OnGpu:
    """A CPU tensor that says it is on the GPU: nothing here launches."""
    is_cuda = True

    def __init__(self, x):
        self.x = x

    def __getattr__(self, name):
        return getattr(self.x, name)

    def data_ptr(self):
        return 4096


def bf16(*shape):
    return OnGpu(torch.zeros(*shape, dtype=torch.bfloat16))


GOOD = dict(d_q=(7, 8, 128), d_k=(7, 2, 128), d_v=(7, 2, 128), d_out=(7, 8, 128))


def tensors(**change):
    t = {k: bf16(*s) for k, s in GOOD.items()}
    t["d_lse"] = OnGpu(torch.zeros(7, 8))
    t.update(change)
    return t


def test_good_tensors_and_addresses(gk):
    batch = gk.PromptBatch([3, 4], None, None, [0, 20], OnGpu(torch.zeros(2, 5, dtype=torch.int32)), 5)
    batch.set_device(**tensors())
    assert (batch.c.q_stride, batch.c.k_stride, batch.c.v_stride, batch.c.out_stride) == (1024, 256, 256, 1024)
    fused = torch.zeros(7, 12 * 128 + 16, dtype=torch.bfloat16)
    q, k, v = (OnGpu(fused[:, a:b].view(7, -1, 128)) for a, b in ((8, 1032), (1032, 1288), (1288, 1544)))
    batch.set_device(**tensors(d_q=q, d_k=k, d_v=v, d_lse=None))
    assert (batch.c.q_stride, batch.c.k_stride, batch.c.v_stride, batch.c.out_stride) == (1552, 1552, 1552, 1024)
    batch.set_device(4096, 4096, 4096, 4096, 4096, 8192, 5)
    assert batch.c.q_stride == 0 and batch.c.d_block_table == 8192
    batch.set_device(**tensors(d_k=4096, d_lse=4096))
    # a single token and none have no stride
    gk.PromptBatch([1]).set_device(*(OnGpu(bf16(1, h, 64).x.expand(1, h, 64)) for h in (4, 2, 2, 4)))
    gk.PromptBatch([0]).set_device(bf16(0, 4, 64), bf16(0, 2, 64), bf16(0, 2, 64), bf16(0, 4, 64), OnGpu(torch.zeros(0, 4)))


@pytest.mark.parametrize("which", sorted(GOOD))
def test_types_shapes_and_strides_of_rows(gk, which):
    heads, d = GOOD[which][1:]
    x = torch.zeros(7, heads, d, dtype=torch.bfloat16)
    bad = [x.to(torch.float16), x.to(torch.int16), x.view(torch.uint16), x.float(), x[:6], x.view(7, heads * d), x.transpose(1, 2),
           x[..., ::2], torch.zeros(8, heads, d, dtype=torch.bfloat16),
           x[:1].expand(7, heads, d),                                       # one token for all: stride 0
           torch.as_strided(x, (7, heads, d), (d, d, 1)),                   # tokens that overlap
           torch.zeros(7, heads + heads, d, dtype=torch.bfloat16), torch.zeros(7, heads, d // 2, dtype=torch.bfloat16)]
    batch = gk.PromptBatch([3, 4])
    for y in bad:
        with pytest.raises(ValueError):
            batch.set_device(**tensors(**{which: OnGpu(y)}))
    with pytest.raises(ValueError, match="on the GPU"):
        batch.set_device(**tensors(**{which: x}))
    assert batch.c.d_q is None and batch.c.q_stride == 0                    # the batch is as it was


def test_lse(gk):
    batch = gk.PromptBatch([3, 4])
    x = torch.zeros(7, 8)
    for y in (x.to(torch.bfloat16), x.double(), x[:6], x.t().contiguous().t(), torch.zeros(7, 16)[:, :8], x[:, :1].expand(7, 8),
              torch.zeros(7, 4), x.view(56)):
        with pytest.raises(ValueError, match="lse"):
            batch.set_device(**tensors(d_lse=OnGpu(y)))
    with pytest.raises(ValueError, match="on the GPU"):
        batch.set_device(**tensors(d_lse=x))


def test_block_table(gk):
    ints = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    for y in (ints(2, 5).long(), ints(2, 5).float(), ints(2, 4), ints(1, 5), ints(5, 2).t(), ints(2, 10)[:, :5]):
        with pytest.raises(ValueError, match="table"):
            gk.PromptBatch([3, 4], None, None, [0, 20], OnGpu(y), 5)
        with pytest.raises(ValueError, match="table"):
            gk.PromptBatch([3, 4]).set_device(**tensors(), d_block_table=OnGpu(y), max_blocks=5)
    # more rows than requests, and the first columns of a table whose rows are as far apart as said
    for y, width in ((ints(9, 5), 5), (ints(4, 64)[:, :3], 64), (ints(1, 64)[:, :3], 64)):
        gk.PromptBatch([3, 4][:len(y)], None, None, None, OnGpu(y), width)
    with pytest.raises(ValueError, match="table"):
        gk.PromptBatch([3, 4], None, None, None, OnGpu(ints(4, 64)[:, :3]), 3)
    batch = gk.PromptBatch([3, 4], None, None, [0, 20], OnGpu(ints(2, 5)), 5)
    with pytest.raises(ValueError, match="table"):
        batch.set_device(**tensors(), max_blocks=6)                         # wider rows than the table has
    assert batch.c.max_blocks == 5


def test_heads_of_the_pool_and_tokens_of_the_plan(gk):
    pools = [gk.gk_pool_create(1, hq, hkv, d, 0, 160, 16) for hq, hkv, d in ((8, 2, 128), (16, 2, 128), (8, 4, 128), (8, 2, 64))]
    try:
        batch, longer = gk.PromptBatch([3, 4]).set_device(**tensors()), gk.PromptBatch([3, 5])
        for pool in pools:
            plan = gk.gk_prompt_plan_build(pool, batch)
            if pool == pools[0]:
                with pytest.raises(gk.GkError, match="no device tables"):   # every check passed
                    gk.gk_prompt_attn(pool, None, 0, batch, plan)
                gk.gk_prompt_plan_update(pool, plan, longer)
                with pytest.raises(ValueError, match="tokens"):
                    gk.gk_prompt_attn(pool, None, 0, batch, plan)
                batch.set_device(4096, 4096, 4096, 4096)
                with pytest.raises(ValueError, match="tokens"):
                    gk.gk_prompt_attn(pool, None, 0, batch, plan)
                batch.set_device(**tensors())
            else:
                with pytest.raises(ValueError, match="heads"):
                    gk.gk_prompt_attn(pool, None, 0, batch, plan)
            gk.gk_prompt_plan_destroy(plan)
    finally:
        for pool in pools:
            gk.gk_pool_destroy(pool)
