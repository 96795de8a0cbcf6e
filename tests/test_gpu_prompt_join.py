"""gk_prompt_attn where partial states are joined, at the edges of how their rows lie:
ragged last blocks, Q tiles that a block does not fill, several stacked runs, pieces of
the requests' own keys beside pieces of the prefix."""
import pytest

from test_gpu_prompt import Prompts

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_pool_gb300 import build
    build.build()


def _run(*a, **k):
    p = Prompts(*a, **k)
    try:
        p.run().verify(str((a, k)))
        return p.info()
    finally:
        p.close()


@pytest.mark.parametrize("d,g", [(64, 1), (64, 2), (128, 1), (128, 4), (128, 5), (128, 8)])
def test_stacked_runs_with_ragged_blocks(d, g):
    """The run's tokens end inside a block of 2 * floor(128 / g), and requests lie across its borders."""
    block = 2 * (128 // g)
    new = [block // 3 + 1, 1, 0, block // 2, 2, block // 4 + 3] + [1] * 5
    info = _run(d, g, 2, new * 2, prefixes=[9000, 6000], which=[0] * 11 + [1] * 11, cold=[0, 130, 0, 5, 700, 0] + [3] * 5 + [0] * 11)
    assert info["stacked_requests"] > 0


@pytest.mark.parametrize("d,g", [(64, 4), (128, 2), (128, 5), (128, 8)])
def test_own_keys_in_pieces(d, g):
    block = 2 * (128 // g)
    for new in ([block + 1], [1, block - 1, block // 2 + 1], [3]):
        info = _run(d, g, 1, new, cold=[7000] + [0] * (len(new) - 1))
        assert info["max_pieces"] > 1


def test_pieces_of_both():
    """Each row's states: pieces of its own 6000 COLD tokens and of the stacked prefix."""
    info = _run(128, 4, 1, [2, 3, 1], prefixes=[20000], which=[0, 0, 0], cold=[6000, 0, 5000])
    assert info["stacked_requests"] == 3 and info["max_pieces"] > 4 and info["partials"] > 16


def test_a_plan_that_grows_and_shrinks():
    """Its partial states move and its buffers are kept: every step of it is right."""
    steps = [([3], [5000]), ([2] * 40, [2000] * 40), ([300], [0]), ([1], [9000]), ([7] * 9, [3000] * 9)]
    ps = [Prompts(128, 4, 2, new, cold=cold) for new, cold in steps]
    from paged_kv_cache_pool_gb300 import binding as gk
    for p in ps:                                   # a plan belongs to a pool: each is replanned on its own
        p.run().verify("first")
        small = gk.PromptBatch([1])
        for batch in (small, p.batch, small, p.batch):
            gk.gk_prompt_plan_update(p.pool, p.plan, batch)
        p.out.fill_(0)
        p.run().verify("again")
        p.close()
