"""Whose stream the tensors belong to that Engine's calls allocate (no GPU: a torch.cuda that keeps account)."""
import contextlib
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")

from paged_kv_cache_pool_gb300 import binding as gk  # noqa: E402
from paged_kv_cache_pool_gb300.engine import Engine  # noqa: E402


class Cuda:
    """Streams by their handle; `current` is the one that allocations belong to."""

    def __init__(self, current):
        self.current = current

    def current_stream(self, device):
        return SimpleNamespace(cuda_stream=self.current)

    def default_stream(self, device):
        return SimpleNamespace(cuda_stream=0)

    def ExternalStream(self, handle, device):
        return SimpleNamespace(cuda_stream=handle)

    @contextlib.contextmanager
    def stream(self, s):
        self.current, before = s.cuda_stream, self.current
        yield
        self.current = before


@pytest.fixture
def engine(monkeypatch):
    """An engine without a pool: current stream -> (engine, streams of its allocations, calls of the library)."""
    def make(current):
        cuda, owners, calls = Cuda(current), [], []

        def empty(*size, **kw):
            owners.append(cuda.current)
            return torch.empty(*size, **{**kw, "device": "cpu"})
        for name in ("gk_read_kv", "gk_tables_step"):
            monkeypatch.setattr(gk, name, lambda pool, stream, *a, name=name: calls.append((name, stream)))
        eng = Engine.__new__(Engine)
        eng.pool = None
        eng.__dict__.update(Hkv=2, d=64, device="cuda", _plans=[], _prompt_plans=[])
        eng.torch = SimpleNamespace(cuda=cuda, empty=empty, empty_like=lambda x: empty(x.shape, dtype=x.dtype), bfloat16=torch.bfloat16,
                                    int64=torch.int64)
        return eng, owners, calls
    return make


SIDE, OTHER = 77, 99


@pytest.mark.parametrize("current,stream,owner", [
    (0, None, 0), (0, 0, 0), (0, SIDE, SIDE), (0, SimpleNamespace(cuda_stream=SIDE), SIDE), (SIDE, SIDE, SIDE),
    (SIDE, SimpleNamespace(cuda_stream=SIDE), SIDE), (SIDE, OTHER, OTHER), (SIDE, 0, 0), (SIDE, SimpleNamespace(cuda_stream=0), 0)])
def test_rows_belong_to_the_stream_that_writes_them(engine, current, stream, owner):
    eng, owners, calls = engine(current)
    slots = torch.zeros(5, dtype=torch.int64)
    k, v = eng.read_kv(0, slots, stream=stream)
    assert owners == [owner, owner] and calls == [("gk_read_kv", stream)] and k.shape == v.shape == (5, 2, 64)
    assert eng.torch.cuda.current == current
    # what is given is taken as it is
    assert eng.read_kv(0, slots, v=v, stream=stream)[1] is v and owners == [owner] * 3
    assert eng.read_kv(0, slots, k, v, stream) == (k, v) and owners == [owner] * 3


def test_rows_of_no_stream_while_another_is_current(engine):
    """The call would run on the default stream, its results be used on the current one."""
    eng, owners, calls = engine(SIDE)
    slots = torch.zeros(5, dtype=torch.int64)
    for given in (dict(), dict(k=torch.empty(5, 2, 64)), dict(v=torch.empty(5, 2, 64))):
        with pytest.raises(ValueError, match="stream"):
            eng.read_kv(0, slots, **given)
    assert not owners and not calls
    eng.read_kv(0, slots, torch.empty(5, 2, 64), torch.empty(5, 2, 64))
    assert calls == [("gk_read_kv", None)]


@pytest.mark.parametrize("current,stream,owner", [(0, None, 0), (0, SIDE, SIDE), (SIDE, SIDE, SIDE), (SIDE, OTHER, OTHER), (SIDE, 0, 0),
                                                  (SIDE, None, 0)])
def test_slots_belong_to_the_stream_that_writes_them(engine, current, stream, owner):
    eng, owners, calls = engine(current)
    tables = SimpleNamespace(length=torch.zeros(3, dtype=torch.int32))
    slots, done = eng.tables_step(tables, None, 7, stream=stream)
    assert owners == [owner, owner] and calls == [("gk_tables_step", stream)] and eng.torch.cuda.current == current
    assert slots.shape == (7,) and slots.dtype is torch.int64 and done.shape == (3,) and done.dtype is torch.int32
