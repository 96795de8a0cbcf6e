"""Conversion of ctypes arguments on the host (no GPU)."""
import timeit

import pytest

gk = pytest.importorskip("paged_kv_cache_pool_gb300.binding")


class Tensor:
    def data_ptr(self):
        return 4096


class Stream:
    cuda_stream = 64


class Address(int):
    def __getattr__(self, name):
        raise AssertionError(f"{name} looked up on an address")


@pytest.mark.parametrize("convert,thing,value", [(gk._ptr, Tensor(), 4096), (gk._stream, Stream(), 64)])
def test_tensors_addresses_and_none(convert, thing, value):
    assert convert(thing) == value and convert(None) is None
    assert convert(0) == 0 and convert(Address(8192)) == 8192
    with pytest.raises(AttributeError):
        convert(object())


@pytest.mark.parametrize("convert,thing", [(gk._ptr, Tensor()), (gk._stream, Stream())])
@pytest.mark.parametrize("plain", [None, 4096])
def test_none_and_addresses_cost_no_more_than_tensors(convert, thing, plain):
    """The default stream and absent arrays are in every call; half as much again is left for noise."""
    cost = [min(timeit.repeat(lambda x=x: convert(x), number=20000, repeat=9)) for x in (plain, thing)]
    assert cost[0] <= 1.5 * cost[1], cost
