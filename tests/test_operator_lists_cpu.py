"""Lists of many tensors are checked in a time that grows with their number, not with its square.  CPU only."""
import time

import pytest
import test_operators_cpu as ops
import torch

BASE = ops.BASE


@pytest.fixture(scope="module")
def B():
    from ring_allreduce_reduction_amd import binding
    binding.lib()
    return binding


def test_one_source_listed_many_times(B):
    """One tensor copied to 2^18 places: any two inputs overlap, and that is allowed.  Pair by pair the check takes a
    minute; a second is ample for one pass."""
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: the list would be made")
    n = 1 << 18
    src, counts, dtypes = (BASE,) * n, (8,) * n, (B.arFloat32,) * n
    dst = [4 * BASE + 64 * i for i in range(n)]
    t0 = time.perf_counter()
    assert ops.lists(B, n=n, src=src, dst=dst, counts=counts, dtypes=dtypes) == B.arHipError   # nothing refused but the GPU
    dst[-1] = BASE   # the last over the shared source
    assert ops.lists(B, n=n, src=src, dst=dst, counts=counts, dtypes=dtypes) == B.arInvalidArgument
    assert time.perf_counter() - t0 < 10


def test_one_tensor_in_place_of_a_list(B):
    """It would be cut into its rows, or its elements.  A CPU tensor stands in: the check comes before the device's."""
    x = torch.zeros(4, 8)
    for args in ((x,), (x[0],), (x, [x]), ([x], x), (x, x)):
        with pytest.raises(ValueError, match="got one tensor"):
            B.TensorList(*args)
    for ts in ([x], (x,), iter([x])):   # any other iterable is read once
        with pytest.raises(ValueError, match="device tensors"):
            B.TensorList(ts)
