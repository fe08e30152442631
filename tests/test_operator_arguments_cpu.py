"""Arguments of the operators at the ends of their documented ranges, without a GPU."""
import pytest
import test_operators_cpu as ops


@pytest.fixture(scope="module")
def B():
    from ring_allreduce_reduction_amd import binding
    binding.lib()
    return binding


def test_every_finite_eps_is_taken(B):
    """The largest float too.  Without rows nothing is launched."""
    for eps in (0.0, 2.0 ** -149, 3.4e38, (2.0 - 2.0 ** -23) * 2.0 ** 127):
        assert ops.forward(B, eps=eps, rows=ops.N(0)) == B.arSuccess
    for eps in (float("inf"), float("-inf"), float("nan"), -2.0 ** -149):
        assert ops.forward(B, eps=eps, rows=ops.N(0)) == B.arInvalidArgument
