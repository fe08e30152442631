"""Arguments of the policy loss that its 32 and 64 bits do not hold are refused, without a GPU."""
import pytest
from test_step_operators_cpu import B, policy  # noqa: F401  (a fixture, a call)


@pytest.mark.parametrize("denominator", [5e-324, 1e-310, 2.0 ** -1022 - 2.0 ** -1074])
def test_a_denominator_whose_inverse_is_infinite(B, denominator):  # noqa: F811
    assert policy(B, den=denominator) == B.arInvalidArgument


@pytest.mark.parametrize("coefficient", [3.5e38, 1e39, 1e300])
def test_a_coefficient_past_32_bits(B, coefficient):  # noqa: F811
    assert policy(B, kl=coefficient) == B.arInvalidArgument
