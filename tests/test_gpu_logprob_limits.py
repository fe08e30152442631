"""The gradient of token log-probabilities where the scale times dlogp is past or below what 32 bits hold."""
import math

import pytest
import test_gpu_logprob as lp
import torch
from test_gpu_logprob import B, _named  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("widths", [[50, 25], [1000, 24], [9000, 0, 193]], ids=str)
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=str)
def test_a_scale_times_dlogp_past_32_bits(B, dt, widths, inplace):  # noqa: F811
    """What its factor makes 0 stays 0, what it makes small enough is finite."""
    n, scale = sum(widths), 2.0 ** 127
    whole = torch.randn(6, n, generator=torch.Generator().manual_seed(n)).to(dt)
    whole[0], whole[1] = 1.5, -3e38            # equally likely
    best = 7
    whole[2:, best] = 30.0                     # certain
    t = torch.tensor([3, n - 1, best, 4, n - 1, -1])
    d = torch.tensor([10.0, -(2.0 ** 127), 10.0, 10.0, -3e38, 10.0])
    xs = [v.contiguous() for v in whole.split(widths, 1)]
    logp, top, log_sum = lp.run_forward(B, xs, t, scale)
    out = torch.cat([o.double().cpu() for o in lp.run_backward(B, d, xs, t, top.cpu(), log_sum.cpu(), scale, inplace=inplace)], 1)
    others = torch.arange(n) != t[0]
    want = -10.0 * scale / n
    # 1 / n: its logarithm's rounding, factor and difference 3 U of ln n, the exponential 2 U; the products; to dt
    bound = abs(want) * ((3 * math.log(n) + 6) * 2.0 ** -24 + 1.01 * torch.finfo(dt).eps / 2)
    assert out[0, t[0]] == math.inf and ((out[0, others] - want).abs() <= bound).all()
    others = torch.arange(n) != t[1]
    assert out[1, t[1]] == -math.inf and (out[1, others] == math.inf).all()
    assert (out[2] == 0).all() and (out[5] == 0).all()
    for i, sign in ((3, 1.0), (4, -1.0)):
        assert out[i, t[i]] == sign * math.inf and out[i, best] == -sign * math.inf
        rest = out[i].clone()
        rest[t[i]] = rest[best] = 0.0
        assert (rest == 0).all()


@pytest.mark.parametrize("widths", [[50, 25], [9000, 0, 193]], ids=str)
def test_a_scale_times_dlogp_below_32_bits(B, widths):  # noqa: F811
    """Rounds to 0; but a row without a distribution and a target past the vocabulary still give NaN, and rows whose
    dlogp is 0 zeros."""
    n, scale = sum(widths), 2.0 ** -100
    whole = torch.randn(6, n, generator=torch.Generator().manual_seed(n))
    whole[1, 20] = whole[4, 20] = math.nan
    t = torch.tensor([3, 4, n, -1, 4, n])
    d = torch.tensor([1e-20, 1e-20, -1e-20, 1e-20, 0.0, 0.0])
    xs = [v.contiguous() for v in whole.split(widths, 1)]
    logp, top, log_sum = lp.run_forward(B, xs, t, scale)
    out = torch.cat([o.cpu() for o in lp.run_backward(B, d, xs, t, top.cpu(), log_sum.cpu(), scale)], 1)
    assert torch.isnan(out[1:3]).all() and (out[[0, 3, 4, 5]] == 0).all()
