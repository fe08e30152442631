"""The policy loss where a number is past what 32 bits hold and at the ends of its arguments' ranges: in one
workgroup, in two passes, and with the denominator known beforehand."""
import math

import pytest
import test_gpu_policy as pol
import torch
from test_gpu_policy import B, _named  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu

FORMS = [([600, 8], {}), ([9000, 100], {}), ([9000, 100], dict(denominator=64.0)), ([40, 2] * 9, {}), ([700] * 18, {})]
forms = pytest.mark.parametrize("tokens,kw", FORMS, ids=["few", "two passes", "known", "few of 18 ranks", "18 ranks"])


def inputs(tokens, seed):
    """Tokens 0 to 7 of the first rank have a weight."""
    data = pol.inputs(tokens, seed)
    data[4][0][:8] = 1.0
    return data


def same(a, b):
    return torch.equal(a[0], b[0]) and all(torch.equal(x, y) for x, y in zip(a[1], b[1]))


@forms
def test_a_kl_of_coefficient_0_is_only_reported(B, tokens, kw):  # noqa: F811
    """However large it is: the loss and the gradient are those without a reference."""
    data = inputs(tokens, 1)
    logp, old, ref, adv, w = data
    ref[0][0], ref[0][1], ref[0][2] = logp[0][0] + 200.0, logp[0][1] + 88.8, 3e38
    want = pol.run(B, data, ref=False, **kw)
    stats, out = pol.run(B, data, kl=0.0, **kw)
    assert stats[2].item() == math.inf
    assert torch.equal(stats[[0, 1, 3, 4]], want[0][[0, 1, 3, 4]]) and all(torch.equal(a, b) for a, b in zip(out, want[1]))
    pol.check(want, data, ref=False, **kw)
    # with a coefficient it counts
    stats, out = pol.run(B, data, kl=0.5, **kw)
    assert stats[0].item() == math.inf and out[0][0].item() == -math.inf
    # a token that the policy's mask rules out
    logp[0][3], logp[0][4], adv[0][3], adv[0][4] = -math.inf, -math.inf, 1.0, -1.0
    want = pol.run(B, data, ref=False, **kw)
    stats, out = pol.run(B, data, kl=0.0, **kw)
    assert torch.isfinite(want[0]).all() and all(torch.isfinite(t).all() for t in out)
    assert torch.equal(stats[[0, 1, 3, 4]], want[0][[0, 1, 3, 4]]) and all(torch.equal(a, b) for a, b in zip(out, want[1]))


@forms
def test_an_advantage_of_0_takes_no_part(B, tokens, kw):  # noqa: F811
    """Whatever the ratio is; but a log-probability that is no number is not hidden."""
    data = inputs(tokens, 2)
    logp, old, ref, adv, w = data
    adv[0][:6] = torch.tensor([0.0, -0.0, 0.0, 0.0, 0.0, 0.0])
    near = [t.clone() for t in logp]
    near[0][:6] = old[0][:6]
    logp[0][:4] = old[0][:4] + torch.tensor([200.0, 800.0, 88.8, 3e38])
    want = pol.run(B, (near, old, ref, adv, w), ref=False, **kw)
    pol.check(want, (near, old, ref, adv, w), ref=False, **kw)
    assert same(pol.run(B, data, ref=False, **kw), want)
    rare = [t.clone() for t in old]
    rare[0][4] = -math.inf
    assert same(pol.run(B, (logp, rare, ref, adv, w), ref=False, **kw), want)
    logp[0][5] = math.nan
    stats, out = pol.run(B, data, ref=False, **kw)
    assert torch.isnan(stats[1]) and torch.isnan(out[0][5]) and sum(torch.isnan(t).sum().item() for t in out) == 1


@forms
def test_an_infinite_difference_has_an_infinite_kl(B, tokens, kw):  # noqa: F811
    """A token that the mask of the policy or of the reference rules out."""
    for where in (0, 2):
        data = inputs(tokens, 3)
        data[where][0][2] = -math.inf
        data[3][0][2] = 1.0
        stats, out = pol.run(B, data, kl=0.5, **kw)
        assert stats[2].item() == math.inf and stats[0].item() == math.inf and torch.isfinite(stats[[1, 3, 4]]).all()
        assert out[0][2].item() == -math.inf if where == 0 else torch.isfinite(out[0][2])
        out[0][2] = 0.0
        assert all(torch.isfinite(t).all() for t in out)
        data[0][0][2] = data[2][0][2] = -math.inf   # by both: no difference
        stats, out = pol.run(B, data, kl=0.5, **kw)
        assert torch.isnan(stats[[0, 2]]).all() and torch.isnan(out[0][2])


@forms
@pytest.mark.parametrize("power", [120, -120])
def test_the_weights_scale_does_not_matter(B, tokens, kw, power):  # noqa: F811
    """A power of two common to all weights, and to a given denominator, moves no bit, though a weight times its
    token's gradient is past what 32 bits hold."""
    data = inputs(tokens, 4)
    for t in data[3]:
        t.mul_(2.0 ** (power // 10))
    want = pol.run(B, data, **kw)
    pol.check(want, data, **kw)
    far = data[:4] + ([t * 2.0 ** power for t in data[4]],)
    if "denominator" in kw:
        kw = dict(denominator=kw["denominator"] * 2.0 ** power)
    stats, out = pol.run(B, far, **kw)
    assert torch.equal(stats[:4], want[0][:4]) and stats[4] == want[0][4] * 2.0 ** power   # in 32 bits: past them infinite
    assert all(torch.equal(a, b) for a, b in zip(out, want[1]))
    assert same((stats, out), pol.run(B, far, inplace=True, **kw))


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("tokens", [[600, 8], [9000, 100]], ids=["few", "two passes"])
def test_a_factor_past_64_bits(B, tokens, sign):  # noqa: F811
    """gradScale / D is infinite: a gradient of 0 stays 0, others are infinite; with the weights' sum for D too."""
    data = inputs(tokens, 5)
    data[3][0][0], data[0][0][1], data[3][0][1] = 0.0, data[1][0][1] + 1.0, 1.0   # no advantage; clipped
    small = data[:4] + ([t * 2.0 ** -140 for t in data[4]],)
    for d, kw in ((data, dict(denominator=2.3e-308, scale=sign * 1e10)), (small, dict(scale=sign * 1e300))):
        stats, out = pol.run(B, d, ref=False, **kw)
        assert not torch.isnan(stats).any() and out[0][0] == 0 and out[0][1] == 0
        for r, t in enumerate([v.cpu() for v in out]):
            assert not torch.isnan(t).any() and (t[d[4][r] == 0] == 0).all()
            if "denominator" in kw:
                live = t[(d[4][r] > 0) & (t != 0)]
                assert torch.isinf(live).all() and len(live) > len(t) // 3
    none = data[:4] + ([torch.zeros_like(t) for t in data[4]],)
    stats, out = pol.run(B, none, denominator=2.3e-308, scale=sign * 1e10)
    assert (stats == 0).all() and all((t == 0).all() for t in out)


@forms
def test_the_smallest_and_largest_coefficients(B, tokens, kw):  # noqa: F811
    """One below 32 bits' range still meets an exponential past it; the largest one no difference at all."""
    data = inputs(tokens, 6)
    logp, old, ref, adv, w = data
    want = pol.run(B, data, ref=False, **kw)
    ref[0][0] = logp[0][0] + 200.0
    stats, out = pol.run(B, data, kl=1e-60, **kw)
    assert stats[0].item() == math.inf and out[0][0].item() == -math.inf
    assert torch.equal(stats[1], want[0][1]) and torch.equal(out[0][1:], want[1][0][1:])
    same_ref = (logp, old, logp, adv, w)
    stats, out = pol.run(B, same_ref, kl=3.4e38, **kw)
    assert stats[2] == 0 and same((stats, out), want)
