"""The clipped policy loss with a KL term over every rank's tokens, and its gradient, against the formulas in 64 bits
(step_util) and against differences."""
import math

import op_util as ou
import pytest
import step_util as su
import torch

pytestmark = pytest.mark.gpu

NAN = float("nan")


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from ring_allreduce_reduction_amd import binding
    binding.lib()
    return binding


@pytest.fixture(autouse=True)
def _named(request):
    import gpu_util
    gpu_util.note(request.node.name)


def inputs(tokens, seed, spread=0.2):
    g = torch.Generator().manual_seed(seed)
    old = [-3 * torch.rand(k, generator=g) for k in tokens]
    logp = [o + spread * torch.randn(len(o), generator=g) for o in old]
    ref = [o + spread * torch.randn(len(o), generator=g) for o in old]
    adv = [torch.randn(k, generator=g) for k in tokens]
    w = [(torch.rand(k, generator=g) < 0.7).float() * (0.5 + torch.rand(k, generator=g)) for k in tokens]
    return logp, old, ref, adv, w


def run(B, data, low=0.2, high=0.28, kl=0.05, denominator=0.0, scale=1.0, ref=True, weight=True, grad=True, inplace=False,
        stream=None, workspace=None):
    logp, old, rf, adv, w = ([t.cuda() for t in ts] for ts in data)
    stats = torch.full((5,), NAN, device="cuda")
    out = None
    if grad:
        out = logp if inplace else [torch.full_like(t, NAN) for t in logp]
    torch.cuda.synchronize()
    B.arPolicyLoss(logp, old, adv, stats, rf if ref else None, w if weight else None, out, low, high, kl if ref else 0.0,
                   denominator, scale, workspace=workspace, stream=stream)
    torch.cuda.synchronize()
    return stats, out


def check(got, data, low=0.2, high=0.28, kl=0.05, denominator=0.0, scale=1.0, ref=True, weight=True):
    logp, old, rf, adv, w = data
    stats, off, grads, doff = su.policy(logp, old, rf if ref else None, adv, w if weight else None, low, high,
                                        kl if ref else 0.0, denominator, scale)
    ou.within(got[0], stats, off, torch.float32, "stats")
    if got[1] is not None:
        for r, (a, b, o) in enumerate(zip(got[1], grads, doff)):
            ou.within(a, b, o, torch.float32, "dlogp of rank %d" % r)


@pytest.mark.parametrize("tokens", [[1], [2, 0, 1], [500, 375, 250, 0], [4096], [4097], [1000] * 5, [70000, 0, 1], [300000, 17],
                                    [200] * 17, [95] * 32, [97] * 32, [90] * 33, [3000] * 40, [1] * 128, [0] * 20 + [9]], ids=lambda t: "%dx%d" % (len(t), max(t)))
def test_policy_loss(B, tokens):
    data = inputs(tokens, len(tokens))
    check(run(B, data), data)


@pytest.mark.parametrize("kw", [dict(ref=False), dict(weight=False), dict(ref=False, weight=False), dict(denominator=7.5),
                                dict(scale=1024.0), dict(low=0.0, high=0.0), dict(low=1.0, high=math.inf), dict(kl=0.0),
                                dict(scale=0.0), dict(scale=-1.0)], ids=str)
@pytest.mark.parametrize("tokens", [[300, 0, 41], [9000, 100]], ids=str)
def test_choices(B, tokens, kw):
    data = inputs(tokens, 3)
    check(run(B, data, **kw), data, **kw)


@pytest.mark.parametrize("tokens", [[300, 0, 41], [9000, 100], [300] * 18], ids=lambda t: str(len(t)))
def test_in_place_and_loss_alone(B, tokens):
    data = inputs(tokens, 4)
    want = run(B, data)
    stats, out = run(B, data, inplace=True)
    assert torch.equal(stats, want[0]) and all(torch.equal(a, b) for a, b in zip(out, want[1]))
    assert torch.equal(run(B, data, grad=False)[0], want[0])


@pytest.mark.parametrize("tokens", [[400], [9000, 5]], ids=str)
def test_on_policy(B, tokens):
    """The first step on a sample: every ratio is 1, nothing is clipped, not even with bounds of 0."""
    logp, _, _, adv, w = inputs(tokens, 5)
    data = (logp, logp, logp, adv, w)
    for kw in (dict(), dict(low=0.0, high=0.0)):
        stats, out = run(B, data, **kw)
        check((stats, out), data, **kw)
        assert stats[3] == 0 and stats[2] == 0


@pytest.mark.parametrize("tokens", [600, 20000])
def test_next_to_the_bounds(B, tokens):
    """Ratios one float step to either side of the bounds: clipped as the formula in 64 bits says."""
    up, down = math.log1p(0.28), math.log1p(-0.2)
    g = torch.Generator().manual_seed(6)
    steps = torch.randint(-3, 4, (tokens,), generator=g)
    base = torch.where(torch.rand(tokens, generator=g) < 0.5, torch.tensor(up), torch.tensor(down)).float()
    logp = (base.view(torch.int32) + steps.int()).view(torch.float32)
    data = ([logp], [torch.zeros(tokens)], [logp], [torch.randn(tokens, generator=g)], [torch.ones(tokens)])
    check(run(B, data), data)


@pytest.mark.parametrize("tokens", [600, 20000])
def test_small_differences_keep_their_kl(B, tokens):
    logp, _, _, adv, w = inputs([tokens], 7)
    ref = [logp[0] + 1e-4 * torch.randn(tokens, generator=torch.Generator().manual_seed(1))]
    data = (logp, logp, ref, [torch.zeros(tokens)], w)
    stats, out = run(B, data, kl=1.0)
    check((stats, out), data, kl=1.0)
    assert 1e-9 < stats[2].item() < 1e-8


@pytest.mark.parametrize("tokens", [[500, 20], [30000]], ids=str)
def test_tokens_without_weight_are_not_looked_at(B, tokens):
    data = inputs(tokens, 8)
    want = run(B, data)
    for ts in data[:4]:
        for t, w in zip(ts, data[4]):
            t[w == 0] = NAN
    stats, out = run(B, data)
    assert torch.equal(stats, want[0]) and all(torch.equal(a, b) for a, b in zip(out, want[1]))
    bad = tuple([t.clone() for t in ts] for ts in data)
    bad[0][0][int(bad[4][0].argmax())] = NAN
    stats, out = run(B, bad)
    assert torch.isnan(stats[0]) and torch.isnan(out[0]).sum() == 1


@pytest.mark.parametrize("tokens", [[500, 20], [30000], [0], [0] * 20, [0, 0]], ids=str)
def test_no_weight_at_all(B, tokens):
    logp, old, ref, adv, w = inputs(tokens, 9)
    data = (logp, old, ref, adv, [torch.zeros_like(t) for t in w])
    stats, out = run(B, data)
    assert (stats == 0).all() and all((t == 0).all() for t in out)


def test_extreme_ratios(B):
    """Ratios past a float's range are infinite where they count and bounds where they are clipped."""
    logp = torch.tensor([800.0, 800.0, -800.0, -800.0, 0.0])
    adv = torch.tensor([1.0, -1.0, 1.0, -1.0, 0.0])
    data = ([logp], [torch.zeros(5)], [torch.zeros(5)], [adv], [torch.ones(5)])
    stats, out = run(B, data, ref=False)
    assert stats[1].item() == math.inf
    want = torch.tensor([0.0, math.inf, 0.0, 0.0, 0.0])
    assert torch.equal(out[0].cpu().abs(), want)


def test_gradient_against_differences(B):
    tokens = [40, 7]
    data = inputs(tokens, 10)
    _, out = run(B, data)
    g = torch.Generator().manual_seed(1)
    # a power of two moves exactly the floats it is added to only where they are coarse: moved on a grid instead
    grid = [(t * 1024).round() / 1024 for t in data[0]]
    data = (grid,) + data[1:]
    _, out = run(B, data)
    h = 2.0 ** -10
    move = [torch.randint(-1, 2, (k,), generator=g).float() for k in tokens]

    def value(k):
        stats, _, _, _ = su.policy([x + k * m for x, m in zip(grid, move)], *[data[i] for i in (1, 2, 3, 4)], 0.2, 0.28, 0.05)
        return stats[0].item()

    inside = [((l.double() - o.double() - b).abs() > 2 * h) for b in (math.log(1.28), math.log(0.8)) for l, o in zip(grid, data[1])]
    inside = [inside[r] & inside[2 + r] for r in range(2)]
    move = [m * i for m, i in zip(move, inside)]
    want = sum((o.double().cpu() * m.double()).sum().item() for o, m in zip(out, move))
    got = (value(h) - value(-h)) / (2 * h)
    assert abs(got - want) <= 10 * h * h + 1e-7


def test_graph_replays(B):
    for tokens in ([500, 3], [20000, 300]):
        sets = inputs(tokens, 11)
        devs = [[t.cuda() for t in ts] for ts in sets]
        out = [torch.empty_like(t) for t in devs[0]]
        stats = torch.empty(5, device="cuda")
        ws = torch.empty(max(16, B.arPolicyLossWorkspace(tokens)), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            B.arPolicyLoss(devs[0], devs[1], devs[3], stats, devs[2], devs[4], out, 0.2, 0.28, 0.05, workspace=ws)
        for k in range(3):
            new = inputs(tokens, 20 + k)
            for ts, hs in zip(devs, new):
                for t, h in zip(ts, hs):
                    t.copy_(h)
            stats.fill_(NAN)
            ws.fill_(255)
            graph.replay()
            torch.cuda.synchronize()
            check((stats, out), new)
            eager = run(B, new)
            assert torch.equal(eager[0], stats)


def test_two_streams(B):
    tokens = [30000, 41]
    sets = []
    for i in range(2):
        data = inputs(tokens, 12 + i)
        d = [[t.cuda() for t in ts] for ts in data]
        sets.append((data, d, [torch.empty_like(t) for t in d[0]], torch.empty(5, device="cuda"), torch.cuda.Stream(),
                     torch.empty(B.arPolicyLossWorkspace(tokens), dtype=torch.uint8, device="cuda")))
    torch.cuda.synchronize()
    for _ in range(20):
        for _, d, out, stats, st, ws in sets:
            B.arPolicyLoss(d[0], d[1], d[3], stats, d[2], d[4], out, 0.2, 0.28, 0.05, workspace=ws, stream=st)
    torch.cuda.synchronize()
    for data, _, out, stats, _, _ in sets:
        check((stats, out), data)


def test_as_many_tokens_as_there_may_be(B):
    """2^31 - 1 tokens of one rank: every token alike, so that the sums are exact."""
    n = (1 << 31) - 1
    zeros, ones = torch.zeros(n, device="cuda"), torch.ones(n, device="cuda")
    out, stats = torch.full((n,), NAN, device="cuda"), torch.empty(5, device="cuda")
    for weights in (None, [ones]):
        out.fill_(NAN)
        B.arPolicyLoss([zeros], [zeros], [ones], stats, weights=weights, dlogps=[out])
        torch.cuda.synchronize()
        assert stats.tolist() == [-1.0, -1.0, 0.0, 0.0, float(torch.tensor(float(n)))]
        want = torch.tensor(-1.0 / n, dtype=torch.float64).float().item()
        assert out.min().item() == want and out.max().item() == want
