"""Token log-probabilities from logits whose vocabulary is cut over the ranks, and their gradient, against the
formulas in 64 bits (step_util) and against differences."""
import math

import op_util as ou
import pytest
import step_util as su
import torch
from test_gpu_layernorm import dev, untouched

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.float16, torch.bfloat16]
INF, NAN = float("inf"), float("nan")
MORE = [0, 0]   # shards that calls get at their end: without columns, and of 33000 columns that are masked out
SHARDS = [[40000, 3], [12345] * 4, [1], [7], [64, 65], [1000], [3, 0, 2049, 1], [4096, 4096], [8191, 8193], [20000, 1, 9], [16000] * 8, [33] * 40]


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


def inputs(rows, shards, dt, seed, ignored=0.2, std=3.0):
    g = torch.Generator().manual_seed(seed)
    xs = [(torch.randn(rows, c, generator=g) * std + 1.0).to(dt) for c in shards]
    t = torch.randint(0, sum(shards), (rows,), generator=g)
    t[torch.rand(rows, generator=g) < ignored] = -100
    return xs, t


@pytest.fixture(params=[(0, 0), (15, 0), (33, 0), (0, 1)], ids=["rows", "ranks", "launches", "pieces"])
def form(request):
    """The forms a call can take: one launch, one of more than 16 ranks, several for more than 32, and for few rows of
    a long vocabulary pieces of them."""
    MORE[:] = request.param
    yield request.param
    MORE[:] = 0, 0


def on_device(xs, pad, offs):
    more = [torch.empty(len(xs[0]), 0, dtype=xs[0].dtype, device="cuda")] * MORE[0]
    more += [torch.full((len(xs[0]), 33000), -INF, dtype=xs[0].dtype, device="cuda") for _ in range(MORE[1])]
    return [dev(x, pad + r % 3, offs) for r, x in enumerate(xs)] + more


def run_forward(B, xs, targets, scale=1.0, pad=0, offs=0, stats=True, stream=None, workspace=None):
    rows = len(targets)
    logp = torch.full((rows,), NAN, device="cuda")
    top, log_sum = (torch.full((rows,), NAN, device="cuda") if stats else None for _ in range(2))
    d, t = on_device(xs, pad, offs), targets.cuda()
    torch.cuda.synchronize()
    B.arTokenLogprob(d, t, logp, top, log_sum, scale, workspace=workspace, stream=stream)
    torch.cuda.synchronize()
    return logp, top, log_sum


def check_forward(got, xs, targets, scale=1.0):
    logp, top, log_sum, d_logp, d_sum = su.logprob(torch.cat(xs, 1), targets, float(torch.tensor(scale)), len(xs))
    ou.within(got[0], logp, d_logp, torch.float32, "logp")
    if got[1] is not None:
        ou.within(got[1], top, torch.zeros_like(top), torch.float32, "top")
        ou.within(got[2], log_sum, d_sum, torch.float32, "logSum")


def statistics(xs, targets, scale):
    """What the forward pass writes, from 64 bits."""
    _, top, log_sum, _, _ = su.logprob(torch.cat(xs, 1), targets, float(torch.tensor(scale)), len(xs))
    return top.float(), log_sum.float()


def run_backward(B, dlogp, xs, targets, top, log_sum, scale=1.0, pad=0, offs=0, inplace=False, stream=None):
    x = on_device(xs, pad, offs)
    out = x if inplace else on_device([torch.full_like(t, NAN) for t in xs], pad + 1, offs)
    t = targets.cuda()
    torch.cuda.synchronize()
    B.arTokenLogprobBackward(dlogp.cuda(), x, t, top.cuda(), log_sum.cuda(), out, scale, stream=stream)
    torch.cuda.synchronize()
    return out


def check_backward(out, dlogp, xs, targets, top, log_sum, scale=1.0):
    want, bound = su.logprob_backward(dlogp, torch.cat(xs, 1), targets, float(torch.tensor(scale)), top, log_sum)
    widths = [x.shape[1] for x in xs]
    for r, (got, w, b) in enumerate(zip(out, want.split(widths, 1), bound.split(widths, 1))):
        if w.shape[1]:
            ou.within(got, w, b, xs[r].dtype, "dlogits of rank %d" % r)
            assert untouched(got)


def gradients(rows, seed):
    g = torch.Generator().manual_seed(seed)
    d = torch.randn(rows, generator=g)
    d[torch.rand(rows, generator=g) < 0.2] = 0.0
    return d


@pytest.mark.parametrize("scale", [1.0, 0.7, 1.25])
@pytest.mark.parametrize("dt", DTYPES, ids=str)
@pytest.mark.parametrize("shards", SHARDS, ids=str)
def test_few_rows(B, shards, dt, scale):
    rows = 9
    xs, t = inputs(rows, shards, dt, sum(shards))
    check_forward(run_forward(B, xs, t, scale), xs, t, scale)
    d, (top, log_sum) = gradients(rows, 5), statistics(xs, t, scale)
    check_backward(run_backward(B, d, xs, t, top, log_sum, scale), d, xs, t, top, log_sum, scale)


@pytest.mark.parametrize("dt", DTYPES, ids=str)
@pytest.mark.parametrize("rows,shards", [(1023, [500, 533]), (1024, [500, 533]), (1025, [3, 0, 1001]), (5000, [65]),
                                         (70001, [9]), (1100, [9] * 17), (1100, [9] * 33), (4100, [130] * 20), (200, [700] * 32),
                                         (66000, [1, 1]), (3000, [2050, 77])], ids=str)
def test_many_rows(B, rows, shards, dt):
    xs, t = inputs(rows, shards, dt, rows)
    check_forward(run_forward(B, xs, t), xs, t)
    d, (top, log_sum) = gradients(rows, 6), statistics(xs, t, 1.0)
    check_backward(run_backward(B, d, xs, t, top, log_sum), d, xs, t, top, log_sum)


@pytest.mark.parametrize("dt", DTYPES, ids=str)
@pytest.mark.parametrize("rows,shards", [(8192, [700, 790]), (4097, [1501, 1, 900, 2300, 703]), (8200, [1400])], ids=str)
def test_narrow_shards_of_very_many_rows(B, rows, shards, dt):
    """16 threads a shard, of few to all vectors they have in flight at a time."""
    xs, t = inputs(rows, shards, dt, rows)
    check_forward(run_forward(B, xs, t, offs=1), xs, t)


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("dt", DTYPES, ids=str)
@pytest.mark.parametrize("widest", [1, 95, 97, 192, 193, 447, 449, 896, 897, 959, 961, 1599, 1601, 1920, 1921, 3200, 3201])
def test_gradients_of_each_width(B, widest, dt, inplace):
    """16 to 256 threads a row, their vectors from the row's first whole line on."""
    rows, shards = 37, [widest, widest // 2, 3]
    xs, t = inputs(rows, shards, dt, widest)
    d, (top, log_sum) = gradients(rows, 11), statistics(xs, t, 1.0)
    for pad, offs in ((0, 0), (3, 1), (8, 24)):
        check_backward(run_backward(B, d, xs, t, top, log_sum, pad=pad, offs=offs, inplace=inplace), d, xs, t, top, log_sum)


@pytest.mark.parametrize("rows", [1, 1200])
@pytest.mark.parametrize("dt", DTYPES, ids=str)
def test_padded_rows_odd_addresses_in_place(B, form, rows, dt):
    xs, t = inputs(rows, [129, 40, 513], dt, 3)
    for pad, offs in ((0, 1), (3, 0), (8, 5)):
        check_forward(run_forward(B, xs, t, pad=pad, offs=offs), xs, t)
        d, (top, log_sum) = gradients(rows, 7), statistics(xs, t, 1.0)
        for inplace in (False, True):
            check_backward(run_backward(B, d, xs, t, top, log_sum, pad=pad, offs=offs, inplace=inplace), d, xs, t, top, log_sum)


@pytest.mark.parametrize("rows", [5, 1100])
def test_logp_alone_and_with_one_statistic(B, form, rows):
    xs, t = inputs(rows, [300, 20], torch.bfloat16, 4)
    check_forward(run_forward(B, xs, t, stats=False), xs, t)
    whole = run_forward(B, xs, t)
    for k in (1, 2):
        out = [torch.full((rows,), NAN, device="cuda") for _ in range(2)]
        B.arTokenLogprob(on_device(xs, 0, 0), t.cuda(), out[0], *[out[1] if i == k else None for i in (1, 2)])
        torch.cuda.synchronize()
        assert torch.equal(out[0], whole[0]) and torch.equal(out[1], whole[k])


@pytest.mark.parametrize("rows", [8, 1104])
@pytest.mark.parametrize("dt", DTYPES, ids=str)
def test_masks(B, form, rows, dt):
    """-inf and the type's lowest value as masks: beside ordinary logits, in whole shards, everywhere but the target,
    and (the lowest value) in a whole row."""
    low = torch.finfo(dt).min
    xs, t = inputs(rows, [700, 900, 30], dt, 6, ignored=0.0)
    whole = torch.cat(xs, 1)
    for i in range(rows):
        m = (-INF, low)[i % 2]
        kind = i // 2 % 4
        keep = whole[i, t[i]].clone()
        if kind == 0:
            whole[i, 1::3] = m
        elif kind == 1:
            whole[i, :700] = m
        elif kind == 2:
            whole[i] = m
        elif kind == 3:
            whole[i, 5:] = m
        if kind != 2 or m == -INF:
            whole[i, t[i]] = keep
    xs = [v.contiguous() for v in whole.split([700, 900, 30], 1)]
    check_forward(run_forward(B, xs, t), xs, t)
    d, (top, log_sum) = gradients(rows, 8), statistics(xs, t, 1.0)
    out = run_backward(B, d, xs, t, top, log_sum)
    check_backward(out, d, xs, t, top, log_sum)
    got = torch.cat([o.cpu() for o in out[:3]], 1)
    masked = whole == -INF
    assert (got[masked] == 0).all()


@pytest.mark.parametrize("rows", [4, 1100])
def test_masked_target(B, form, rows):
    """logp is -inf; the gradient is that of the others."""
    xs, t = inputs(rows, [100, 60], torch.float32, 9, ignored=0.0)
    whole = torch.cat(xs, 1)
    whole[torch.arange(rows), t] = -INF
    xs = [v.contiguous() for v in whole.split([100, 60], 1)]
    logp, top, log_sum = run_forward(B, xs, t)
    assert (logp == -INF).all()
    want = torch.logsumexp(whole.double(), 1)
    assert ((top.double() + log_sum.double()).cpu() - want).abs().max() < 1e-5
    d, (top, log_sum) = gradients(rows, 10), statistics(xs, t, 1.0)
    check_backward(run_backward(B, d, xs, t, top, log_sum), d, xs, t, top, log_sum)


@pytest.mark.parametrize("rows", [6, 1104])
def test_rows_without_a_distribution(B, form, rows):
    """NaN, +inf or nothing but -inf give NaN, in these rows and no others; ignored rows are not looked at."""
    xs, t = inputs(rows, [640, 333], torch.bfloat16, 11, ignored=0.0)
    xs[0][0, 17], xs[1][1, 330] = NAN, INF
    xs[0][2], xs[1][2] = -INF, -INF
    xs[0][3], xs[1][3] = NAN, NAN
    t[3] = -1
    xs[1][4, 2] = NAN
    t[4] = -(1 << 62)
    logp, top, log_sum = run_forward(B, xs, t)
    assert torch.isnan(logp[:3]).all() and (logp[3:5] == 0).all() and (top[3:5] == 0).all() and (log_sum[3:5] == 0).all()
    rest = [x[5:] for x in xs]
    check_forward((logp[5:], top[5:], log_sum[5:]), rest, t[5:])
    out = run_backward(B, torch.ones(rows), xs, t, top.cpu(), log_sum.cpu())
    got = torch.cat([o.float().cpu() for o in out[:2]], 1)
    assert torch.isnan(got[0]).all() and torch.isnan(got[1, 640 + 330]) and torch.isnan(got[2]).all()
    assert (got[3:5] == 0).all() and torch.isfinite(got[5:]).all()
    zero = run_backward(B, torch.zeros(rows), xs, t, top.cpu(), log_sum.cpu())
    assert all((o == 0).all() for o in zero)


@pytest.mark.parametrize("rows", [4, 1100])
def test_a_target_past_the_vocabulary(B, form, rows):
    xs, t = inputs(rows, [50, 70], torch.float32, 12, ignored=0.0)
    t[0], t[1] = 120 + 33000 * MORE[1], (1 << 62)
    t[2] = 119
    logp, top, log_sum = run_forward(B, xs, t)
    assert torch.isnan(logp[:2]).all() and torch.isfinite(logp[2:]).all()
    d = torch.ones(rows)
    d[1] = 0.0
    out = torch.cat([o.cpu() for o in run_backward(B, d, xs, t, top.cpu(), log_sum.cpu())[:2]], 1)
    assert torch.isnan(out[0]).all() and (out[1] == 0).all() and torch.isfinite(out[2:]).all()


@pytest.mark.parametrize("rows", [3, 1100])
def test_far_logits(B, form, rows):
    """Large offsets cancel, and neither large nor small logits overflow."""
    xs, t = inputs(rows, [900, 200], torch.float32, 13, ignored=0.0)
    for scale, shift in ((1.0, 1000.0), (1.0, -30000.0), (64.0, 0.0), (2.0 ** -10, 0.0)):
        far = [x + shift for x in xs]
        check_forward(run_forward(B, far, t, scale), far, t, scale)
    for scale, size in ((1e-37, 1e37), (1.0, 1e30), (2.0 ** 127, 1.0)):
        big = [x * size for x in xs]
        check_forward(run_forward(B, big, t, scale), big, t, scale)


@pytest.mark.parametrize("rows", [2, 1100])
def test_equal_logits(B, form, rows):
    """Every token equally likely: logSum is ln n."""
    for v in (0.0, 5.5, -65000.0, 2900.0, 1e30, -3e38, torch.finfo(torch.float32).max):
        xs = [torch.full((rows, c), v) for c in (1000, 24)]
        t = torch.arange(rows) % 1024
        logp, top, log_sum = run_forward(B, xs, t)
        assert (top == v).all() and (log_sum.double() - math.log(1024)).abs().max() <= 8 * ou.U * math.log(1024)
        check_forward((logp, top, log_sum), xs, t)


def test_gradient_sums_to_zero_and_agrees_with_differences(B):
    rows, shards, scale = 7, [40, 25], 1.25
    xs, t = inputs(rows, shards, torch.float32, 14, ignored=0.0, std=1.0)
    g = torch.Generator().manual_seed(2)
    d = torch.randn(rows, generator=g)
    top, log_sum = statistics(xs, t, scale)
    grad = torch.cat([o.double().cpu() for o in run_backward(B, d, xs, t, top, log_sum, scale)], 1)
    assert (grad.sum(1).abs() <= 65 * 40 * ou.U * d.abs().double()).all()
    move = torch.randn(rows, sum(shards), generator=g)
    h = 2.0 ** -6

    def value(k):
        far = [(x + k * m) for x, m in zip(xs, move.split(shards, 1))]
        logp = run_forward(B, [v.contiguous() for v in far], t, scale)[0]
        return (logp.double().cpu() * d.double())

    slope = (value(h) - value(-h)) / (2 * h)
    want = (grad * move.double()).sum(1)
    # the third derivative of logp along a move is at most that of a log-sum-exp: 2 (spread of the move)^3
    third = 2 * (scale * (move.amax(1) - move.amin(1)).double()) ** 3 * d.abs().double()
    assert ((slope - want).abs() <= third * h * h / 6 + 400 * ou.U / h * d.abs().double()).all()


@pytest.mark.parametrize("rows,shards", [(3, [5000, 5001]), (3, [25000, 15001]), (1200, [500, 300])], ids=str)
def test_graphs_replayed_side_by_side(B, rows, shards):
    """Two graphs, each with its own workspace, replayed on two streams with new logits."""
    sets = []
    for i in range(2):
        xs, t = inputs(rows, shards, torch.bfloat16, 30 + i)
        x, tt = [v.cuda() for v in xs], t.cuda()
        logp, top, log_sum, d = (torch.empty(rows, device="cuda") for _ in range(4))
        d.fill_(1.0)
        out = [torch.empty_like(v) for v in x]
        ws = torch.empty(max(16, B.arTokenLogprobWorkspace(rows, shards)), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            B.arTokenLogprob(x, tt, logp, top, log_sum, workspace=ws)
            B.arTokenLogprobBackward(d, x, tt, top, log_sum, out)
        sets.append((x, tt, logp, top, log_sum, d, out, ws, graph, torch.cuda.Stream()))
    for k in range(3):
        hosts = []
        for i, s in enumerate(sets):
            xs, t = inputs(rows, shards, torch.bfloat16, 50 + 2 * k + i)
            for a, b in zip(s[0], xs):
                a.copy_(b)
            s[1].copy_(t)
            for v in (s[2], s[3], s[4]):
                v.fill_(NAN)
            hosts.append((xs, t))
        torch.cuda.synchronize()
        for s in sets:
            with torch.cuda.stream(s[9]):
                s[8].replay()
        torch.cuda.synchronize()
        for s, (xs, t) in zip(sets, hosts):
            check_forward((s[2], s[3], s[4]), xs, t)
            check_backward(s[6], torch.ones(rows), xs, t, s[3].cpu(), s[4].cpu())


@pytest.mark.parametrize("rows", [3, 1100])
def test_row_strides_past_32_bits(B, rows):
    """The last row starts past 2^32 elements, forward, backward and in place."""
    cols = 37
    stride = ((1 << 32) + 64) // (rows - 1) + 1
    buf = torch.empty(stride * (rows - 1) + cols, dtype=torch.bfloat16, device="cuda")
    view = buf.as_strided((rows, cols), (stride, 1))
    xs, t = inputs(rows, [cols], torch.bfloat16, 15, ignored=0.0)
    view.copy_(xs[0])
    logp, top, log_sum = (torch.empty(rows, device="cuda") for _ in range(3))
    B.arTokenLogprob([view], t.cuda(), logp, top, log_sum)
    B.arTokenLogprobBackward(torch.ones(rows, device="cuda"), [view], t.cuda(), top, log_sum, [view])
    torch.cuda.synchronize()
    check_forward((logp, top, log_sum), xs, t)
    check_backward([view.clone()], torch.ones(rows), xs, t, top.cpu(), log_sum.cpu())


def test_a_long_vocabulary(B):
    """2^26 + 5 columns in one shard and a few in others."""
    shards = [(1 << 26) + 5, 3, 1000]
    xs = [torch.randn(2, c) for c in shards]
    t = torch.tensor([(1 << 26) + 4, sum(shards) - 1])
    check_forward(run_forward(B, xs, t), xs, t)
    d, (top, log_sum) = torch.tensor([1.0, -2.0]), statistics(xs, t, 1.0)
    check_backward(run_backward(B, d, xs, t, top, log_sum), d, xs, t, top, log_sum)


def test_no_rows(B):
    e = torch.empty(0, device="cuda")
    x = [torch.empty(0, 20, device="cuda")]
    t = torch.empty(0, dtype=torch.int64, device="cuda")
    B.arTokenLogprob(x, t, e, e, e)
    B.arTokenLogprobBackward(e, x, t, e, e, x)
    torch.cuda.synchronize()


@pytest.mark.parametrize("rows", [7, 1300])
def test_column_slices_of_one_buffer(B, rows):
    """The shards as slices of one wide logits tensor, the gradient in place."""
    shards = [100, 37, 3, 250]
    xs, t = inputs(rows, shards, torch.float16, 21)
    wide = torch.cat(xs, 1).cuda()
    views = list(wide.split(shards, 1))
    logp, top, log_sum = (torch.full((rows,), NAN, device="cuda") for _ in range(3))
    B.arTokenLogprob(views, t.cuda(), logp, top, log_sum)
    d = gradients(rows, 22)
    B.arTokenLogprobBackward(d.cuda(), views, t.cuda(), top, log_sum, views)
    torch.cuda.synchronize()
    check_forward((logp, top, log_sum), xs, t)
    check_backward([v.contiguous() for v in views], d, xs, t, top.cpu(), log_sum.cpu())
