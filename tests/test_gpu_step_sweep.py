"""A seeded random sweep of dropout, token log-probabilities and the policy loss: ranks, ragged and empty rows, widths
from 1 to 40000, types, padding, odd addresses, in place, many ranks; calls from two host threads at once; errors of
other calls; streams of another device."""
import ctypes
import math
import random
import threading

import op_util as ou
import pytest
import step_util as su
import test_gpu_dropout as dp
import test_gpu_logprob as lp
import test_gpu_policy as pol
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from ring_allreduce_reduction_amd import binding
    binding.lib()
    return binding


def log_int(rng, most):
    return max(1, int(math.exp(rng.uniform(0, math.log(most)))))


@pytest.mark.parametrize("seed", range(40))
def test_random_dropout(B, seed):
    import gpu_util
    rng = random.Random(3000 + seed)
    dt, wt = rng.choice(ou.TYPES)
    n, cols = rng.choice([1, 1, 2, 3, 5, 8, 17, 20]), log_int(rng, 40000)
    most = max(1, (4000000 if seed % 8 == 0 else 300000) // cols)
    rows = [min(20000, rng.choice([0, 1, rng.randint(0, max(1, 2 * most // n))])) for _ in range(n)]
    p, pad, offs, into = rng.choice([0.0, 0.1, 0.5, 0.9, 1.0]), rng.choice([0, 1, 3, 8]), rng.choice([0, 1, 7]), rng.choice([None, "x", "z"])
    first = None if rng.random() < 0.5 else [rng.randint(0, (1 << 32) - 20000) for _ in rows]
    key, offset = rng.getrandbits(64), rng.getrandbits(64)
    gpu_util.note("dropout sweep %d: %s %s cols %d rows %s p %g pad %d offset %d in place %s" % (seed, dt, wt, cols, rows, p, pad, offs, into))
    xs, zs, bs = dp.inputs(rows, cols, dt, wt, seed)
    kept = dp.masks(rows, cols, p, key, offset, first)
    zs = zs if into == "z" or rng.random() < 0.7 else None
    bs = bs if rng.random() < 0.7 else None
    dp.check_forward(dp.run_forward(B, xs, zs, bs, p, key, offset, None, first, pad, offs, into), xs, zs, bs, kept, p)
    dp.check_backward(*dp.run_backward(B, xs, wt, p, key, offset, None, first, pad, offs, inplace=into == "x"), xs, kept, p)


@pytest.mark.parametrize("seed", range(40))
def test_random_logprob(B, seed):
    import gpu_util
    rng = random.Random(4000 + seed)
    dt, n = rng.choice(lp.DTYPES), rng.choice([1, 1, 2, 3, 4, 5, 8, 16, 17, 30])
    width = log_int(rng, 60000 // n)
    shards = [max(0, width - rng.choice([0, 0, 1, 5, width])) for _ in range(n)]
    shards[rng.randrange(n)] = width
    rows = min(5000, log_int(rng, max(2, (6000000 if seed % 8 == 0 else 1000000) // sum(shards))))
    scale, pad, offs, inplace = rng.choice([1.0, 0.5, 1.3]), rng.choice([0, 1, 3, 8]), rng.choice([0, 1, 7]), rng.random() < 0.4
    gpu_util.note("logprob sweep %d: %s rows %d shards %s scale %g pad %d offset %d" % (seed, dt, rows, shards, scale, pad, offs))
    xs, t = lp.inputs(rows, shards, dt, seed)
    lp.check_forward(lp.run_forward(B, xs, t, scale, pad, offs, stats=rng.random() < 0.8), xs, t, scale)
    d, (top, log_sum) = lp.gradients(rows, seed), lp.statistics(xs, t, scale)
    out = lp.run_backward(B, d, xs, t, top, log_sum, scale, pad, offs, inplace=inplace)
    lp.check_backward(out, d, xs, t, top, log_sum, scale)


@pytest.mark.parametrize("seed", range(24))
def test_random_policy(B, seed):
    import gpu_util
    rng = random.Random(5000 + seed)
    n = rng.choice([1, 1, 2, 3, 8, 16, 17, 33])
    tokens = [rng.choice([0, 1, log_int(rng, 200000 // n)]) for _ in range(n)]
    kw = dict(low=rng.choice([0.1, 0.2, 1.0]), high=rng.choice([0.2, 0.3, 5.0]), kl=rng.choice([0.0, 0.01, 1.0]),
              denominator=rng.choice([0.0, 0.0, 123.0]), scale=rng.choice([1.0, 256.0]), ref=rng.random() < 0.7, weight=rng.random() < 0.7)
    gpu_util.note("policy sweep %d: %s %s" % (seed, tokens, kw))
    data = pol.inputs(tokens, seed, spread=rng.choice([0.05, 0.3, 2.0]))
    pol.check(pol.run(B, data, inplace=rng.random() < 0.3, **kw), data, **kw)


@pytest.mark.parametrize("rows,cols", [(20, 300), (1300, 1030)], ids=str)
def test_two_threads_at_once(B, rows, cols):
    import gpu_util
    gpu_util.note("two threads, %d x %d" % (rows, cols))
    sets, failures = [], []
    for i in range(2):
        xs, zs, bs = dp.inputs([rows, 3], cols, torch.bfloat16, torch.float32, 10 * i + 1)
        ls, t = lp.inputs(rows, [cols, 7], torch.float32, i)
        data = pol.inputs([5 * rows, 9], i)
        h = dict(host=(xs, zs, bs, ls, t, data), stream=torch.cuda.Stream())
        h["x"], h["z"], h["b"], h["l"] = ([v.cuda() for v in ts] for ts in (xs, zs, bs, ls))
        h["y"], h["dx"], h["db"] = ([torch.empty_like(v) for v in ts] for ts in (h["x"], h["x"], h["b"]))
        h["dl"], h["t"] = [torch.empty_like(v) for v in h["l"]], t.cuda()
        h["s"] = [torch.empty(rows, device="cuda") for _ in range(3)]
        h["p"] = [[v.cuda() for v in ts] for ts in data]
        h["g"], h["stats"] = [torch.empty_like(v) for v in h["p"][0]], torch.empty(5, device="cuda")
        sets.append(h)
    ones = torch.ones(rows, device="cuda")
    torch.cuda.synchronize()

    def work(i, h):
        try:
            for _ in range(15):
                B.arDropoutAdd(h["x"], h["y"], 0.3, i, 5, None, h["b"], h["z"], stream=h["stream"])
                B.arDropoutAddBackward(h["x"], h["dx"], 0.3, i, 5, None, h["db"], stream=h["stream"])
                B.arTokenLogprob(h["l"], h["t"], *h["s"], stream=h["stream"])
                B.arTokenLogprobBackward(ones, h["l"], h["t"], h["s"][1], h["s"][2], h["dl"], stream=h["stream"])
                p = h["p"]
                B.arPolicyLoss(p[0], p[1], p[3], h["stats"], p[2], p[4], h["g"], 0.2, 0.28, 0.05, stream=h["stream"])
        except Exception as e:   # reported by the test's own thread
            failures.append(e)

    threads = [threading.Thread(target=work, args=(i, h)) for i, h in enumerate(sets)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failures, failures
    for i, h in enumerate(sets):
        xs, zs, bs, ls, t, data = h["host"]
        kept = dp.masks([rows, 3], cols, 0.3, i, 5)
        dp.check_forward(h["y"], xs, zs, bs, kept, 0.3)
        dp.check_backward(h["dx"], h["db"], xs, kept, 0.3)
        lp.check_forward(h["s"], ls, t)
        lp.check_backward(h["dl"], torch.ones(rows), ls, t, h["s"][1].cpu(), h["s"][2].cpu())
        pol.check((h["stats"], h["g"]), data)


def calls(B):
    """One call of each operator on small tensors, as functions of a stream, and what they write."""
    x, t, f = torch.randn(4, 8, device="cuda"), torch.arange(4, device="cuda"), torch.zeros(4, device="cuda")
    y, d, out = torch.empty_like(x), torch.empty_like(x), [torch.empty(4, device="cuda") for _ in range(3)]
    db, g, s = torch.empty(8, device="cuda"), torch.empty(4, device="cuda"), torch.empty(5, device="cuda")
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    return [lambda st=None: B.arDropoutAdd([x], [y], 0.5, 1, stream=st),
            lambda st=None: B.arDropoutAddBackward([x], [d], 0.5, 1, dbiases=[db], workspace=ws, stream=st),
            lambda st=None: B.arTokenLogprob([x], t, *out, workspace=ws, stream=st),
            lambda st=None: B.arTokenLogprobBackward(f, [x], t, out[1], out[2], [d], stream=st),
            lambda st=None: B.arPolicyLoss([f], [f], [f], s, dlogps=[g], workspace=ws, stream=st)], (x, y, d, out, db, g, s)


def test_an_earlier_error_is_not_reported(B):
    """A HIP call of the program's own that failed (an ordinal no device has) before each operator."""
    hip = ctypes.CDLL("libamdhip64.so.7")   # the runtime torch has loaded
    fs, _ = calls(B)
    try:
        for f in fs:
            assert hip.hipSetDevice(9999) != 0
            f()
    finally:
        hip.hipGetLastError()
    torch.cuda.synchronize()


class StreamElsewhere:
    """A stream of a second device, as torch's streams look."""
    def __init__(self, device_index):
        self.device_index = device_index
        self.cuda_stream = 0


def test_a_stream_of_another_device_is_refused(B):
    here = torch.cuda.current_device()
    fs, _ = calls(B)
    for f in fs:
        with pytest.raises(ValueError, match="stream is on cuda:%d" % (here + 1)):
            f(StreamElsewhere(here + 1))
        f(StreamElsewhere(here))
    torch.cuda.synchronize()


def test_workspaces_are_allocated_where_none_is_given(B):
    """On the stream that uses them; too small ones are refused."""
    st = torch.cuda.Stream()
    xs, t = lp.inputs(5, [30000, 20000], torch.float32, 2)
    lp.check_forward(lp.run_forward(B, xs, t, stream=st), xs, t)
    small = torch.empty(8, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="workspace must be contiguous and hold"):
        lp.run_forward(B, xs, t, workspace=small)
    dys, _, _ = dp.inputs([40], 70, torch.float32, torch.float32, 1)
    dp.check_backward(*dp.run_backward(B, dys, torch.float32, 0.5, stream=st), dys, dp.masks([40], 70, 0.5, dp.SEED, dp.OFFSET), 0.5)
    with pytest.raises(ValueError, match="workspace must be contiguous and hold"):
        dp.run_backward(B, dys, torch.float32, 0.5, workspace=small)
    data = pol.inputs([9000], 1)
    pol.check(pol.run(B, data, stream=st), data)
    with pytest.raises(ValueError, match="workspace must be contiguous and hold"):
        pol.run(B, data, workspace=small)


def test_equal_calls_give_equal_bits(B):
    """Every sum has a fixed order."""
    dys, _, _ = dp.inputs([900, 700], 1000, torch.float32, torch.float32, 4)
    a, b = (dp.run_backward(B, dys, torch.float32, 0.3)[1][0] for _ in range(2))
    assert torch.equal(a, b)
    for rows, shards in ((3, [9000, 9000]), (3, [30000, 9000]), (1100, [900, 800])):
        xs, t = lp.inputs(rows, shards, torch.bfloat16, 3)
        a, b = (lp.run_forward(B, xs, t) for _ in range(2))
        assert all(torch.equal(u, v) for u, v in zip(a, b))
    data = pol.inputs([30000, 500], 3)
    a, b = (pol.run(B, data) for _ in range(2))
    assert torch.equal(a[0], b[0]) and all(torch.equal(u, v) for u, v in zip(a[1], b[1]))
