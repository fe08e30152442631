"""Dropout and token log-probabilities of calls that move more than 256 MB, which load and store past the caches:
every such form of them, at odd widths, odd addresses and in place, against the 64-bit forms (step_util) on the device."""
import device_util as du
import op_util as ou
import pytest
import step_util as su
import torch

CACHES = 256 << 20
SEED, OFFSET = 0x9ABCDEF012345678, 0x1122334455667788
DTYPES = [torch.float32, torch.float16, torch.bfloat16]


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


def size_of(dt):
    return torch.finfo(dt).bits // 8


@pytest.mark.parametrize("rows,first,cols,seed,offset", [(3, 0, 20, 0, 0), (5, (1 << 32) - 5, 8, (1 << 64) - 1, (1 << 64) - 2),
                                                         (2, 9, 1030, SEED, OFFSET)])
def test_the_device_generator(rows, first, cols, seed, offset):
    assert torch.equal(du.drawn(rows, first, cols, seed, offset, "cpu"), su.drawn(rows, first, cols, seed, offset))


def shares(total, n):
    """Rows of n ranks, uneven, one of them without any."""
    if n == 3:
        return [total - total // 3, 0, total // 3]
    return [0] + [total // (n - 1) + 1 - r % 2 for r in range(1, n)]


def values(shape, dt, g, std=1.0, mean=0.0):
    return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dt)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [3, 17])
@pytest.mark.parametrize("dt,wt", ou.TYPES, ids=str)
@pytest.mark.parametrize("cols", [515, 2048, 8191])
def test_dropout(B, cols, dt, wt, n):
    """With bias and residual, in place of neither, the rows and the residual; and with neither."""
    p, g = 0.3, torch.Generator(device="cuda").manual_seed(cols + n)
    into = {515: None, 2048: "x", 8191: "z"}[cols]
    rows = shares(CACHES // (3 * size_of(dt) * cols) + 50, n)
    assert 3 * size_of(dt) * cols * sum(rows) > CACHES
    xs, zs = [values((k, cols), dt, g) for k in rows], [values((k, cols), dt, g, 2.0) for k in rows]
    bias = values((cols,), wt, g, 0.3)
    kept = du.masks(rows, cols, p, SEED, OFFSET, "cuda")
    x, z = [du.padded(t, 3, 1) for t in xs], [du.padded(t, 8, 5) for t in zs]
    y = {"x": x, "z": z}.get(into) or [du.padded(torch.full_like(t, float("nan")), 1, 0) for t in xs]
    B.arDropoutAdd(x, y, p, SEED, OFFSET, None, [bias.clone() for _ in rows], z)
    for r in range(n):
        if rows[r]:
            want, bound = su.dropout(xs[r], bias, zs[r], kept[r], p)
            du.within(y[r], want, bound, "y of rank %d" % r)
            assert (du.around(y[r]) == 77).all()
    del x, y, z, zs
    more = [torch.cat((t, t[: (len(t) + 1) // 2 + 1])) for t in xs]   # two buffers a call in place of three
    rows = [len(t) for t in more]
    assert 2 * size_of(dt) * cols * sum(rows) > CACHES
    kept = du.masks(rows, cols, p, SEED, OFFSET, "cuda")
    y = [du.padded(torch.full_like(t, float("nan")), 1, 0) for t in more]
    B.arDropoutAdd([du.padded(t, 3, 1) for t in more], y, p, SEED, OFFSET)
    for r in range(n):
        if rows[r]:
            want, bound = su.dropout(more[r], None, None, kept[r], p)
            du.within(y[r], want, bound, "y of rank %d without residual" % r)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [3, 17])
@pytest.mark.parametrize("dt,wt", ou.TYPES, ids=str)
@pytest.mark.parametrize("cols", [515, 2048, 8191])
def test_dropout_backward(B, cols, dt, wt, n):
    """Whole numbers up to 8 and a scale of 2: every sum is exact, whatever its order.  dx and dbias, dx alone, dbias
    alone, the last in place of nothing, the others in place or not."""
    p, g = 0.5, torch.Generator(device="cuda").manual_seed(cols + n)
    rows = shares(CACHES // (2 * size_of(dt) * cols) + 50, n)
    assert 2 * size_of(dt) * cols * sum(rows) > CACHES and 16 * sum(rows) < 1 << 24
    dys = [torch.randint(-8, 9, (k, cols), generator=g, device="cuda").to(dt) for k in rows]
    dxs = [torch.where(k, 2.0 * d, 0.0).to(dt) for k, d in zip(du.masks(rows, cols, p, SEED, OFFSET, "cuda"), dys)]
    dbias = sum(d.double().sum(0) for d in dxs).to(wt)
    for inplace in (False, True):
        dy = [du.padded(t, 3, 1) for t in dys]
        dx = dy if inplace else [du.padded(torch.full_like(t, float("nan")), 1, 0) for t in dys]
        db = [torch.full((cols,), float("nan"), dtype=wt, device="cuda") for _ in rows]
        B.arDropoutAddBackward(dy, dx, p, SEED, OFFSET, None, db)
        assert all(torch.equal(a, b) for a, b in zip(dx, dxs))
        assert all((du.around(a) == 77).all() for a in dx)
        assert all(torch.equal(b, dbias) for b in db)
    dx = [torch.full_like(t, float("nan")) for t in dys]
    B.arDropoutAddBackward(dys, dx, p, SEED, OFFSET)
    assert all(torch.equal(a, b) for a, b in zip(dx, dxs))
    more = [torch.cat((t, t)) for t in dys]   # one buffer a call in place of two
    db = [torch.full((cols,), float("nan"), dtype=wt, device="cuda") for _ in rows]
    B.arDropoutAddBackward(more, None, p, SEED, OFFSET, None, db)
    kept = du.masks([len(t) for t in more], cols, p, SEED, OFFSET, "cuda")
    dbias = sum(torch.where(k, 2.0 * d, 0.0).double().sum(0) for k, d in zip(kept, more)).to(wt)
    assert all(torch.equal(b, dbias) for b in db)


# Shards by how many vectors of 16 bytes they have and how many elements more: 16 threads a shard of four, of two and of
# 17; eight wavefronts for five shards and for 17; four for four; a wavefront a row; four wavefronts for two shards; four
# and eight together
ROWS = {"narrow": [(101, -3), (99, 1), (0, 0), (100, 0)], "narrow, two": [(100, 1), (90, -1)], "narrow, 17": [(20, 3)] * 17,
        "five": [(400, 3), (0, 1), (900, -1), (500, 0), (600, 1)], "17": [(400, 1)] * 16 + [(0, 0)], "four": [(400, 1)] * 4,
        "one": [(900, 3)], "two": [(800, 1), (801, 0)], "wide": [(1200, 3)], "wider": [(2000, -1)]}


def logits(shards, dt, most, seed):
    """Logits of more than `most` bytes and targets, a tenth of them ignored."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = 16 // size_of(dt)
    widths = [k * v + more for k, more in shards]
    rows = most // (sum(widths) * size_of(dt)) + 77
    assert rows * sum(widths) * size_of(dt) > most
    xs = [values((rows, c), dt, g, 3.0, 1.0) for c in widths]
    t = torch.randint(0, sum(widths), (rows,), generator=g, device="cuda")
    t[torch.rand(rows, generator=g, device="cuda") < 0.1] = -100
    return xs, t


def blocks(xs):
    rows, width = len(xs[0]), sum(x.shape[1] for x in xs)
    each = max(1, (1 << 25) // width)
    for i in range(0, rows, each):
        yield slice(i, i + each), torch.cat([x[i:i + each] for x in xs], 1)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES, ids=str)
@pytest.mark.parametrize("form", ROWS)
def test_logprob(B, form, dt):
    xs, t = logits(ROWS[form], dt, CACHES, len(form))
    x = [du.padded(v, 1 + r % 3, r % 2) for r, v in enumerate(xs)]
    for scale in (1.0, 0.7):
        logp, top, log_sum = (torch.full((len(t),), float("nan"), device="cuda") for _ in range(3))
        B.arTokenLogprob(x, t, logp, top, log_sum, scale)
        for at, whole in blocks(xs):
            want, m, s, d_want, d_s = su.logprob(whole, t[at], float(torch.tensor(scale)), len(xs))
            du.within(logp[at], want, d_want, "logp")
            assert torch.equal(top[at].double(), m)
            du.within(log_sum[at], s, d_s, "logSum")


@pytest.mark.gpu
@pytest.mark.parametrize("ranks", [3, 17])
@pytest.mark.parametrize("dt", DTYPES, ids=str)
@pytest.mark.parametrize("widest", [20, 100, 200, 380, 1100])
def test_logprob_backward(B, widest, dt, ranks):
    """16, 32, 64, 128 and 256 threads a row, beside the logits and in their place."""
    xs, t = logits([(widest, 3), (widest // 2, -1), (0, 3)] + [(1, r) for r in range(ranks - 3)], dt, CACHES // 2, widest)
    g = torch.Generator(device="cuda").manual_seed(1)
    d = torch.randn(len(t), generator=g, device="cuda")
    d[torch.rand(len(t), generator=g, device="cuda") < 0.1] = 0.0
    top, log_sum = (torch.empty(len(t), device="cuda") for _ in range(2))
    for at, whole in blocks(xs):
        _, m, s, _, _ = su.logprob(whole, t[at], 1.25, ranks)
        top[at], log_sum[at] = m.float(), s.float()
    for inplace in (False, True):
        x = [du.padded(v, 1 + r % 3, r % 2) for r, v in enumerate(xs)]
        out = x if inplace else [du.padded(torch.full_like(v, float("nan")), 2 + r % 3, r % 4) for r, v in enumerate(xs)]
        B.arTokenLogprobBackward(d, x, t, top, log_sum, out, 1.25)
        for at, whole in blocks(xs):
            want, bound = su.logprob_backward(d[at], whole, t[at], 1.25, top[at], log_sum[at])
            du.within(torch.cat([o[at] for o in out], 1), want, bound, "dlogits")
        assert all((du.around(o) == 77).all() for o in out)
