"""Layer norm over the ranks' rows, forward and backward with the weights' gradient summed over all ranks,
against the formulas in 64 bits (bounds in op_util) and against differences of the forward pass."""
import op_util as ou
import pytest
import torch

pytestmark = pytest.mark.gpu

COLS = [1, 2, 7, 64, 65, 255, 1000, 1024, 2047, 2048, 4097, 8192, 10000, 16384, 16391, 40000]


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


def dev(t, pad=0, offset=0):
    """t on the device, its rows pad elements apart and the first one offset elements into the allocation; every
    other element holds NaN."""
    if t is None:
        return None
    if t.dim() == 1:
        buf = torch.full((offset + t.numel(),), float("nan"), dtype=t.dtype, device="cuda")
        buf[offset:].copy_(t)
        return buf[offset:]
    k, c = t.shape
    buf = torch.full((offset + k * (c + pad),), float("nan"), dtype=t.dtype, device="cuda")
    view = buf[offset:].view(k, c + pad)[:, :c]
    view.copy_(t)
    return view


def untouched(view):
    """The bytes between a padded view's rows still hold NaN."""
    k, c = view.shape
    if k < 2 or view.stride(0) == c:
        return True
    gaps = view.as_strided((k - 1, view.stride(0) - c), (view.stride(0), 1), view.storage_offset() + c)
    return bool(torch.isnan(gaps.float()).all())


def inputs(rows, cols, dt, wt, seed, affine=True):
    g = torch.Generator().manual_seed(seed)
    xs = [ou.rows_of(g, (k, cols), dt, 0.5 + r % 3, (r % 3) - 1.0) for r, k in enumerate(rows)]
    dys = [ou.rows_of(g, (k, cols), dt, 0.1) for k in rows]
    gam = [ou.rows_of(g, (cols,), wt, 0.3, 1.0) for _ in rows] if affine else None
    bet = [ou.rows_of(g, (cols,), wt, 0.2) for _ in rows] if affine else None
    return xs, dys, gam, bet


def run_forward(B, xs, gam, bet, eps, pad=0, offset=0, ypad=None, stats=True, stream=None, inplace=False):
    dx = [dev(x, pad, offset) for x in xs]
    ys = dx if inplace else [dev(torch.full_like(x, float("nan")), pad if ypad is None else ypad, offset) for x in xs]
    m = [torch.full((len(x),), float("nan"), device="cuda") for x in xs] if stats else None
    s = [torch.full((len(x),), float("nan"), device="cuda") for x in xs] if stats else None
    dg = None if gam is None else [dev(t, 0, offset) for t in gam]
    db = None if bet is None else [dev(t, 0, offset) for t in bet]
    torch.cuda.synchronize()
    B.arLayerNorm(dx, ys, dg, db, m, s, eps=eps, stream=stream)
    torch.cuda.synchronize()
    return ys, m, s


def check_forward(xs, gam, bet, eps, ys, m, s):
    for r, x in enumerate(xs):
        y, mean, rstd, ey, em, es = ou.ln_forward(x, None if gam is None else gam[r], None if bet is None else bet[r], eps)
        ou.within(ys[r], y, ey, x.dtype, "y of rank %d" % r)
        assert untouched(ys[r])
        if m is not None:
            ou.within(m[r], mean, em, torch.float32, "mean of rank %d" % r)
            ou.within(s[r], rstd, es, torch.float32, "rstd of rank %d" % r)


def run_backward(B, dys, xs, gam, eps, pad=0, offset=0, dx=True, dg=True, db=True, into=None, stream=None,
                 workspace=None):
    """Device results and the float statistics used."""
    means = [x.double().mean(1).float() for x in xs]
    rstds = [((x.double() - x.double().mean(1, keepdim=True)).square().mean(1) + eps).rsqrt().float() for x in xs]
    d, x = [dev(t, pad, offset) for t in dys], [dev(t, pad, offset) for t in xs]
    out = None
    if dx:
        out = {"dy": d, "x": x}.get(into) or [dev(torch.full_like(t, float("nan")), pad, offset) for t in xs]
    cols, wt = xs[0].shape[1], xs[0].dtype if gam is None else gam[0].dtype
    gg = [torch.full((cols,), float("nan"), dtype=wt, device="cuda") for _ in xs] if dg else None
    gb = [torch.full((cols,), float("nan"), dtype=wt, device="cuda") for _ in xs] if db else None
    torch.cuda.synchronize()
    B.arLayerNormBackward(d, x, [dev(t) for t in means], [dev(t) for t in rstds],
                          None if gam is None else [dev(t, 0, offset) for t in gam], out, gg, gb, stream=stream,
                          workspace=workspace)
    torch.cuda.synchronize()
    return out, gg, gb, means, rstds


def check_backward(dys, xs, gam, out, gg, gb, means, rstds):
    cols = xs[0].shape[1]
    sums = [torch.zeros(cols, dtype=torch.float64) for _ in range(4)]
    nrows = sum(len(x) for x in xs)
    for r, x in enumerate(xs):
        dx, bound, p, d = ou.ln_backward(dys[r], x, means[r], rstds[r], None if gam is None else gam[r])
        if out is not None:
            ou.within(out[r], dx, bound, x.dtype, "dx of rank %d" % r)
            assert untouched(out[r])
        for s, t in zip(sums, (p, p.abs(), d, d.abs())):
            s += t.sum(0)
    # a column's sum: any order of nrows additions, and for dgamma the roundings of h and of the product
    for name, got, want, size in (("dgamma", gg, sums[0], sums[1]), ("dbeta", gb, sums[2], sums[3])):
        if got is not None:
            for t in got:
                ou.within(t, want, (nrows + 4) * ou.U * size, t.dtype, name)


@pytest.mark.parametrize("dt,wt", ou.TYPES, ids=str)
@pytest.mark.parametrize("cols", COLS)
def test_forward(B, cols, dt, wt):
    rows = [5, 0, 3] if cols > 3000 else [37, 0, 18, 1]
    xs, _, gam, bet = inputs(rows, cols, dt, wt, cols)
    check_forward(xs, gam, bet, 1e-5, *run_forward(B, xs, gam, bet, 1e-5))


@pytest.mark.parametrize("dt,wt", ou.TYPES, ids=str)
@pytest.mark.parametrize("cols", COLS)
def test_backward(B, cols, dt, wt):
    rows = [5, 0, 3] if cols > 3000 else [37, 0, 18, 1]
    xs, dys, gam, _ = inputs(rows, cols, dt, wt, cols + 1)
    check_backward(dys, xs, gam, *run_backward(B, dys, xs, gam, 1e-5))


@pytest.mark.parametrize("cols", [3, 64, 770, 2049, 9000, 20000])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=str)
def test_padded_rows_and_odd_addresses(B, cols, dt):
    """Rows inside wider ones, the first at an odd element: what lies between them is neither read nor written."""
    for pad, offset in ((1, 0), (8, 1), (5, 3)):
        xs, dys, gam, bet = inputs([6, 2], cols, dt, torch.float32, cols + pad)
        check_forward(xs, gam, bet, 1e-5, *run_forward(B, xs, gam, bet, 1e-5, pad, offset, ypad=pad + 2))
        check_backward(dys, xs, gam, *run_backward(B, dys, xs, gam, 1e-5, pad, offset))


@pytest.mark.parametrize("n", [2, 16, 17, 32, 33, 72, 128])
def test_many_ranks(B, n):
    """Past 16 ranks the rows take several launches; ranks without rows still receive the weights' gradient."""
    rows = [(3 * r + 2) % 5 for r in range(n)]
    xs, dys, gam, bet = inputs(rows, 130, torch.float32, torch.float32, n)
    check_forward(xs, gam, bet, 1e-5, *run_forward(B, xs, gam, bet, 1e-5))
    check_backward(dys, xs, gam, *run_backward(B, dys, xs, gam, 1e-5))


@pytest.mark.parametrize("cols", [64, 1000, 4096, 20000])
def test_without_weights_and_parts(B, cols):
    xs, dys, gam, _ = inputs([9, 4], cols, torch.float16, torch.float16, 3)
    check_forward(xs, None, None, 1e-5, *run_forward(B, xs, None, None, 1e-5, stats=False))
    check_backward(dys, xs, None, *run_backward(B, dys, xs, None, 1e-5))
    for dx, dg, db in ((True, False, False), (False, True, False), (False, False, True), (True, True, False)):
        check_backward(dys, xs, gam, *run_backward(B, dys, xs, gam, 1e-5, dx=dx, dg=dg, db=db))


@pytest.mark.parametrize("cols", [7, 1024, 5000, 20000])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=str)
def test_in_place(B, cols, dt):
    xs, dys, gam, bet = inputs([11, 3], cols, dt, torch.float32, 5)
    check_forward(xs, gam, bet, 1e-5, *run_forward(B, xs, gam, bet, 1e-5, pad=2, inplace=True))
    for into in ("dy", "x"):
        check_backward(dys, xs, gam, *run_backward(B, dys, xs, gam, 1e-5, pad=2, into=into))


@pytest.mark.parametrize("rows", [[0], [0, 0, 0]])
def test_no_rows(B, rows):
    xs, dys, gam, bet = inputs(rows, 100, torch.float32, torch.float32, 5)
    run_forward(B, xs, gam, bet, 1e-5)
    _, gg, gb, _, _ = run_backward(B, dys, xs, gam, 1e-5)
    for t in gg + gb:
        assert torch.equal(t.cpu(), torch.zeros(100))


def test_large_offset_and_constant_rows(B):
    """A mean a thousand times the spread; rows of one value have variance 0 and come out as beta."""
    g = torch.Generator().manual_seed(1)
    for cols in (600, 5000, 30000):
        x = ou.rows_of(g, (6, cols), torch.float32, 1.0, 1000.0)
        x[2] = 5.0
        x[4] = 0.0
        gam, bet = [ou.rows_of(g, (cols,), torch.float32)], [ou.rows_of(g, (cols,), torch.float32)]
        ys, m, s = run_forward(B, [x], gam, bet, 1e-3)
        check_forward([x], gam, bet, 1e-3, ys, m, s)
        assert torch.equal(ys[0][2].cpu(), bet[0]) and torch.equal(ys[0][4].cpu(), bet[0])


@pytest.mark.parametrize("cols", [64, 1000, 4100, 20000])
def test_nan_and_infinity_stay_in_their_row(B, cols):
    xs, dys, gam, bet = inputs([8], cols, torch.bfloat16, torch.float32, 9)
    xs[0][3, cols // 2] = float("nan")
    xs[0][5, 0] = float("inf")
    ys, m, s = run_forward(B, xs, gam, bet, 1e-5)
    y = ys[0].float().cpu()
    assert torch.isnan(y[3]).all() and torch.isnan(y[5]).all()
    keep = [0, 1, 2, 4, 6, 7]
    check_forward([xs[0][keep]], gam, bet, 1e-5, [ys[0][keep]], [m[0][keep]], [s[0][keep]])
    xs, dys, gam, _ = inputs([8], cols, torch.bfloat16, torch.float32, 9)
    dys[0][2, 1] = float("nan")
    out, gg, gb, means, rstds = run_backward(B, dys, xs, gam, 1e-5)
    assert torch.isnan(out[0][2].float()).all() and torch.isfinite(out[0][[0, 1, 3, 4, 5, 6, 7]].float()).all()
    for t in gg + gb:
        assert torch.isnan(t[1]) and int(torch.isnan(t).sum()) == 1


@pytest.mark.parametrize("rows,cols", [([5000], 48), ([9000, 3000, 7001], 520), ([2500, 1], 4096), ([700], 17000)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=str)
def test_sums_over_many_rows_exactly(B, rows, cols, dt):
    """Small whole gradients and whole h (x = 0 or 1, mean 0, rstd 1): every partial sum is a whole number below
    2^24, so the sums are exact in 32 bits whatever their order, and no row may be missed or counted twice."""
    g = torch.Generator().manual_seed(cols)
    xs = [torch.randint(0, 2, (k, cols), generator=g).to(dt) for k in rows]
    dys = [torch.randint(-8, 9, (k, cols), generator=g).to(dt) for k in rows]
    gg = [torch.empty(cols, device="cuda") for _ in rows]
    gb = [torch.empty(cols, device="cuda") for _ in rows]
    B.arLayerNormBackward([t.cuda() for t in dys], [t.cuda() for t in xs], [torch.zeros(k, device="cuda") for k in rows],
                          [torch.ones(k, device="cuda") for k in rows], [torch.ones(cols, device="cuda") for _ in rows],
                          [torch.empty(k, cols, dtype=dt, device="cuda") for k in rows], gg, gb)
    want_b = sum(t.double().sum(0) for t in dys).float()
    want_g = sum((t.double() * x.double()).sum(0) for t, x in zip(dys, xs)).float()
    for t in gb:
        assert torch.equal(t.cpu(), want_b)
    for t in gg:
        assert torch.equal(t.cpu(), want_g)


@pytest.mark.parametrize("cols", [5, 70, 1030])
def test_gradients_against_differences(B, cols):
    """dL/dx, dL/dgamma, dL/dbeta of L = sum(dy * y) by central differences of the 64-bit forward pass: off by
    step^2 = 1e-8 times third derivatives of the order of rstd^3, so 1e-5 of the largest gradient covers both."""
    eps, step = 1e-2, 1e-4
    xs, dys, gam, bet = inputs([4], cols, torch.float32, torch.float32, 11)
    out, gg, gb, _, _ = run_backward(B, dys, xs, gam, eps)

    def loss(x, g, b):
        e = x - x.mean(1, keepdim=True)
        y = e / torch.sqrt((e * e).mean(1, keepdim=True) + eps) * g + b
        return (dys[0].double() * y).sum(1)

    x, g, b = xs[0].double(), gam[0].double(), bet[0].double()
    for c in range(0, cols, max(1, cols // 16)):
        e = torch.zeros(cols, dtype=torch.float64)
        e[c] = step
        dx = (loss(x + e, g, b) - loss(x - e, g, b)) / (2 * step)
        dg = ((loss(x, g + e, b) - loss(x, g - e, b)) / (2 * step)).sum()
        db = ((loss(x, g, b + e) - loss(x, g, b - e)) / (2 * step)).sum()
        for got, want, top in ((out[0][:, c], dx, out[0]), (gg[0][c], dg, gg[0]), (gb[0][c], db, gb[0])):
            assert (got.cpu().double() - want).abs().max() <= 1e-5 * top.abs().max().item()


@pytest.mark.parametrize("cols", [200, 3000])
def test_other_stream_and_graph(B, cols):
    """On a stream of the caller's, then captured (without an eager call first) and replayed on new inputs."""
    xs, dys, gam, bet = inputs([30, 7], cols, torch.bfloat16, torch.float32, 13)
    st = torch.cuda.Stream()
    check_forward(xs, gam, bet, 1e-5, *run_forward(B, xs, gam, bet, 1e-5, stream=st))
    check_backward(dys, xs, gam, *run_backward(B, dys, xs, gam, 1e-5, stream=st))
    d = {"x": [dev(t) for t in xs], "dy": [dev(t) for t in dys], "g": [dev(t) for t in gam], "b": [dev(t) for t in bet]}
    ys, dxs = [torch.empty_like(t) for t in d["x"]], [torch.empty_like(t) for t in d["x"]]
    m, s = [torch.empty(30, device="cuda"), torch.empty(7, device="cuda")], [torch.empty(30, device="cuda"), torch.empty(7, device="cuda")]
    gg, gb = [torch.empty_like(t) for t in d["g"]], [torch.empty_like(t) for t in d["g"]]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        B.arLayerNorm(d["x"], ys, d["g"], d["b"], m, s)
        B.arLayerNormBackward(d["dy"], d["x"], m, s, d["g"], dxs, gg, gb)
    for rep in range(3):
        xs, dys, gam, bet = inputs([30, 7], cols, torch.bfloat16, torch.float32, 14 + rep)
        for k, new in (("x", xs), ("dy", dys), ("g", gam), ("b", bet)):
            for a, t in zip(d[k], new):
                a.copy_(t)
        for t in ys + dxs + m + s + gg + gb:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check_forward(xs, gam, bet, 1e-5, ys, m, s)
        check_backward(dys, xs, gam, dxs, gg, gb, [t.cpu() for t in m], [t.cpu() for t in s])


def test_runs_are_bit_equal(B):
    xs, dys, gam, bet = inputs([301, 77], 1500, torch.float32, torch.float32, 17)
    first = None
    for _ in range(3):
        ys, m, s = run_forward(B, xs, gam, bet, 1e-5)
        out, gg, gb, _, _ = run_backward(B, dys, xs, gam, 1e-5)
        now = [t.cpu() for t in ys + m + s + out + gg + gb]
        first = first or now
        assert all(torch.equal(a, b) for a, b in zip(first, now))


def test_rows_far_apart(B):
    """Element offsets past 2^32: 70 rows 2^26 elements apart."""
    k, c, stride = 70, 513, 1 << 26
    big = [torch.empty(k * stride, dtype=torch.bfloat16, device="cuda").view(k, stride)[:, :c] for _ in range(3)]
    xs, dys, gam, bet = inputs([k], c, torch.bfloat16, torch.float32, 19)
    big[0].copy_(xs[0])
    big[1].copy_(dys[0])
    m, s = torch.empty(k, device="cuda"), torch.empty(k, device="cuda")
    B.arLayerNorm([big[0]], [big[2]], [gam[0].cuda()], [bet[0].cuda()], [m], [s])
    torch.cuda.synchronize()
    check_forward(xs, gam, bet, 1e-5, [big[2].contiguous()], [m], [s])
    gg, gb = [torch.empty(c, device="cuda")], [torch.empty(c, device="cuda")]
    B.arLayerNormBackward([big[1]], [big[0]], [m], [s], [gam[0].cuda()], [big[2]], gg, gb)
    torch.cuda.synchronize()
    check_backward(dys, xs, gam, [big[2].contiguous()], gg, gb, [m.cpu()], [s.cpu()])


def test_single_rows_of_other_shapes(B):
    """A 1-D row, and rows of a 3-D activation."""
    g = torch.Generator().manual_seed(2)
    x = ou.rows_of(g, (1, 900), torch.bfloat16)
    y = torch.empty(900, dtype=torch.bfloat16, device="cuda")
    B.arLayerNorm([x[0].cuda()], [y])
    check_forward([x], None, None, 1e-5, [y.view(1, 900)], None, None)
    x = ou.rows_of(g, (6, 40), torch.float32)
    y = torch.empty(2, 3, 40, device="cuda")
    B.arLayerNorm([x.view(2, 3, 40).cuda()], [y])
    check_forward([x], None, None, 1e-5, [y.view(6, 40)], None, None)


@pytest.mark.parametrize("rows", [[511], [512], [513], [500, 12], [500, 13, 0], [32] * 16, [16] * 32, [16] * 33, [1, 0, 511, 0]], ids=str)
@pytest.mark.parametrize("cols,dt", [(8, torch.bfloat16), (200, torch.bfloat16), (1031, torch.float32)], ids=str)
def test_around_the_few_rows_rule(B, rows, cols, dt):
    """Both sides of the row count where the weights' gradients change from one launch to two."""
    xs, dys, gam, _ = inputs(rows, cols, dt, torch.float32, sum(rows) + cols)
    check_backward(dys, xs, gam, *run_backward(B, dys, xs, gam, 1e-5))
    check_backward(dys, xs, gam, *run_backward(B, dys, xs, gam, 1e-5, dx=False))


def test_column_slices_of_one_buffer(B):
    """Inputs and outputs as columns of the same rows: they interleave and do not overlap."""
    xs, dys, gam, bet = inputs([20], 96, torch.bfloat16, torch.float32, 23)
    wide = torch.full((20, 400), float("nan"), dtype=torch.bfloat16, device="cuda")
    x, y, dy, dx = (wide[:, i:i + 96] for i in (0, 96, 200, 300))
    x.copy_(xs[0])
    dy.copy_(dys[0])
    m, s = [torch.empty(20, device="cuda")], [torch.empty(20, device="cuda")]
    B.arLayerNorm([x], [y], [gam[0].cuda()], [bet[0].cuda()], m, s)
    gg, gb = [torch.empty(96, device="cuda")], [torch.empty(96, device="cuda")]
    B.arLayerNormBackward([dy], [x], m, s, [gam[0].cuda()], [dx], gg, gb)
    torch.cuda.synchronize()
    check_forward(xs, gam, bet, 1e-5, [y.contiguous()], m, s)
    check_backward(dys, xs, gam, [dx.contiguous()], gg, gb, [m[0].cpu()], [s[0].cpu()])
    for lo, hi in ((192, 200), (296, 300), (396, 400)):
        assert torch.isnan(wide[:, lo:hi].float()).all()
    with pytest.raises(B.ArError):
        B.arLayerNorm([x], [wide[:, 95:191]])


def test_other_devices_and_lazy_negation_are_refused(B):
    x = torch.zeros(2, 8, device="cuda")
    with pytest.raises(ValueError, match="device tensors"):
        B.arLayerNorm([x], [x], [torch.zeros(8)])
    z = torch.zeros(2, 8, dtype=torch.complex64, device="cuda").conj().imag
    assert z.is_neg()
    with pytest.raises(ValueError):
        B.arLayerNorm([z], [x])
    with pytest.raises(ValueError, match="workspace"):
        B.arLayerNormBackward([x], [x], [x[:, 0].contiguous()], [x[:, 0].contiguous()], None, None,
                              [torch.zeros(8, device="cuda")], workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("rows,cols,wt", [(7, 300, torch.bfloat16), (700, 300, torch.bfloat16), (9, 20000, torch.float32)])
def test_two_streams_at_once(B, rows, cols, wt):
    """The same call on two streams side by side, each with a workspace of its own."""
    sets = [inputs([rows], cols, torch.bfloat16, wt, 60 + i) for i in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    held = []
    for xs, dys, gam, bet in sets:
        means = [(xs[0].double()).mean(1).float()]
        rstds = [torch.ones(rows)]
        held.append(dict(x=[dev(xs[0])], dy=[dev(dys[0])], g=[dev(gam[0])], m=[dev(means[0])], s=[dev(rstds[0])],
                         dx=[torch.empty_like(dev(xs[0]))], gg=[torch.empty(cols, dtype=wt, device="cuda")],
                         gb=[torch.empty(cols, dtype=wt, device="cuda")], host=(means, rstds)))
    torch.cuda.synchronize()
    for _ in range(5):
        for h, st in zip(held, streams):
            B.arLayerNormBackward(h["dy"], h["x"], h["m"], h["s"], h["g"], h["dx"], h["gg"], h["gb"], stream=st)
    torch.cuda.synchronize()
    for h, (xs, dys, gam, bet) in zip(held, sets):
        check_backward(dys, xs, gam, h["dx"], h["gg"], h["gb"], *h["host"])


def test_streams_given_as_handles(B):
    """A stream object, its raw handle, the default stream as 0, and none: torch's current stream."""
    xs, dys, gam, bet = inputs([700, 9], 600, torch.float32, torch.float32, 71)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, 0, None):
        check_forward(xs, gam, bet, 1e-5, *run_forward(B, xs, gam, bet, 1e-5, stream=stream))
        check_backward(dys, xs, gam, *run_backward(B, dys, xs, gam, 1e-5, stream=stream))
    with torch.cuda.stream(side):
        check_backward(dys, xs, gam, *run_backward(B, dys, xs, gam, 1e-5))


@pytest.mark.parametrize("rows,cols,dt", [([40000], 64, torch.bfloat16), ([30000, 12345], 264, torch.bfloat16),
                                          ([20011], 1032, torch.float32), ([7000, 3, 6500], 2056, torch.float16),
                                          ([9001], 4104, torch.bfloat16)], ids=str)
def test_several_rounds_of_workgroups(B, rows, cols, dt):
    """Row counts past what the GPU holds at once, with a part round at the end: every row of every rank, checked on
    the device against a 64-bit form (bounds as elsewhere)."""
    g = torch.Generator(device="cuda").manual_seed(cols)
    xs = [torch.randn(k, cols, generator=g, device="cuda").to(dt) for k in rows]
    gam = [torch.randn(cols, generator=g, device="cuda") for _ in rows]
    bet = [torch.randn(cols, generator=g, device="cuda") for _ in rows]
    ys = [torch.full_like(x, float("nan")) for x in xs]
    m, s = [torch.full((k,), float("nan"), device="cuda") for k in rows], [torch.full((k,), float("nan"), device="cuda") for k in rows]
    B.arLayerNorm(xs, ys, gam, bet, m, s)
    for r, x in enumerate(xs):
        for i in range(0, len(x), 4096):
            part = slice(i, i + 4096)
            want = ou.ln_forward(x[part].cpu(), gam[r].cpu(), bet[r].cpu(), 1e-5)
            ou.within(ys[r][part], want[0], want[3], dt, "y of rank %d from row %d" % (r, i))
            ou.within(m[r][part], want[1], want[4], torch.float32, "mean")
            ou.within(s[r][part], want[2], want[5], torch.float32, "rstd")


@pytest.mark.parametrize("rows", [[520, 0, 30], [40] * 18], ids=["3 ranks", "18 ranks"])
@pytest.mark.parametrize("cols,dt", [(5, torch.bfloat16), (16388, torch.bfloat16), (16391, torch.float32)], ids=str)
def test_rows_that_registers_do_not_hold(B, rows, cols, dt):
    """More than 512 rows of such widths, in one launch of ranks and in two, beside x and dy and over them."""
    xs, dys, gam, _ = inputs(rows, cols, dt, torch.float32, 90 + cols)
    for into in (None, "dy", "x"):
        check_backward(dys, xs, gam, *run_backward(B, dys, xs, gam, 1e-5, pad=3, into=into))
    check_backward(dys, xs, gam, *run_backward(B, dys, xs, gam, 1e-5, dx=False))
    check_backward(dys, xs, gam, *run_backward(B, dys, xs, gam, 1e-5, dg=False, db=False))
