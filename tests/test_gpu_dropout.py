"""Dropout with bias and residual over the ranks' rows and its gradients, against the formulas in 64 bits with a
plain generator (step_util), and against differences of the forward pass."""
import op_util as ou
import pytest
import step_util as su
import torch
from test_gpu_layernorm import dev, untouched

pytestmark = pytest.mark.gpu

COLS = [1, 2, 7, 8, 9, 64, 65, 127, 255, 1000, 1024, 2047, 2048, 4097, 8192, 10000, 16391, 40000]
SEED, OFFSET = 0x9ABCDEF012345678, 0x1122334455667788


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


def inputs(rows, cols, dt, wt, seed):
    g = torch.Generator().manual_seed(seed)
    xs = [ou.rows_of(g, (k, cols), dt, 0.5 + r % 3, (r % 3) - 1.0) for r, k in enumerate(rows)]
    zs = [ou.rows_of(g, (k, cols), dt, 2.0) for k in rows]
    bias = ou.rows_of(g, (cols,), wt, 0.3)
    return xs, zs, [bias.clone() for _ in rows]


def firsts(rows, first=None):
    return list(first) if first is not None else [sum(rows[:r]) for r in range(len(rows))]


def masks(rows, cols, p, seed, offset, first=None):
    return [su.drawn(k, f, cols, seed, offset) >= su.threshold(p) for k, f in zip(rows, firsts(rows, first))]


def nans(t):
    return torch.full_like(t, float("nan"))


def run_forward(B, xs, zs, bs, p, seed=SEED, offset=OFFSET, step=None, first=None, pad=0, offs=0, into=None, stream=None):
    x, z = [dev(t, pad, offs) for t in xs], None if zs is None else [dev(t, pad + 2, offs) for t in zs]
    y = {"x": x, "z": z}.get(into) or [dev(nans(t), pad + 5, offs) for t in xs]
    b = None if bs is None else [dev(t, 0, offs) for t in bs]
    torch.cuda.synchronize()
    B.arDropoutAdd(x, y, p, seed, offset, step, b, z, first, stream=stream)
    torch.cuda.synchronize()
    return y


def check_forward(ys, xs, zs, bs, kept, p):
    for r, y in enumerate(ys):
        want, bound = su.dropout(xs[r], bs[r] if bs is not None else None, zs[r] if zs is not None else None, kept[r], p)
        ou.within(y, want, bound, xs[r].dtype, "y of rank %d" % r)
        assert untouched(y)


def run_backward(B, dys, wt, p, seed=SEED, offset=OFFSET, step=None, first=None, pad=0, offs=0, dx=True, dbias=True,
                 inplace=False, stream=None, workspace=None):
    d = [dev(t, pad, offs) for t in dys]
    out = None
    if dx:
        out = d if inplace else [dev(nans(t), pad + 5, offs) for t in dys]
    gb = [torch.full((dys[0].shape[1],), float("nan"), dtype=wt, device="cuda") for _ in dys] if dbias else None
    torch.cuda.synchronize()
    B.arDropoutAddBackward(d, out, p, seed, offset, step, gb, first, workspace=workspace, stream=stream)
    torch.cuda.synchronize()
    return out, gb


def check_backward(out, gb, dys, kept, p):
    s = su.scale_of(p)
    dxs = [torch.where(k, d.double() * s, 0.0) for k, d in zip(kept, dys)]
    if out is not None:
        for r, t in enumerate(out):
            ou.within(t, dxs[r], 2.01 * ou.U * dxs[r].abs(), dys[r].dtype, "dx of rank %d" % r)
            assert untouched(t)
    if gb is not None:
        want, size = sum(d.sum(0) for d in dxs), sum(d.abs().sum(0) for d in dxs)
        for t in gb:   # any order of the rows' additions, then the scale
            ou.within(t, want, (sum(len(d) for d in dys) + 4) * ou.U * size, t.dtype, "dbias")


@pytest.mark.parametrize("dt,wt", ou.TYPES, ids=str)
@pytest.mark.parametrize("cols", COLS)
def test_forward(B, cols, dt, wt):
    rows = [5, 0, 3] if cols > 3000 else [37, 0, 18, 1]
    xs, zs, bs = inputs(rows, cols, dt, wt, cols)
    check_forward(run_forward(B, xs, zs, bs, 0.3), xs, zs, bs, masks(rows, cols, 0.3, SEED, OFFSET), 0.3)


@pytest.mark.parametrize("dt,wt", ou.TYPES, ids=str)
@pytest.mark.parametrize("cols", COLS)
def test_backward(B, cols, dt, wt):
    rows = [5, 0, 3] if cols > 3000 else [37, 0, 18, 1]
    dys, _, _ = inputs(rows, cols, dt, wt, cols + 1)
    check_backward(*run_backward(B, dys, wt, 0.3), dys, masks(rows, cols, 0.3, SEED, OFFSET), 0.3)


@pytest.mark.parametrize("cols", [3, 64, 770, 2049, 9000])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=str)
def test_many_rows(B, cols, dt):
    """More rows than one round of workgroups takes, ragged, with sums over all of them."""
    most = 6000000 // cols
    rows = [min(most, 30000) // 2 + 1, 3, 0, min(most, 30000) // 3]
    dys, zs, bs = inputs(rows, cols, dt, torch.float32, cols + 2)
    kept = masks(rows, cols, 0.1, SEED, OFFSET)
    check_backward(*run_backward(B, dys, torch.float32, 0.1), dys, kept, 0.1)
    check_forward(run_forward(B, dys, zs, bs, 0.1), dys, zs, bs, kept, 0.1)


# workgroups that follow each other through the rows, one tile of all columns, tiles of whole lines, even tiles
@pytest.mark.parametrize("cols", [40, 264, 515, 576, 768, 1032, 1368, 1600, 2041, 2056, 5000, 8191])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=str)
def test_ways_to_cut_rows(B, cols, dt):
    """Enough rows for each way to cut them; padded to odd strides, eight slices' tiles lie on one XCD, but for the
    last slices."""
    most = 2000000 // cols
    rows = [most // 2 + 1, 3, 0, most // 3]
    dys, zs, bs = inputs(rows, cols, dt, torch.float32, cols + 4)
    kept = masks(rows, cols, 0.1, SEED, OFFSET)
    for pad, offs in ((0, 0), (3, 1)):
        check_backward(*run_backward(B, dys, torch.float32, 0.1, pad=pad, offs=offs), dys, kept, 0.1)
        check_forward(run_forward(B, dys, zs, bs, 0.1, pad=pad, offs=offs), dys, zs, bs, kept, 0.1)


@pytest.mark.parametrize("into", [None, "x", "z"])
@pytest.mark.parametrize("cols", [3, 64, 770, 2049])
@pytest.mark.parametrize("dt", [torch.float32, torch.float16], ids=str)
def test_padded_rows_odd_addresses_in_place(B, cols, dt, into):
    rows, first = [4, 9], [7, 7]
    xs, zs, bs = inputs(rows, cols, dt, dt, cols + 3)
    kept = masks(rows, cols, 0.5, SEED, OFFSET, first)
    for pad, offs in ((0, 1), (3, 0), (8, 5)):
        check_forward(run_forward(B, xs, zs, bs, 0.5, first=first, pad=pad, offs=offs, into=into), xs, zs, bs, kept, 0.5)
        check_backward(*run_backward(B, xs, dt, 0.5, first=first, pad=pad, offs=offs, inplace=into == "x"), xs, kept, 0.5)


@pytest.mark.parametrize("p", [0.0, 1.0, 2.0 ** -18, 2.0 ** -17, 1 - 2.0 ** -18, 0.99999, 0.5])
def test_probabilities(B, p):
    """The ends of the range: T of 0, 1, 65535 and 65536."""
    rows, cols = [40, 5], 1030
    xs, zs, bs = inputs(rows, cols, torch.float32, torch.float32, 5)
    kept = masks(rows, cols, p, SEED, OFFSET)
    check_forward(run_forward(B, xs, zs, bs, p), xs, zs, bs, kept, p)
    check_forward(run_forward(B, xs, None, None, p), xs, None, None, kept, p)
    check_backward(*run_backward(B, xs, torch.float32, p), xs, kept, p)
    if p == 1.0:
        assert not any(k.any() for k in kept)


def test_dropped_values_do_not_matter(B):
    """NaN and infinity in dropped places leave no trace; in kept ones they stay."""
    rows, cols, p = [33], 515, 0.4
    xs, zs, bs = inputs(rows, cols, torch.bfloat16, torch.bfloat16, 6)
    kept = masks(rows, cols, p, SEED, OFFSET)[0]
    xs[0][~kept] = float("nan")
    ys = run_forward(B, xs, zs, bs, p)
    assert torch.isfinite(ys[0]).all()
    check_forward(ys, xs, zs, bs, [kept], p)
    out, gb = run_backward(B, xs, torch.bfloat16, p)
    assert torch.isfinite(out[0]).all() and torch.isfinite(gb[0]).all()
    xs[0][3, 4:9] = float("inf")
    check_forward(run_forward(B, xs, zs, bs, p), xs, zs, bs, [kept], p)


def test_replicas_draw_alike_and_ranks_do_not(B):
    rows, cols, p = [64, 64], 768, 0.5
    ones = [torch.ones(64, cols) for _ in rows]
    same = run_forward(B, ones, None, None, p, first=[100, 100])
    assert torch.equal(same[0], same[1])
    apart = run_forward(B, ones, None, None, p)
    assert not torch.equal(apart[0], apart[1])
    # however the rows are shared out, over one rank, two or seventeen
    whole = run_forward(B, [torch.ones(128, cols)], None, None, p)[0]
    assert torch.equal(torch.cat(list(apart)), whole)
    many = run_forward(B, [torch.ones(8, cols) for _ in range(16)], None, None, p)
    assert torch.equal(torch.cat(list(many)), whole)
    assert torch.equal(run_forward(B, [torch.ones(128, cols, dtype=torch.float16)], None, None, p)[0].float(), whole)


@pytest.mark.parametrize("n", [17, 32, 33, 40, 128])
def test_many_ranks(B, n):
    rows, cols = [3 * r % 5 for r in range(n)], 130
    xs, zs, bs = inputs(rows, cols, torch.bfloat16, torch.float32, n)
    kept = masks(rows, cols, 0.2, SEED, OFFSET)
    check_forward(run_forward(B, xs, zs, bs, 0.2), xs, zs, bs, kept, 0.2)
    check_backward(*run_backward(B, xs, torch.float32, 0.2), xs, kept, 0.2)


def test_no_rows(B):
    xs = [torch.zeros(0, 20) for _ in range(3)]
    run_forward(B, xs, xs, None, 0.5)
    _, gb = run_backward(B, xs, torch.float32, 0.5)
    assert all((t == 0).all() for t in gb)


@pytest.mark.parametrize("seed,offset,step", [(0, 0, 0), ((1 << 64) - 1, (1 << 64) - 2, 5), (1 << 32, 1 << 32, (1 << 63) - 1),
                                              (1, 7, -3)], ids=str)
def test_seeds_offsets_steps_and_far_rows(B, seed, offset, step):
    """Words past 32 bits, offsets that wrap at 64, rows up to the last of 2^32."""
    rows, cols, p = [6, 2], 100, 0.25
    first = [(1 << 32) - 6, (1 << 31) - 1]
    xs, zs, bs = inputs(rows, cols, torch.float32, torch.float32, 8)
    kept = masks(rows, cols, p, seed, offset + step, first)
    s = torch.tensor([step], device="cuda")
    check_forward(run_forward(B, xs, zs, bs, p, seed, offset, s, first), xs, zs, bs, kept, p)
    check_backward(*run_backward(B, xs, torch.float32, p, seed, offset, s, first), xs, kept, p)


def test_shares_kept_and_independence(B):
    """4 million draws: the share that stays is within five deviations of 1 - p, and two layers, seeds, steps, rows
    or columns agree as often as independent ones."""
    rows, cols, p = 2000, 2048, 0.25
    ones = [torch.ones(rows, cols)]
    base = run_forward(B, ones, None, None, p)[0] != 0
    n = rows * cols
    assert abs(base.double().mean().item() - 0.75) < 5 * (p * 0.75 / n) ** 0.5
    others = [run_forward(B, ones, None, None, p, seed=SEED + 1)[0] != 0, run_forward(B, ones, None, None, p, offset=OFFSET + 1)[0] != 0,
              run_forward(B, ones, None, None, p, first=[rows])[0] != 0, base.roll(1, 0), base.roll(1, 1), base.roll(8, 1)]
    both = 0.75 * 0.75
    for o in others:
        assert abs((base & o).double().mean().item() - both) < 5 * (both * (1 - both) / n) ** 0.5


@pytest.mark.parametrize("kw", [dict(dx=False), dict(dbias=False)], ids=str)
@pytest.mark.parametrize("rows", [[300, 20], [30, 4]], ids=str)
def test_one_gradient_alone(B, rows, kw):
    cols = 1234
    dys, _, _ = inputs(rows, cols, torch.bfloat16, torch.bfloat16, 9)
    check_backward(*run_backward(B, dys, torch.bfloat16, 0.1, **kw), dys, masks(rows, cols, 0.1, SEED, OFFSET), 0.1)


def test_gradients_against_differences(B):
    """y is linear in x and the bias: differences are exact up to rounding."""
    rows, cols, p = [6, 3], 50, 0.3
    xs, zs, bs = inputs(rows, cols, torch.float32, torch.float32, 10)
    g = torch.Generator().manual_seed(3)
    dys = [torch.randn(k, cols, generator=g) for k in rows]
    move = [torch.randn(k, cols, generator=g) for k in rows]
    turn = torch.randn(cols, generator=g)
    dx, db = run_backward(B, dys, torch.float32, p)

    def value(h):
        ys = run_forward(B, [x + h * m for x, m in zip(xs, move)], zs, [b + h * turn for b in bs], p)
        return sum((y.double().cpu() * d.double()).sum().item() for y, d in zip(ys, dys))

    slope = (value(1.0) - value(-1.0)) / 2.0
    want = sum((d.double().cpu() * m.double()).sum().item() for d, m in zip(dx, move)) + (db[0].double().cpu() * turn.double()).sum().item()
    size = sum((2 * d.double().abs() * (x.abs() + m.abs() + b.abs() + turn.abs() + z.abs() + 1)).sum().item()
               for d, x, m, b, z in zip(dys, xs, move, bs, zs))
    assert abs(slope - want) <= 20 * ou.U * size


def test_a_replayed_graph_draws_anew(B):
    """Forward and backward captured once, the step's number raised between replays, eager calls in between."""
    rows, cols, p = [700, 30], 520, 0.2
    xs, zs, bs = inputs(rows, cols, torch.bfloat16, torch.float32, 11)
    x, z, b = ([t.cuda() for t in ts] for ts in (xs, zs, bs))
    y, dx = [torch.empty_like(t) for t in x], [torch.empty_like(t) for t in x]
    db = [torch.empty(cols, device="cuda") for _ in x]
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    ws = torch.empty(B.arDropoutAddBackwardWorkspace(rows, cols), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.arDropoutAdd(x, y, p, SEED, OFFSET, step, b, z)
        B.arDropoutAddBackward(x, dx, p, SEED, OFFSET, step, db, workspace=ws)
    seen = []
    for i in range(4):
        step.fill_(3 * i)
        for t in y + dx + db:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        kept = masks(rows, cols, p, SEED, OFFSET + 3 * i)
        check_forward(y, xs, zs, bs, kept, p)
        check_backward(dx, db, xs, kept, p)
        seen.append(y[0].clone())
        eager = run_forward(B, xs, zs, bs, p, step=step)
        assert torch.equal(eager[0], y[0])
    assert not torch.equal(seen[0], seen[1])


def test_side_by_side_on_two_streams(B):
    rows, cols, p = [900], 1030, 0.1
    sets = []
    for i in range(2):
        dys, _, _ = inputs(rows, cols, torch.float16, torch.float32, 20 + i)
        sets.append((dys, [t.cuda() for t in dys], [torch.empty(rows[0], cols, dtype=torch.float16, device="cuda")],
                     [torch.empty(cols, device="cuda")], torch.cuda.Stream(),
                     torch.empty(B.arDropoutAddBackwardWorkspace(rows, cols), dtype=torch.uint8, device="cuda")))
    torch.cuda.synchronize()
    for _ in range(20):
        for i, (_, d, o, gb, st, ws) in enumerate(sets):
            B.arDropoutAddBackward(d, o, p, SEED + i, 0, None, gb, workspace=ws, stream=st)
    torch.cuda.synchronize()
    for i, (dys, _, o, gb, _, _) in enumerate(sets):
        check_backward(o, gb, dys, masks(rows, cols, p, SEED + i, 0), p)


def test_row_strides_past_32_bits(B):
    """Three rows 2^31 + 8 elements apart: the last one starts past 2^32 elements."""
    cols, stride, p = 33, (1 << 31) + 8, 0.3
    buf = torch.empty(2 * stride + cols, dtype=torch.bfloat16, device="cuda")
    view = buf.as_strided((3, cols), (stride, 1))
    x = torch.randn(3, cols).bfloat16()
    kept = masks([3], cols, p, SEED, OFFSET)
    view.copy_(x)
    B.arDropoutAdd([view], [view], p, SEED, OFFSET)
    torch.cuda.synchronize()
    check_forward([view.clone()], [x], None, None, kept, p)
    view.copy_(x)
    db = [torch.empty(cols, device="cuda")]
    B.arDropoutAddBackward([view], [view], p, SEED, OFFSET, None, db)
    torch.cuda.synchronize()
    check_backward([view.clone()], db, [x], kept, p)


def test_wide_rows(B):
    """A row of 2^24 + 3 columns; the sums of one row are the row."""
    cols, p = (1 << 24) + 3, 0.5
    x = torch.randn(1, cols, dtype=torch.float32)
    kept = masks([1], cols, p, SEED, OFFSET)
    check_forward(run_forward(B, [x], None, None, p), [x], None, None, kept, p)
    check_backward(*run_backward(B, [x], torch.float32, p), [x], kept, p)


@pytest.mark.parametrize("cols", [1 << 30, (1 << 26) + 5])
def test_the_widest_rows_of_several_ranks(B, cols):
    """Eight ranks' rows of 2^30 columns (more than 2^32 threads at 8 columns each), in place, and their sums; windows
    at the ends and across 2^29."""
    n, p, wide = 8, 0.5, 4096
    xs = [torch.full((1, cols), r + 1.0, dtype=torch.bfloat16, device="cuda") for r in range(n)]
    starts = [0, min(1 << 29, cols // 2 // 8 * 8), (cols - wide) // 8 * 8]
    B.arDropoutAdd(xs, xs, p, SEED, OFFSET)
    torch.cuda.synchronize()
    for r in range(n):
        for s in starts:
            kept = su.drawn(1, r, min(wide, cols - s), SEED, OFFSET, s) >= su.threshold(p)
            assert torch.equal(xs[r][:, s:s + wide].float().cpu(), torch.where(kept, 2.0 * (r + 1), 0.0)), (r, s)
    few = xs[:2] if cols > 1 << 28 else xs
    for x in xs:
        x.fill_(1.0)
    db = [torch.empty(cols, dtype=torch.bfloat16, device="cuda") for _ in few]
    B.arDropoutAddBackward(few, few, p, SEED, OFFSET, None, db)
    torch.cuda.synchronize()
    for s in starts:
        kept = [su.drawn(1, r, min(wide, cols - s), SEED, OFFSET, s) >= su.threshold(p) for r in range(len(few))]
        want = torch.cat(kept).float().mul(2.0)
        assert torch.equal(torch.cat([x[:, s:s + wide] for x in few]).float().cpu(), want)
        assert torch.equal(db[0][s:s + wide].float().cpu(), want.sum(0)) and torch.equal(db[-1][s:s + wide], db[0][s:s + wide])
