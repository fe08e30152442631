"""Layer norm backward over more than 512 rows, where each width has a kernel layout of its own (fewer rows take one
kernel for all widths): every layout, against the formulas in 64 bits with the bounds of op_util."""
import op_util as ou
import pytest
import test_gpu_layernorm as ln
import torch

pytestmark = pytest.mark.gpu

# one width of each layout: vectors of a row up to 16, 32, 64, 128, 256, 512, 1 to 4 times 1024, past them, and
# less than one vector (16-bit rows: 8 columns a vector, of which registers hold 2048)
COLS = {torch.float32: [3, 40, 100, 200, 500, 1000, 2000, 4000, 6000, 10000, 14000, 17000],
        torch.bfloat16: [7, 90, 200, 500, 1000, 2000, 4000, 8000, 12000, 17000]}


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


@pytest.mark.parametrize("size,grad", [(1e-20, 0.1), (1e25, 1e20), (1e-18, 1e-25)])
@pytest.mark.parametrize("dt,cols", [(t, c) for t in COLS for c in COLS[t]], ids=str)
def test_rows_of_extreme_spread(B, dt, cols, size, grad):
    """eps 0 and rows whose rstd^2, or dy (x - mean), passes the ends of a float though h, q and their sums do not."""
    for rows in ([9], [520, 0, 3]):
        g = torch.Generator().manual_seed(cols)
        xs = [ou.rows_of(g, (k, cols), dt, size, size) for k in rows]
        dys = [ou.rows_of(g, (k, cols), dt, grad) for k in rows]
        gam = [ou.rows_of(g, (cols,), torch.float32, 0.3, 1.0) for _ in rows]
        ln.check_backward(dys, xs, gam, *ln.run_backward(B, dys, xs, gam, 0.0))


def edges(dt):
    """The least and the largest width of each layout; rows of less than a vector, and past registers."""
    v, last = (4, 4096) if dt == torch.float32 else (8, 2048)
    tops = [t for t in (16, 32, 64, 128, 256, 512, 1024, 2048, 3 * 1024, 4096) if t <= last]
    return [1, v - 1, v] + [w for lo, hi in zip([0] + tops, tops) for w in (lo * v + 1, hi * v) if w > v] + [last * v + 1]


@pytest.mark.parametrize("dt,wt,cols", [(d, w, c) for d, w in ou.TYPES for c in edges(d)], ids=str)
def test_every_layout_and_its_edges(B, dt, wt, cols):
    xs, dys, gam, _ = ln.inputs([514, 0, 3], cols, dt, wt, cols)
    ln.check_backward(dys, xs, gam, *ln.run_backward(B, dys, xs, gam, 1e-5))


@pytest.mark.parametrize("dt,cols", [(t, c) for t in COLS for c in COLS[t]], ids=str)
def test_every_layout_over_many_ranks(B, dt, cols):
    """18 ranks of few rows, which take two launches: padded rows at odd addresses, with and without weights, in place,
    and in parts."""
    rows = [2, 0, 1] * 6
    for wt in (dt, torch.float32):
        xs, dys, gam, _ = ln.inputs(rows, cols, dt, wt, cols + 5)
        for pad, offset, into in ((3, 1, None), (0, 3, "dy"), (8, 0, "x")):
            ln.check_backward(dys, xs, gam, *ln.run_backward(B, dys, xs, gam, 1e-5, pad, offset, into=into))
        for parts in (dict(dg=False, db=False), dict(dx=False, db=False), dict(dx=False, dg=False), dict(db=False)):
            ln.check_backward(dys, xs, gam, *ln.run_backward(B, dys, xs, gam, 1e-5, **parts))
    ln.check_backward(dys, xs, None, *ln.run_backward(B, dys, xs, None, 1e-5))


@pytest.mark.parametrize("dt,cols", [(t, c) for t in COLS for c in COLS[t]], ids=str)
def test_nan_and_infinity_stay_in_their_row(B, dt, cols):
    """One dy of a row NaN, one x of another infinite, at the row's end, which the last vector and the one before may
    both read: dx of those rows alone, and of dgamma and dbeta the columns they reach."""
    rows = [2, 0, 3] + [1] * 15
    xs, dys, gam, _ = ln.inputs(rows, cols, dt, torch.float32, cols + 7)
    _, _, _, means, rstds = ln.run_backward(B, dys, xs, gam, 1e-5)
    dys[2][1, cols - 1] = float("nan")
    xs[5][0, cols - 1] = float("inf")
    out = [torch.empty(x.shape, dtype=dt, device="cuda") for x in xs]
    gg, gb = [torch.empty(cols, device="cuda") for _ in xs], [torch.empty(cols, device="cuda") for _ in xs]
    B.arLayerNormBackward([t.cuda() for t in dys], [t.cuda() for t in xs], [t.cuda() for t in means],
                          [t.cuda() for t in rstds], [t.cuda() for t in gam], out, gg, gb)
    for r, k in enumerate(rows):
        for i in range(k):
            row = out[r][i].float().cpu()
            if (r, i) in ((2, 1), (5, 0)):
                assert not torch.isfinite(row).any()
            else:
                assert torch.isfinite(row).all()
    assert torch.isnan(out[2][1].float()).all()
    for t in gg + gb:
        assert torch.isnan(t[cols - 1]) and torch.isfinite(t[:cols - 1]).all()
