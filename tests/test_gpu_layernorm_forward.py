"""Layer norm forward: every layout at its edges, and rows whose mean has to come out to the last bit."""
import op_util as ou
import pytest
import test_gpu_layernorm as ln
import torch

pytestmark = pytest.mark.gpu

# one width of each layout (16 x 1 up to 1024 x 4 vectors), where the product of the exact sum with a rounded
# 1 / cols misses the mean of some of VALUES; less than a vector; past registers
COLS = {torch.float32: [3, 61, 121, 237, 503, 751, 953, 2023, 2973, 4071, 6133, 8165, 12237, 16339, 16999],
        torch.bfloat16: [7, 61, 237, 503, 953, 1531, 2023, 4071, 6133, 8165, 12237, 16339, 24557, 32747, 33383]}
VALUES = [1.0, 5.0, 1000.0, -3.0, 0.0]


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


@pytest.mark.parametrize("dt,cols", [(t, c) for t in COLS for c in COLS[t]], ids=str)
def test_rows_of_one_value(B, dt, cols):
    """Every partial sum is a value of at most 7 bits times a number up to 33383, which 24 bits hold: the mean is the
    value, the variance 0, y beta."""
    x = torch.tensor(VALUES).to(dt)[:, None].expand(len(VALUES), cols).contiguous()
    g = torch.Generator().manual_seed(cols)
    gam, bet = [ou.rows_of(g, (cols,), torch.float32, 0.3, 1.0)], [ou.rows_of(g, (cols,), torch.float32)]
    ys, m, s = ln.run_forward(B, [x], gam, bet, 1e-5)
    assert torch.equal(m[0].cpu(), torch.tensor(VALUES))
    assert torch.equal(ys[0].cpu(), bet[0].to(dt).expand(len(VALUES), cols))
    ou.within(s[0], torch.full((len(VALUES),), 1e-5, dtype=torch.float64).rsqrt(), 1e-5 ** -0.5 * 4 * ou.U,
              torch.float32, "rstd")


def edges(dt):
    """The least and the largest width of each layout; rows of less than a vector, and past registers."""
    v = 4 if dt == torch.float32 else 8
    tops = [16, 32, 64, 128, 192, 256, 512, 768, 1024, 1536, 2048, 3 * 1024, 4096]
    return [1, v - 1, v] + [w for lo, hi in zip([0] + tops, tops) for w in (lo * v + 1, hi * v) if w > v] + [4096 * v + 1]


@pytest.mark.parametrize("dt,wt,cols", [(d, w, c) for d, w in ou.TYPES for c in edges(d)], ids=str)
def test_every_layout_and_its_edges(B, dt, wt, cols):
    """Dense rows, padded ones at odd addresses over themselves, and without weights or statistics."""
    xs, _, gam, bet = ln.inputs([9, 0, 4], cols, dt, wt, cols)
    ln.check_forward(xs, gam, bet, 1e-5, *ln.run_forward(B, xs, gam, bet, 1e-5))
    ln.check_forward(xs, gam, bet, 1e-5, *ln.run_forward(B, xs, gam, bet, 1e-5, 3, 1, inplace=True))
    ln.check_forward(xs, None, None, 1e-5, *ln.run_forward(B, xs, None, None, 1e-5, stats=False))


@pytest.mark.parametrize("dt,cols", [(t, c) for t in COLS for c in COLS[t]], ids=str)
def test_range_of_the_statistics(B, dt, cols):
    """eps 0: rows of tiny and of large spread as any others; past the range, what the header says."""
    g = torch.Generator().manual_seed(cols)
    gam, bet = [ou.rows_of(g, (cols,), torch.float32, 0.3, 1.0)], [ou.rows_of(g, (cols,), torch.float32)]
    for size in (1e-18, 1e16):
        x = [ou.rows_of(g, (3, cols), dt, size, size)]
        ln.check_forward(x, gam, bet, 0.0, *ln.run_forward(B, x, gam, bet, 0.0))
    x = ou.rows_of(g, (3, cols), dt)
    x[0] = 3e38                                   # the sum overflows
    x[1] = torch.tensor([1e20, -1e20]).repeat(cols)[:cols].to(dt)   # the squares alone do
    ys, m, s = ln.run_forward(B, [x], gam, bet, 1e-5)
    assert not torch.isfinite(m[0][0]) and not torch.isfinite(ys[0][0].float()).any()
    assert torch.isfinite(m[0][1]) and s[0][1] == 0 and torch.equal(ys[0][1].cpu(), bet[0].to(dt))
    ln.check_forward([x[2:]], gam, bet, 1e-5, [ys[0][2:]], [m[0][2:]], [s[0][2:]])
