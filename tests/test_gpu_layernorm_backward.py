"""Layer norm backward over more than 512 rows, where each width has a kernel layout of its own (fewer rows take one
kernel for all widths): every layout, against the formulas in 64 bits with the bounds of op_util."""
import op_util as ou
import pytest
import test_gpu_layernorm as ln
import torch

pytestmark = pytest.mark.gpu

# one width of each layout: vectors of a row up to 16, 32, 64, 128, 256, 512, 1024, 2048, 3072, 4096, past them, and
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
