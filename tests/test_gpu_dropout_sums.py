"""The bias gradient of dropout over many rows, exactly: whole numbers up to 8 and a scale of 2 make every sum of
fewer than 2^20 rows exact in 32 bits, so that one row, line or slice left out or counted twice shows, however many
there are."""
import device_util as du
import pytest
import torch

pytestmark = pytest.mark.gpu

SEED, OFFSET = 0x0123456789ABCDEF, 5


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


def check(B, rows, cols, dt, wt=torch.float32, pad=0, offs=0):
    assert 16 * sum(rows) < 1 << 24
    g = torch.Generator(device="cuda").manual_seed(cols + len(rows))
    dys = [torch.randint(-8, 9, (k, cols), generator=g, device="cuda").to(dt) for k in rows]
    dxs = [torch.where(k, 2.0 * d, 0.0).to(dt) for k, d in zip(du.masks(rows, cols, 0.5, SEED, OFFSET, "cuda"), dys)]
    dbias = sum(d.double().sum(0) for d in dxs).to(wt)
    dy = [du.padded(t, pad, offs) for t in dys]
    for dx in ([torch.full_like(t, float("nan")) for t in dys], None, dy):
        db = [torch.full((cols,), float("nan"), dtype=wt, device="cuda") for _ in rows]
        B.arDropoutAddBackward(dy, dx, 0.5, SEED, OFFSET, None, db)
        assert all(torch.equal(b, dbias) for b in db)
        assert dx is None or all(torch.equal(a, b) for a, b in zip(dx, dxs))


COLS = [1, 3, 8, 9, 40, 64, 100, 256, 264, 515, 576, 768, 1032, 1368, 1600, 2041, 2048, 2056, 5000, 8191, 12119, 16391]


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("cols", COLS)
def test_many_rows(B, cols, dt):
    most = min(300000, 8000000 // cols)
    check(B, [most // 2 + 1, 3, 0, most // 3], cols, dt)
    check(B, [most // 2 + 1, 3, 0, most // 3], cols, dt, pad=3, offs=1)


@pytest.mark.parametrize("cols", COLS)
def test_one_more_row_than_a_step(B, cols):
    """Row counts around those where a slice, a step of a workgroup, or the few rows of one launch end."""
    for rows in (1, 2, 31, 33, 255, 256, 257, 511, 513, 1025):
        check(B, [rows], cols, torch.float16, torch.float16)


@pytest.mark.parametrize("ranks", [2, 16, 17, 32, 33, 128])
@pytest.mark.parametrize("cols", [7, 130, 1032, 4096])
def test_rows_of_many_ranks(B, cols, ranks):
    check(B, [(37 * r) % 61 for r in range(ranks)], cols, torch.bfloat16)
    check(B, [1 + 400 * (r % 3) for r in range(ranks)], cols, torch.bfloat16)
