"""The operators around the AllReduce at the ends of the ranges their documentation gives."""
import op_util as ou
import pytest
import torch

pytestmark = pytest.mark.gpu


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
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("cols,inplace", [((1 << 29) + 5, False), ((1 << 28) + 3, True)], ids=["2^29+5", "2^28+3 in place"])
def test_backward_of_the_widest_rows(B, cols, inplace):
    """One row whose weights' gradients take 2^32 threads at one column group a workgroup.  x is 0 or 1, mean 0,
    rstd 1 and dy a small whole number: dgamma and dbeta are exact, and so are the row's two sums, since no partial
    sum of their random signs comes near 2^24.  dx takes a division of each sum, two products and two differences:
    six roundings of values below 8 + 1 + 1."""
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.randint(0, 2, (1, cols), generator=g, device="cuda", dtype=torch.int8).float()
    dy = torch.randint(-8, 9, (1, cols), generator=g, device="cuda", dtype=torch.int8).float()
    keep = x.clone() if inplace else x
    dx = x if inplace else torch.full_like(x, float("nan"))
    gg, gb = torch.full((cols,), float("nan"), device="cuda"), torch.full((cols,), float("nan"), device="cuda")
    zero, one = torch.zeros(1, device="cuda"), torch.ones(1, device="cuda")
    B.arLayerNormBackward([dy], [x], [zero], [one], None, [dx], [gg], [gb])
    torch.cuda.synchronize()
    s = t = 0.0
    for a, b in zip(dy[0].split(1 << 26), keep[0].split(1 << 26)):
        s += a.sum(dtype=torch.float64).item() / cols
        t += (a * b).sum(dtype=torch.float64).item() / cols
    assert torch.equal(gb, dy[0])
    assert torch.equal(gg, dy[0] * keep[0])
    for got, a, b in zip(dx[0].split(1 << 26), dy[0].split(1 << 26), keep[0].split(1 << 26)):
        assert (got.double() - (a.double() - s - b.double() * t)).abs().max().item() <= 6 * 10 * ou.U
