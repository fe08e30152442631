"""The operators around the AllReduce at the ends of the ranges their documentation gives."""
import op_util as ou
import pytest
import test_gpu_layernorm as ln
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


@pytest.mark.parametrize("rows", [4, 520], ids=["few rows", "many rows"])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=str)
def test_sums_of_wide_rows(B, dt, rows, monkeypatch):
    """Rows of 2^22 columns (of 2^16 where there are many), of one value and not: a thread's thousands of additions
    cost no more than few.  A vector's own up to 8 additions, then one, 6 steps inside a wavefront and 16 to join
    them: 40 covers the chain, whatever the row's width."""
    cols = (1 << 22) + 3 if rows == 4 else (1 << 16) + 3
    monkeypatch.setattr(ou, "chain", lambda n: 40)
    g = torch.Generator().manual_seed(rows)
    x = ou.rows_of(g, (4, cols), dt, 1.0, 1000.0)
    x[0], x[2] = 1000.1, 0.1
    dy = ou.rows_of(g, (4, cols), dt)
    dy[0], dy[1] = 0.1, 0.3
    ys, m, s = ln.run_forward(B, [x], None, None, 1e-5)
    ln.check_forward([x], None, None, 1e-5, ys, m, s)
    rest = rows - 4      # rows like the second add to the count, not to the checking
    out = torch.empty(rows, cols, dtype=dt, device="cuda")
    X = torch.cat([x, x[1:2].expand(rest, cols)]).cuda()
    D = torch.cat([dy, dy[1:2].expand(rest, cols)]).cuda()
    means = x.double().mean(1).float()
    rstds = torch.full((4,), 0.5)
    M, R = (torch.cat([t, t[1:2].expand(rest)]).cuda() for t in (means, rstds))
    B.arLayerNormBackward([D], [X], [M], [R], None, [out], [torch.empty(cols, dtype=dt, device="cuda")])
    want, bound, _, _ = ou.ln_backward(dy, x, means, rstds, None)
    ou.within(out[:4], want, bound, dt, "dx")
    assert all(torch.equal(out[i], out[1]) for i in range(4, rows))


@pytest.mark.parametrize("rows", [2, 3])
def test_row_strides_past_32_bits(B, rows):
    """bf16 rows 2^32 + 8 elements apart."""
    cols, stride = 777, (1 << 32) + 8
    xs, dys, gam, bet = ln.inputs([rows], cols, torch.bfloat16, torch.float32, rows)
    X, D, Y = (torch.empty((rows - 1) * stride + cols, dtype=torch.bfloat16, device="cuda")
               .as_strided((rows, cols), (stride, 1)) for _ in range(3))
    X.copy_(xs[0])
    D.copy_(dys[0])
    m, s = [torch.empty(rows, device="cuda")], [torch.empty(rows, device="cuda")]
    B.arLayerNorm([X], [Y], [gam[0].cuda()], [bet[0].cuda()], m, s)
    torch.cuda.synchronize()
    ln.check_forward(xs, gam, bet, 1e-5, [Y.contiguous()], m, s)
    gg, gb = [torch.empty(cols, device="cuda")], [torch.empty(cols, device="cuda")]
    B.arLayerNormBackward([D], [X], m, s, [gam[0].cuda()], [Y], gg, gb)
    torch.cuda.synchronize()
    ln.check_backward(dys, xs, gam, [Y.contiguous()], gg, gb, [m[0].cpu()], [s[0].cpu()])
    B.arLayerNormBackward([D], [X], m, s, [gam[0].cuda()], [D], gg, gb)
    torch.cuda.synchronize()
    ln.check_backward(dys, xs, gam, [D.contiguous()], gg, gb, [m[0].cpu()], [s[0].cpu()])
