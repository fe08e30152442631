"""The global norm over a list of tensors and clipping by it, against 64-bit sums; and the step the operators
belong to: layer norm on every rank, its weights' gradients, AllReduce, norm, clip."""
import math

import op_util as ou
import pytest
import torch

pytestmark = pytest.mark.gpu

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


def grads(sizes, dtypes, seed, offset=0, std=1.0):
    """Host tensors and their device copies, `offset` elements into their allocations, NaN around them."""
    g = torch.Generator().manual_seed(seed)
    host, devs = [], []
    for i, n in enumerate(sizes):
        dt = dtypes[i % len(dtypes)]
        t = (torch.randn(n, generator=g) * std * 2.0 ** -(i % 7)).to(dt)
        buf = torch.full((offset + n + 9,), float("nan"), dtype=dt, device="cuda")
        buf[offset:offset + n].copy_(t)
        host.append(t)
        devs.append(buf[offset:offset + n])
    return host, devs


def norm_of(host, kind):
    if kind == "max":
        return max([0.0] + [t.double().abs().max().item() for t in host if t.numel()])
    return math.sqrt(sum([(t.double() ** 2).sum().item() for t in host]))


def check_norm(got, want):
    """Summed in 64 bits (off by 1e-12 at most here) and rounded to a float once."""
    assert abs(got.item() - want) <= want * (ou.U + 1e-12), (got.item(), want)


def check_clip(outs, host, norm, scale, bound, eps=1e-6):
    c = 1.0 if norm + eps <= bound else bound / (norm + eps)
    f = float(torch.tensor(scale * c, dtype=torch.float64).float())
    for i, (o, t) in enumerate(zip(outs, host)):
        want = t.double() * f
        # the factor may round the other way at a tie of its own (a whole step), and the product rounds twice
        ou.within(o, want, 3 * ou.U * want.abs(), t.dtype, "tensor %d" % i)


SIZES = [[1], [0, 5, 0], [7, 1, 1024, 3], [4096] * 3, [100003], [1 << 20, 17, 0, 300001], [33] * 700,
         [5000011, 1, 64, 64, 2000000] + [777] * 50]


@pytest.mark.parametrize("kind", ["2", "max"])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "%dx%d" % (len(s), sum(s)))
@pytest.mark.parametrize("dtypes", [[t] for t in DTYPES] + [DTYPES], ids=str)
def test_norm_and_clip(B, sizes, dtypes, kind):
    host, devs = grads(sizes, dtypes, len(sizes) + sum(sizes))
    want = 0.125 * norm_of(host, kind)
    norm = torch.full((1,), float("nan"), device="cuda")
    with B.TensorList(devs) as lst:
        B.arGradNorm(lst, norm, kind=kind, scale=-0.125)
        check_norm(norm, want)
        with pytest.raises(B.ArError):
            B.arGradClip(lst, norm, 1.0)    # a list without outputs
    for bound in (want * 0.5, want * 2 + 1.0):
        outs = [torch.full_like(t, float("nan")) for t in devs]
        norm.fill_(float("nan"))
        with B.TensorList(devs, outs) as lst:
            B.arGradClip(lst, norm, bound, kind=kind, scale=0.125)
            torch.cuda.synchronize()
        check_norm(norm, want)
        check_clip(outs, host, want, 0.125, bound)
        for t, h in zip(devs, host):
            assert torch.equal(t.cpu(), h)    # the gradients themselves stay


@pytest.mark.parametrize("offset", [1, 2, 3, 5])
@pytest.mark.parametrize("dt", DTYPES, ids=str)
def test_odd_addresses(B, dt, offset):
    """Tensors at odd elements, outputs at others, neighbours untouched."""
    sizes = [1, 15, 16, 17, 70001, 257]
    host, devs = grads(sizes, [dt], 3, offset)
    for oo in (0, 1, offset):
        bufs = [torch.full((n + oo + 8,), float("nan"), dtype=dt, device="cuda") for n in sizes]
        outs = [b[oo:oo + n] for b, n in zip(bufs, sizes)]
        norm = torch.empty(1, device="cuda")
        with B.TensorList(devs, outs) as lst:
            B.arGradClip(lst, norm, 0.5, scale=0.25)
            torch.cuda.synchronize()
        check_norm(norm, 0.25 * norm_of(host, "2"))
        check_clip(outs, host, 0.25 * norm_of(host, "2"), 0.25, 0.5)
        for b, n in zip(bufs, sizes):
            assert torch.isnan(b[:oo].float()).all() and torch.isnan(b[oo + n:].float()).all()


@pytest.mark.parametrize("bound", [0.0, 0.01, 1e9, math.inf])
def test_in_place(B, bound):
    """Clipped where they lie; below the bound with scale 1 every bit stays."""
    host, devs = grads([70001, 5, 300], DTYPES, 21)
    want = norm_of(host, "2")
    norm = torch.empty(1, device="cuda")
    with B.TensorList(devs, devs) as lst:
        B.arGradClip(lst, norm, bound)
        torch.cuda.synchronize()
    check_norm(norm, want)
    if bound > want:
        assert all(torch.equal(d.cpu(), h) for d, h in zip(devs, host))
    else:
        check_clip(devs, host, want, 1.0, bound)


def test_extreme_values(B):
    """Squares that overflow or vanish in 32 bits."""
    norm = torch.empty(1, device="cuda")
    for v in (3e30, 1e-30, 2.0 ** -149, 3.4e38):
        t = torch.full((1000,), v, device="cuda")
        with B.TensorList([t, t]) as lst:
            B.arGradNorm(lst, norm, scale=2.0 ** -6)
            check_norm(norm, math.sqrt(2000.0) * t[0].double().item() * 2.0 ** -6) if v != 2.0 ** -149 else None
            B.arGradNorm(lst, norm, kind="max")
            assert norm.item() == t[0].item()
    t = torch.full((5,), 2.0 ** -24, dtype=torch.float16, device="cuda")
    with B.TensorList([t]) as lst:
        B.arGradNorm(lst, norm)
        check_norm(norm, math.sqrt(5.0) * 2.0 ** -24)


@pytest.mark.parametrize("kind", ["2", "max"])
def test_nan_and_infinity(B, kind):
    for n, at in ((900, 0), (900000, 899999)):
        for v in (math.nan, math.inf, -math.inf):
            t = torch.ones(n, device="cuda")
            t[at] = v
            o = torch.zeros_like(t)
            norm = torch.empty(1, device="cuda")
            with B.TensorList([torch.ones(3, device="cuda"), t], [torch.zeros(3, device="cuda"), o]) as lst:
                B.arGradClip(lst, norm, 1.0, kind=kind)
                torch.cuda.synchronize()
            rest = torch.cat([o[:at], o[at + 1:]])
            if math.isnan(v):
                assert math.isnan(norm.item()) and torch.isnan(o).all()
            else:
                assert norm.item() == math.inf and math.isnan(o[at].item()) and (rest == 0).all()
            with B.TensorList([t]) as lst:
                B.arGradNorm(lst, norm, kind=kind)
                assert math.isnan(norm.item()) if math.isnan(v) else norm.item() == math.inf


def test_empty_lists(B):
    norm = torch.full((1,), 7.0, device="cuda")
    for ts in ([], [torch.empty(0, device="cuda")] * 3):
        with B.TensorList(ts, ts) as lst:
            B.arGradNorm(lst, norm)
            assert norm.item() == 0.0
            norm.fill_(7.0)
            B.arGradClip(lst, norm, 1.0)
            assert norm.item() == 0.0
            B.arGradClip(lst, None, 1.0)
            norm.fill_(7.0)


def test_a_tensor_listed_twice_counts_twice(B):
    t = torch.full((1000,), 2.0, device="cuda")
    norm = torch.empty(1, device="cuda")
    with B.TensorList([t, t]) as lst:
        B.arGradNorm(lst, norm)
        check_norm(norm, math.sqrt(2000 * 4.0))
    with pytest.raises(B.ArError):
        B.TensorList([t, t], [t, t])


def test_elements_past_32_bits(B):
    """A tensor of 2^32 + 77 elements, all zero but a few near its end."""
    n = (1 << 32) + 77
    t = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    t[n - 1] = 3.0
    t[1 << 31] = 4.0
    t[(1 << 32) + 1] = 12.0
    norm = torch.empty(1, device="cuda")
    with B.TensorList([t], [t]) as lst:
        B.arGradClip(lst, norm, 6.5, eps=0.0)
        torch.cuda.synchronize()
    assert norm.item() == 13.0
    assert t[n - 1].item() == 1.5 and t[1 << 31].item() == 2.0 and t[(1 << 32) + 1].item() == 6.0


def test_streams_graphs_and_workspaces(B):
    """Two graphs over two lists with workspaces of their own, replayed side by side on two streams, and an eager
    call between replays; every replay sees the gradients of its time."""
    runs = []
    for i, sizes in enumerate(([300, 70001, 5], [1 << 20, 99])):
        host, devs = grads(sizes, DTYPES, 30 + i)
        outs = [torch.empty_like(t) for t in devs]
        norm = torch.empty(1, device="cuda")
        lst = B.TensorList(devs, outs)
        st = torch.cuda.Stream()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            B.arGradClip(lst, norm, 0.75)
        runs.append((sizes, devs, outs, norm, lst, st, graph))
    for rep in range(3):
        hosts = []
        for i, (sizes, devs, outs, norm, lst, st, graph) in enumerate(runs):
            host, _ = grads(sizes, DTYPES, 40 + 10 * rep + i)
            for d, h in zip(devs, host):
                d.copy_(h)
            hosts.append(host)
        other = torch.empty(1, device="cuda")
        torch.cuda.synchronize()
        for r in runs:
            with torch.cuda.stream(r[5]):
                r[6].replay()
        torch.cuda.synchronize()
        B.arGradNorm(runs[0][4], other, stream=runs[1][5])
        torch.cuda.synchronize()
        check_norm(other, norm_of(hosts[0], "2"))
        for (sizes, devs, outs, norm, lst, st, graph), host in zip(runs, hosts):
            check_norm(norm, norm_of(host, "2"))
            check_clip(outs, host, norm_of(host, "2"), 1.0, 0.75)
    for r in runs:
        r[4].close()


def test_runs_are_bit_equal(B):
    host, devs = grads([3000001, 77, 500000], DTYPES, 51)
    norm = torch.empty(1, device="cuda")
    seen = set()
    with B.TensorList(devs) as lst:
        for _ in range(4):
            B.arGradNorm(lst, norm)
            seen.add(norm.item())
    assert len(seen) == 1


def test_a_training_step(B):
    """4 ranks' batches through layer norm and back, the weights' gradients formed two ways -- summed over the ranks
    by the backward pass, and per rank then added by one group of AllReduces -- and clipped by their global norm
    together with a ReduceScatter's shards."""
    n, cols, dt = 4, 260, torch.float32
    g = torch.Generator().manual_seed(77)
    rows = [50, 61, 7, 33]
    xs = [ou.rows_of(g, (k, cols), dt, 2.0, 0.5) for k in rows]
    dys = [ou.rows_of(g, (k, cols), dt) for k in rows]
    gam, bet = ou.rows_of(g, (cols,), dt, 0.2, 1.0), ou.rows_of(g, (cols,), dt)
    X, D = [t.cuda() for t in xs], [t.cuda() for t in dys]
    G, Be = [gam.cuda() for _ in xs], [bet.cuda() for _ in xs]
    Y, DX = [torch.empty_like(t) for t in X], [torch.empty_like(t) for t in X]
    M, S = [torch.empty(k, device="cuda") for k in rows], [torch.empty(k, device="cuda") for k in rows]
    DG, DB = [torch.empty(cols, device="cuda") for _ in xs], [torch.empty(cols, device="cuda") for _ in xs]
    B.arLayerNorm(X, Y, G, Be, M, S)
    B.arLayerNormBackward(D, X, M, S, G, DX, DG, DB)
    LG, LB = [torch.empty(cols, device="cuda") for _ in xs], [torch.empty(cols, device="cuda") for _ in xs]
    for r in range(n):
        B.arLayerNormBackward([D[r]], [X[r]], [M[r]], [S[r]], [G[r]], None, [LG[r]], [LB[r]])
    with B.Comm(n, 2, "simple") as comm:
        with B.Group():
            comm.allreduce(LG, LG)
            comm.allreduce(LB, LB)
        shards = [torch.empty(65, device="cuda") for _ in xs]
        comm.reduce_scatter(LG, shards)
        torch.cuda.synchronize()
        assert comm.async_error() == B.arSuccess
    pg = torch.zeros(cols, dtype=torch.float64)
    pa = torch.zeros(cols, dtype=torch.float64)
    for r in range(n):
        _, _, p, _ = ou.ln_backward(dys[r], xs[r], M[r].cpu(), S[r].cpu(), gam)
        pg, pa = pg + p.sum(0), pa + p.abs().sum(0)
    db = sum(t.double().sum(0) for t in dys)
    ba = sum(t.double().abs().sum(0) for t in dys)
    for r in range(n):
        for got in (DG[r], LG[r]):
            ou.within(got, pg, (sum(rows) + 8) * ou.U * pa, dt, "dgamma")
        for got in (DB[r], LB[r]):
            ou.within(got, db, (sum(rows) + 8) * ou.U * ba, dt, "dbeta")
    host = [t.cpu() for t in [DG[0], DB[0]] + shards]
    outs = [torch.empty_like(t) for t in [DG[0], DB[0]] + shards]
    norm = torch.empty(1, device="cuda")
    with B.TensorList([DG[0], DB[0]] + shards, outs) as lst:
        B.arGradClip(lst, norm, 1.0, scale=1.0 / n)
        torch.cuda.synchronize()
    check_norm(norm, norm_of(host, "2") / n)
    check_clip(outs, host, norm_of(host, "2") / n, 1.0 / n, 1.0)


@pytest.mark.parametrize("tiles", [15, 16, 17, 63, 64, 65, 511, 512, 513, 4100])
@pytest.mark.parametrize("kind", ["2", "max"])
def test_around_the_launch_rules(B, tiles, kind):
    """Lists on both sides of the sizes where the number of launches and of workgroups changes."""
    host, devs = grads([1024] * (tiles - 1) + [1000], [torch.float32], tiles)
    want = norm_of(host, kind)
    outs = [torch.full_like(t, float("nan")) for t in devs]
    norm = torch.full((1,), float("nan"), device="cuda")
    with B.TensorList(devs, outs) as lst:
        B.arGradNorm(lst, norm, kind=kind)
        check_norm(norm, want)
        norm.fill_(float("nan"))
        B.arGradClip(lst, norm, 0.5 * want, kind=kind)
        torch.cuda.synchronize()
    check_norm(norm, want)
    check_clip(outs, host, want, 1.0, 0.5 * want)


def test_refusals_on_a_list(B):
    t = torch.ones(100, device="cuda")
    o = torch.empty_like(t)
    norm = torch.empty(1, device="cuda")
    with B.TensorList([t], [o]) as lst:
        ws = torch.empty(lst.workspace(), dtype=torch.uint8, device="cuda")
        for kw in (dict(maxNorm=-1.0), dict(maxNorm=math.nan), dict(maxNorm=1.0, eps=-1.0), dict(maxNorm=1.0, eps=math.inf),
                   dict(maxNorm=1.0, scale=math.inf), dict(maxNorm=1.0, scale=math.nan), dict(maxNorm=1.0, kind=7)):
            with pytest.raises(B.ArError):
                B.arGradClip(lst, norm, workspace=ws, **kw)
        with pytest.raises(B.ArError):
            B.arGradNorm(lst, None)
        with pytest.raises(B.ArError):
            B.arGradNorm(lst, ws[:4].view(torch.float32), workspace=ws)
        with pytest.raises(ValueError, match="workspace"):
            B.arGradNorm(lst, norm, workspace=ws[:8])
        with pytest.raises(ValueError, match="norm"):
            B.arGradNorm(lst, torch.empty(2, device="cuda"), workspace=ws)
        B.lib().arGroupStart()
        with pytest.raises(B.ArError):
            B.arGradNorm(lst, norm, workspace=ws)
        assert B.lib().arGroupEnd() == B.arInvalidUsage
    with pytest.raises(ValueError, match="open TensorList"):
        B.arGradNorm(lst, norm)
    big = torch.ones(200, device="cuda")
    for dst in (big[50:150], big[100:]):   # over part of its own tensor, over the other one
        with pytest.raises(B.ArError):
            B.TensorList([big[:100], big[100:]], [dst, o[:100]])
