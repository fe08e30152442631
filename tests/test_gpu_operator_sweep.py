"""A seeded random sweep of the operators around the AllReduce: ranks, ragged and empty rows, widths from 1 to
45000, types, padding, odd addresses, in place, lists of mixed tensors; against the 64-bit forms of op_util with
the bounds used elsewhere."""
import math
import random

import op_util as ou
import pytest
import test_gpu_gradnorm as gn
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


@pytest.mark.parametrize("seed", range(48))
def test_random_layer_norms(B, seed):
    import gpu_util
    rng = random.Random(1000 + seed)
    dt, wt = rng.choice(ou.TYPES)
    n = rng.choice([1, 1, 2, 3, 5, 8, 17, 20])
    cols = int(math.exp(rng.uniform(0, math.log(45000))))
    if rng.random() < 0.3:
        cols = max(1, cols // 8 * 8)
    most = max(1, (8000000 if seed % 8 == 0 else 300000) // cols)
    rows = [rng.choice([0, 1, rng.randint(0, max(1, 2 * most // n))]) for _ in range(n)]
    if sum(rows) > 60000:
        rows = [r % 5000 for r in rows]
    pad, offset, into = rng.choice([0, 0, 1, 3, 8]), rng.choice([0, 0, 1, 2, 7]), rng.choice([None, None, "dy", "x"])
    affine, eps = rng.random() < 0.8, rng.choice([1e-5, 1e-3, 1e-6])
    gpu_util.note("layer norm sweep %d: %s %s ranks %d cols %d rows %s pad %d offset %d in place %s affine %s"
                  % (seed, dt, wt, n, cols, rows, pad, offset, into, affine))
    xs, dys, gam, bet = ln.inputs(rows, cols, dt, wt, 7 * seed, affine)
    ln.check_forward(xs, gam, bet, eps, *ln.run_forward(B, xs, gam, bet, eps, pad, offset, inplace=into is not None,
                                                        ypad=None if into else pad + rng.choice([0, 5]),
                                                        stats=rng.random() < 0.7))
    ln.check_backward(dys, xs, gam, *ln.run_backward(B, dys, xs, gam, eps, pad, offset, into=into,
                                                     dx=into is not None or rng.random() < 0.9, db=rng.random() < 0.9))


@pytest.mark.parametrize("seed", range(32))
def test_random_norms_and_clips(B, seed):
    import gpu_util
    rng = random.Random(2000 + seed)
    m = rng.choice([1, 3, 20, 200])
    sizes = [rng.choice([0, 1, rng.randint(1, 50), rng.randint(1, 600000 // m + 2)]) for _ in range(m)]
    dtypes, kind = rng.choice([[t] for t in gn.DTYPES] + [gn.DTYPES]), rng.choice(["2", "max"])
    scale, in_place = rng.choice([1.0, -0.5, 0.0625]), rng.random() < 0.4
    gpu_util.note("gradient norm sweep %d: %d tensors of %d elements, %s, %s, scale %g, in place %s"
                  % (seed, m, sum(sizes), dtypes, kind, scale, in_place))
    host, devs = gn.grads(sizes, dtypes, seed, rng.choice([0, 1, 5]))
    want = abs(scale) * gn.norm_of(host, kind)
    bound = torch.tensor(rng.choice([0.3, 2.0]) * want).float().item()    # as the call receives it
    outs = devs if in_place else [torch.full_like(t, float("nan")) for t in devs]
    norm = torch.empty(1, device="cuda")
    with B.TensorList(devs, outs) as lst:
        B.arGradNorm(lst, norm, kind=kind, scale=scale)
        gn.check_norm(norm, want)
        norm.fill_(float("nan"))
        B.arGradClip(lst, norm, bound, eps=0.0, kind=kind, scale=scale)
        torch.cuda.synchronize()
    gn.check_norm(norm, want)
    if want > 0:
        gn.check_clip(outs, host, want, scale, bound, 0.0)
