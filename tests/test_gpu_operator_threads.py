"""Calls of the operators from several host threads at once, each on a stream and a workspace of its own."""
import threading

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


@pytest.mark.parametrize("rows,cols", [(20, 300), (700, 1030), (600, 17000)], ids=str)
def test_two_threads_at_once(B, rows, cols):
    import gpu_util
    gpu_util.note("two threads, %d x %d" % (rows, cols))
    sets, failures = [], []
    for i in range(2):
        xs, dys, gam, bet = ln.inputs([rows, 3], cols, torch.bfloat16, torch.float32, 10 * i + 1)
        host, devs = gn.grads([cols, 70001, 5], gn.DTYPES, i)
        sets.append(dict(host=(xs, dys, gam, bet), x=[t.cuda() for t in xs], dy=[t.cuda() for t in dys],
                         g=[t.cuda() for t in gam], b=[t.cuda() for t in bet], y=[torch.empty_like(t.cuda()) for t in xs],
                         dx=[torch.empty_like(t.cuda()) for t in xs], m=[torch.empty(len(t), device="cuda") for t in xs],
                         s=[torch.empty(len(t), device="cuda") for t in xs], gg=[torch.empty(cols, device="cuda") for _ in xs],
                         gb=[torch.empty(cols, device="cuda") for _ in xs], grads=host, outs=[torch.empty_like(t) for t in devs],
                         devs=devs, norm=torch.empty(1, device="cuda"), stream=torch.cuda.Stream(),
                         ws=torch.empty(B.arLayerNormBackwardWorkspace([rows, 3], cols), dtype=torch.uint8, device="cuda")))
    torch.cuda.synchronize()

    def work(h):
        try:
            for _ in range(20):
                B.arLayerNorm(h["x"], h["y"], h["g"], h["b"], h["m"], h["s"], stream=h["stream"])
                B.arLayerNormBackward(h["dy"], h["x"], h["m"], h["s"], h["g"], h["dx"], h["gg"], h["gb"], h["ws"],
                                      stream=h["stream"])
                with B.TensorList(h["devs"], h["outs"]) as lst:
                    B.arGradClip(lst, h["norm"], 0.5, stream=h["stream"])
        except Exception as e:   # reported by the test's own thread
            failures.append(e)

    threads = [threading.Thread(target=work, args=(h,)) for h in sets]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failures, failures
    for h in sets:
        xs, dys, gam, bet = h["host"]
        ln.check_forward(xs, gam, bet, 1e-5, h["y"], h["m"], h["s"])
        ln.check_backward(dys, xs, gam, h["dx"], h["gg"], h["gb"], [t.cpu() for t in h["m"]], [t.cpu() for t in h["s"]])
        want = gn.norm_of(h["grads"], "2")
        gn.check_norm(h["norm"], want)
        gn.check_clip(h["outs"], h["grads"], want, 1.0, 0.5)
