"""Results of the operators around the AllReduce are their own: errors of other calls are not theirs, and their
failures leave nothing behind."""
import ctypes

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


@pytest.fixture(autouse=True)
def _named(request):
    import gpu_util
    gpu_util.note(request.node.name)


@pytest.fixture(scope="module")
def hip(B):
    return ctypes.CDLL("libamdhip64.so.7")   # the runtime torch has loaded


@pytest.mark.parametrize("rows,cols", [(3, 40), (600, 40), (600, 5), (600, 17000)], ids=str)
def test_an_earlier_error_is_not_reported(B, hip, rows, cols):
    """A HIP call of the program's own that failed (an ordinal no device has) before each operator."""
    xs, dys, gam, bet = ln.inputs([rows], cols, torch.float32, torch.float32, cols)
    x, dy, g, b = ([t[0].cuda()] for t in (xs, dys, gam, bet))
    y, dx = [torch.empty_like(x[0])], [torch.empty_like(x[0])]
    m, s = [torch.empty(rows, device="cuda")], [torch.empty(rows, device="cuda")]
    gg, gb = [torch.empty(cols, device="cuda")], [torch.empty(cols, device="cuda")]
    ws = torch.empty(B.arLayerNormBackwardWorkspace([rows], cols), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    try:
        assert hip.hipSetDevice(9999) != 0
        B.arLayerNorm(x, y, g, b, m, s)
        assert hip.hipSetDevice(9999) != 0
        B.arLayerNormBackward(dy, x, m, s, g, dx, gg, gb, workspace=ws)
        assert hip.hipSetDevice(9999) != 0
        B.arLayerNormBackward(dy, x, m, s, g, dx)
    finally:
        hip.hipGetLastError()
    torch.cuda.synchronize()
    ln.check_forward(xs, gam, bet, 1e-5, y, m, s)
    ln.check_backward(dys, xs, gam, dx, gg, gb, [m[0].cpu()], [s[0].cpu()])


@pytest.mark.parametrize("n", [100, 3000000])
def test_an_earlier_error_is_not_reported_by_norms(B, hip, n):
    host, devs = gn.grads([n], [torch.float32], n)
    outs = [torch.empty_like(devs[0])]
    norm = torch.empty(1, device="cuda")
    with B.TensorList(devs, outs) as lst:
        ws = torch.empty(lst.workspace(), dtype=torch.uint8, device="cuda")
        try:
            assert hip.hipSetDevice(9999) != 0
            B.arGradNorm(lst, norm, workspace=ws)
            assert hip.hipSetDevice(9999) != 0
            B.arGradClip(lst, norm, 0.5, workspace=ws)
        finally:
            hip.hipGetLastError()
        torch.cuda.synchronize()
    gn.check_norm(norm, gn.norm_of(host, "2"))
    gn.check_clip(outs, host, gn.norm_of(host, "2"), 1.0, 0.5)


def test_a_list_that_cannot_be_freed_stays_whole(B, hip):
    """While a stream is being captured memory may not be freed: the list is still there afterwards, works, and is
    destroyed then."""
    host, devs = gn.grads([70001, 5], [torch.float32], 3)
    norm = torch.empty(1, device="cuda")
    lst = B.TensorList(devs)
    stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
    assert hip.hipStreamCreateWithFlags(ctypes.byref(stream), 1) == 0
    torch.cuda.synchronize()
    assert hip.hipStreamBeginCapture(stream, 0) == 0
    try:
        with pytest.raises(B.ArError):
            lst.close()
    finally:
        hip.hipStreamEndCapture(stream, ctypes.byref(graph))   # the capture was invalidated
        if graph.value:
            hip.hipGraphDestroy(graph)
        hip.hipGetLastError()
    assert lst.handle is not None
    B.arGradNorm(lst, norm)
    gn.check_norm(norm, gn.norm_of(host, "2"))
    lst.close()
    assert lst.handle is None
    lst.close()
    assert hip.hipStreamDestroy(stream) == 0


class StreamElsewhere:
    """A stream of a second device, as torch's streams look."""
    def __init__(self, device_index):
        self.device_index = device_index
        self.cuda_stream = 0


def test_a_stream_of_another_device_is_refused(B):
    x, w = torch.ones(4, 8, device="cuda"), torch.ones(8, device="cuda")
    y, m, s, norm = torch.empty_like(x), torch.empty(4, device="cuda"), torch.empty(4, device="cuda"), torch.empty(1, device="cuda")
    ws = torch.empty(B.arLayerNormBackwardWorkspace([4], 8), dtype=torch.uint8, device="cuda")
    here = torch.cuda.current_device()
    with B.TensorList([x], [y]) as lst:
        lws = torch.empty(lst.workspace(), dtype=torch.uint8, device="cuda")
        calls = [lambda st: B.arLayerNorm([x], [y], [w], [w], [m], [s], stream=st),
                 lambda st: B.arLayerNormBackward([x], [x], [m], [s], [w], [y], [torch.empty_like(w)], None, ws, stream=st),
                 lambda st: B.arGradNorm(lst, norm, workspace=lws, stream=st),
                 lambda st: B.arGradClip(lst, norm, 1.0, workspace=lws, stream=st)]
        for call in calls:
            with pytest.raises(ValueError, match="stream is on cuda:%d" % (here + 1)):
                call(StreamElsewhere(here + 1))
            call(StreamElsewhere(here))
        torch.cuda.synchronize()


def test_any_object_with_a_stream_handle_is_a_stream(B):
    """One that does not name a device is taken at its word, as a raw handle is."""
    class Handle:
        cuda_stream = 0
    x = torch.ones(4, 8, device="cuda")
    y, norm = torch.full_like(x, 9.0), torch.empty(1, device="cuda")
    B.arLayerNorm([x], [y], stream=Handle())
    with B.TensorList([x]) as lst:
        ws = torch.empty(lst.workspace(), dtype=torch.uint8, device="cuda")
        B.arGradNorm(lst, norm, workspace=ws, stream=Handle())
        torch.cuda.synchronize()
    assert (y == 0).all() and abs(norm.item() - 32 ** 0.5) <= 1e-6
