"""Refusals of the operators around the AllReduce, through the C ABI and the binding, without a GPU: bad
arguments are found before anything reaches HIP."""
import ctypes
import math

import pytest
import torch


@pytest.fixture(scope="module")
def B():
    from ring_allreduce_reduction_amd import binding
    binding.lib()
    return binding


def P(*v):
    return (ctypes.c_void_p * len(v))(*v)


def N(*v):
    return (ctypes.c_size_t * len(v))(*v)


BASE = 1 << 20   # made-up addresses: none of these calls reaches the device


def forward(B, **kw):
    a = dict(x=P(BASE), gamma=None, beta=None, y=P(2 * BASE), mean=None, rstd=None, rows=N(4), nranks=1, cols=16,
             xs=16, ys=16, eps=1e-5, dtype=B.arFloat32, wtype=B.arFloat32)
    a.update(kw)
    return B.lib().arLayerNorm(a["x"], a["gamma"], a["beta"], a["y"], a["mean"], a["rstd"], a["rows"], a["nranks"],
                               a["cols"], a["xs"], a["ys"], a["eps"], a["dtype"], a["wtype"], None)


def backward(B, **kw):
    a = dict(dy=P(BASE), x=P(2 * BASE), gamma=None, mean=P(3 * BASE), rstd=P(4 * BASE), dx=P(5 * BASE),
             dg=P(6 * BASE), db=P(7 * BASE), rows=N(4), nranks=1, cols=16, ds=16, xs=16, os=16, dtype=B.arFloat32,
             wtype=B.arFloat32, ws=8 * BASE, wb=1 << 20)
    a.update(kw)
    return B.lib().arLayerNormBackward(a["dy"], a["x"], a["gamma"], a["mean"], a["rstd"], a["dx"], a["dg"], a["db"],
                                       a["rows"], a["nranks"], a["cols"], a["ds"], a["xs"], a["os"], a["dtype"],
                                       a["wtype"], a["ws"], a["wb"], None)


def test_forward_refusals(B):
    bad = [dict(rows=None), dict(nranks=0), dict(nranks=129), dict(cols=0), dict(cols=(1 << 30) + 1, xs=1 << 31, ys=1 << 31),
           dict(xs=15), dict(ys=15), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(dtype=B.arInt32),
           dict(dtype=B.arUint64), dict(dtype=9), dict(wtype=B.arBfloat16), dict(dtype=B.arFloat16, wtype=B.arBfloat16),
           dict(x=None), dict(y=None), dict(x=P(0)), dict(y=P(0)), dict(x=P(BASE + 2)), dict(mean=P(3 * BASE)),
           dict(rstd=P(3 * BASE)), dict(gamma=P(0)), dict(beta=P(BASE + 1)), dict(mean=P(3 * BASE), rstd=P(0)),
           dict(rows=N(1 << 31)), dict(rows=N(1 << 30, 1 << 30), nranks=2, x=P(BASE, BASE), y=P(2 * BASE, 3 * BASE)), dict(rows=N(1 << 40), xs=1 << 32, ys=1 << 32)]
    for kw in bad:
        assert forward(B, **kw) == B.arInvalidArgument, kw
    # nothing to do
    assert forward(B, rows=N(0), x=None, y=None) == B.arSuccess
    assert forward(B, rows=N(0), x=P(0), y=P(0)) == B.arSuccess


def test_forward_overlaps(B):
    row = 16 * 4
    bad = [dict(y=P(BASE + 4)), dict(y=P(BASE + 3 * row)), dict(y=P(BASE), ys=20),
           dict(gamma=P(2 * BASE)), dict(mean=P(BASE), rstd=P(3 * BASE)), dict(mean=P(3 * BASE), rstd=P(3 * BASE + 8)),
           dict(x=P(BASE, 3 * BASE), y=P(2 * BASE, 2 * BASE + row), rows=N(4, 4), nranks=2),
           # rank 1 writes over rank 0's input
           dict(x=P(BASE, 3 * BASE), y=P(2 * BASE, BASE), rows=N(4, 4), nranks=2),
           # column slices that share a column
           dict(y=P(BASE + 15 * 4), xs=64, ys=64)]
    for kw in bad:
        assert forward(B, **kw) == B.arInvalidArgument, kw


def test_backward_refusals(B):
    bad = [dict(dx=None, dg=None, db=None), dict(dy=None), dict(x=None), dict(mean=None), dict(rstd=None), dict(ds=3),
           dict(os=15), dict(dy=P(0)), dict(x=P(0)), dict(mean=P(0)), dict(rstd=P(2)), dict(dx=P(0)), dict(dg=P(0)),
           dict(db=P(0)), dict(gamma=P(0)), dict(ws=None), dict(ws=8 * BASE + 8), dict(wb=16 * 8 - 1),
           dict(dtype=B.arInt32), dict(wtype=B.arFloat16), dict(nranks=0), dict(cols=0),
           # outputs over inputs, each other or the workspace
           dict(dx=P(BASE + 4)), dict(dx=P(BASE), os=20), dict(dg=P(7 * BASE + 4)), dict(dg=P(5 * BASE)),
           dict(db=P(2 * BASE + 8)), dict(ws=5 * BASE), dict(ws=2 * BASE), dict(gamma=P(6 * BASE))]
    for kw in bad:
        assert backward(B, **kw) == B.arInvalidArgument, kw


def test_backward_workspace(B):
    b = ctypes.c_size_t()
    f = B.lib().arLayerNormBackwardWorkspace
    assert f(None, 1, 16, ctypes.byref(b)) == B.arInvalidArgument
    assert f(N(4), 1, 16, None) == B.arInvalidArgument
    assert f(N(4), 0, 16, ctypes.byref(b)) == B.arInvalidArgument
    assert f(N(4), 1, 0, ctypes.byref(b)) == B.arInvalidArgument
    for rows in ([0], [1], [100], [1 << 30], [5] * 72):
        n = B.arLayerNormBackwardWorkspace(rows, 33)
        assert n >= 2 * 33 * 4 and n <= 8 * 1024 * 2 * 33 * 4 * ((len(rows) + 31) // 32)


def lists(B, n=2, src=(BASE, 2 * BASE), dst=None, counts=(8, 8), dtypes=(1, 1), out=True):
    h = ctypes.c_void_p(5)
    rc = B.lib().arTensorListCreate(ctypes.byref(h) if out else None, n, None if src is None else P(*src),
                                    None if dst is None else P(*dst), None if counts is None else N(*counts),
                                    None if dtypes is None else (ctypes.c_int * len(dtypes))(*dtypes))
    assert not out or rc == B.arSuccess or h.value is None
    return rc


def test_list_refusals(B):
    bad = [dict(out=False), dict(n=-1), dict(n=(1 << 20) + 1), dict(src=None), dict(counts=None), dict(dtypes=None),
           dict(src=(0, BASE)), dict(src=(BASE + 2, 2 * BASE)), dict(dst=(0, BASE)), dict(dst=(3 * BASE + 1, 4 * BASE)),
           dict(dtypes=(0, 1)), dict(dtypes=(1, 4)), dict(counts=((1 << 40) + 1, 1)),
           dict(counts=(1 << 40, 1)), dict(counts=(1 << 38, 1)),   # more tiles than a list may have
           # outputs over each other, another tensor, part of their own, the same tensor twice in place
           dict(dst=(3 * BASE, 3 * BASE + 16)), dict(dst=(2 * BASE, 3 * BASE)), dict(dst=(BASE + 4, 2 * BASE)),
           dict(src=(BASE, BASE), dst=(BASE, BASE))]
    for kw in bad:
        assert lists(B, **kw) == B.arInvalidArgument, kw
    if not torch.cuda.is_available():
        assert lists(B) == B.arHipError


def test_calls_without_a_list(B):
    L = B.lib()
    junk = ctypes.create_string_buffer(4096)
    b = ctypes.c_size_t()
    for h in (None, ctypes.cast(junk, ctypes.c_void_p)):
        assert L.arGradNorm(h, 0, 1.0, BASE, BASE, 1 << 20, None) == B.arInvalidArgument
        assert L.arGradClip(h, 0, 1.0, 1.0, 0.0, BASE, BASE, 1 << 20, None) == B.arInvalidArgument
        assert L.arTensorListWorkspace(h, ctypes.byref(b)) == B.arInvalidArgument
    assert L.arTensorListDestroy(None) == B.arSuccess
    assert L.arTensorListDestroy(ctypes.cast(junk, ctypes.c_void_p)) == B.arInvalidArgument


def test_an_open_group_refuses_them(B):
    """They do not queue: inside a group they are refused, and the group reports it."""
    L = B.lib()
    assert L.arGroupStart() == B.arSuccess
    assert forward(B) == B.arInvalidUsage
    assert backward(B) == B.arInvalidUsage
    assert L.arGroupEnd() == B.arInvalidUsage
    assert L.arGroupStart() == B.arSuccess
    assert L.arGroupEnd() == B.arSuccess


def test_binding_refusals(B):
    """CPU tensors stand in: shape and type checks come before the one for the device."""
    x, w = torch.zeros(4, 8), torch.zeros(8)
    with pytest.raises(ValueError, match="at least one rank"):
        B.arLayerNorm([], [])
    for args in ((x, [x]), ([x], x), ([x], [x], x)):
        with pytest.raises(ValueError, match="got one tensor"):
            B.arLayerNorm(*args)
    with pytest.raises(TypeError, match="list of tensors"):
        B.arLayerNorm(5, [x])
    with pytest.raises(ValueError, match="expected a tensor"):
        B.arLayerNorm([5], [x])
    with pytest.raises(ValueError, match="at most 128"):
        B.arLayerNorm([x] * 129, [x] * 129)
    with pytest.raises(ValueError, match="float32, float16 or bfloat16"):
        B.arLayerNorm([x.double()], [x.double()])
    with pytest.raises(ValueError, match="at least one column"):
        B.arLayerNorm([torch.zeros(4, 0)], [torch.zeros(4, 0)])
    with pytest.raises(ValueError, match="need 1 output"):
        B.arLayerNorm([x], [])
    with pytest.raises(ValueError, match="expected rows of 8"):
        B.arLayerNorm([x], [torch.zeros(4, 9)])
    with pytest.raises(ValueError, match="has 3 rows, expected 4"):
        B.arLayerNorm([x], [torch.zeros(3, 8)])
    with pytest.raises(ValueError, match="like the others"):
        B.arLayerNorm([x], [x.half()])
    with pytest.raises(ValueError, match="contiguous rows"):
        B.arLayerNorm([torch.zeros(8, 4).t()], [x])
    with pytest.raises(ValueError, match="contiguous rows"):
        B.arLayerNorm([x[:1].expand(4, 8)], [x])
    with pytest.raises(ValueError, match="row stride 8, the others 12"):
        B.arLayerNorm([torch.zeros(4, 12)[:, :8], x], [x, x])
    with pytest.raises(ValueError, match="gamma buffer 0 must hold 8"):
        B.arLayerNorm([x], [x], [w[:7]])
    with pytest.raises(ValueError, match="weights must be"):
        B.arLayerNorm([x], [x], [w.half()])
    with pytest.raises(ValueError, match="beta buffer 0 is"):
        B.arLayerNorm([x.half()], [x.half()], [w.half()], [w])
    with pytest.raises(ValueError, match="both means and rstds"):
        B.arLayerNorm([x], [x], means=[torch.zeros(4)])
    with pytest.raises(ValueError, match="mean buffer 0"):
        B.arLayerNorm([x], [x], means=[torch.zeros(3)], rstds=[torch.zeros(4)])
    with pytest.raises(ValueError, match="device tensors"):
        B.arLayerNorm([x], [x], [w], [w])
    with pytest.raises(ValueError, match="need 1 output gradient"):
        B.arLayerNormBackward([], [x], [torch.zeros(4)], [torch.zeros(4)])
    with pytest.raises(ValueError, match="rstd buffer 0"):
        B.arLayerNormBackward([x], [x], [torch.zeros(4)], [torch.zeros(5)])
    with pytest.raises(ValueError, match="device tensors"):
        B.arLayerNormBackward([x], [x], [torch.zeros(4)], [torch.zeros(4)], [w], [x], [w], [w])
    with pytest.raises(ValueError, match="need 1 outputs"):
        B.arTensorListCreate([x], [])
    with pytest.raises(ValueError, match="tensor 0 is"):
        B.arTensorListCreate([x.int()])
    with pytest.raises(ValueError, match="output 0 must hold"):
        B.arTensorListCreate([x], [x.half()])
    with pytest.raises(ValueError, match="tensor 0 must hold"):
        B.arTensorListCreate([x.t()])
    with pytest.raises(ValueError, match="device tensors"):
        B.arTensorListCreate([x])
    with pytest.raises(ValueError, match="open TensorList"):
        B.arGradNorm(None, w[:1])
