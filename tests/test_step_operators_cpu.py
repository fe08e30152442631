"""Refusals of dropout, token log-probabilities and the policy loss, through the C ABI and the binding, without a
GPU: bad arguments are found before anything reaches HIP.  And the plain generator the tests compare with."""
import ctypes
import math

import pytest
import step_util as su
import torch
from test_operators_cpu import BASE, N, P


@pytest.fixture(scope="module")
def B():
    from ring_allreduce_reduction_amd import binding
    binding.lib()
    return binding


def Q(*v):
    return (ctypes.c_uint64 * len(v))(*v)


def drop(B, **kw):
    a = dict(x=P(BASE), bias=None, residual=None, y=P(2 * BASE), rows=N(4), first=None, nranks=1, cols=16, xs=16, zs=16,
             ys=16, p=0.1, seed=1, offset=2, step=None, dtype=B.arFloat32, wtype=B.arFloat32)
    a.update(kw)
    return B.lib().arDropoutAdd(a["x"], a["bias"], a["residual"], a["y"], a["rows"], a["first"], a["nranks"], a["cols"],
                                a["xs"], a["zs"], a["ys"], a["p"], a["seed"], a["offset"], a["step"], a["dtype"],
                                a["wtype"], None)


def drop_back(B, **kw):
    a = dict(dy=P(BASE), dx=P(2 * BASE), db=P(3 * BASE), rows=N(4), first=None, nranks=1, cols=16, ds=16, os=16, p=0.1,
             seed=1, offset=2, step=None, dtype=B.arFloat32, wtype=B.arFloat32, ws=8 * BASE, wb=1 << 20)
    a.update(kw)
    return B.lib().arDropoutAddBackward(a["dy"], a["dx"], a["db"], a["rows"], a["first"], a["nranks"], a["cols"], a["ds"],
                                        a["os"], a["p"], a["seed"], a["offset"], a["step"], a["dtype"], a["wtype"],
                                        a["ws"], a["wb"], None)


def logprob(B, **kw):
    """Few rows of a vocabulary long enough to need the workspace."""
    a = dict(x=P(BASE), cols=N(40000), strides=None, nranks=1, rows=4, t=2 * BASE, scale=1.0, logp=3 * BASE, top=4 * BASE,
             ls=5 * BASE, dtype=B.arFloat32, ws=8 * BASE, wb=1 << 20)
    a.update(kw)
    return B.lib().arTokenLogprob(a["x"], a["cols"], a["strides"], a["nranks"], a["rows"], a["t"], a["scale"], a["logp"],
                                  a["top"], a["ls"], a["dtype"], a["ws"], a["wb"], None)


def logprob_back(B, **kw):
    a = dict(d=6 * BASE, x=P(BASE), cols=N(16), strides=None, nranks=1, rows=4, t=2 * BASE, scale=1.0, top=4 * BASE,
             ls=5 * BASE, dx=P(7 * BASE), ds=None, dtype=B.arFloat32)
    a.update(kw)
    return B.lib().arTokenLogprobBackward(a["d"], a["x"], a["cols"], a["strides"], a["nranks"], a["rows"], a["t"],
                                          a["scale"], a["top"], a["ls"], a["dx"], a["ds"], a["dtype"], None)


def policy(B, **kw):
    a = dict(logp=P(BASE), old=P(2 * BASE), ref=P(3 * BASE), adv=P(4 * BASE), w=P(5 * BASE), d=P(6 * BASE), tokens=N(9000),
             nranks=1, low=0.2, high=0.2, kl=0.1, den=0.0, scale=1.0, stats=7 * BASE, ws=8 * BASE, wb=1 << 20)
    a.update(kw)
    return B.lib().arPolicyLoss(a["logp"], a["old"], a["ref"], a["adv"], a["w"], a["d"], a["tokens"], a["nranks"], a["low"],
                                a["high"], a["kl"], a["den"], a["scale"], a["stats"], a["ws"], a["wb"], None)


def refused(call, B, cases):
    for kw in cases:
        assert call(B, **kw) == B.arInvalidArgument, kw


def test_dropout_refusals(B):
    common = [dict(rows=None), dict(nranks=0), dict(nranks=129), dict(cols=0), dict(p=-0.01), dict(p=1.01), dict(p=math.nan),
              dict(dtype=B.arInt32), dict(dtype=9), dict(wtype=B.arBfloat16), dict(step=BASE + 4), dict(rows=N(1 << 31)),
              dict(first=Q((1 << 32) - 3)), dict(first=Q((1 << 32) + 1)), dict(first=Q((1 << 64) - 2))]
    refused(drop, B, common + [
        dict(x=None), dict(y=None), dict(x=P(0)), dict(y=P(2 * BASE + 1)), dict(residual=P(0)), dict(bias=P(0)), dict(xs=15),
        dict(ys=15), dict(residual=P(3 * BASE), zs=15), dict(cols=(1 << 30) + 1, xs=1 << 31, ys=1 << 31),
        dict(rows=N(1 << 40), xs=1 << 32, ys=1 << 32),
        # outputs over other buffers
        dict(y=P(BASE + 4)), dict(y=P(BASE), ys=20), dict(bias=P(2 * BASE)), dict(residual=P(2 * BASE + 64)),
        dict(step=2 * BASE), dict(x=P(BASE, 3 * BASE), y=P(2 * BASE, BASE), rows=N(4, 4), nranks=2)])
    refused(drop_back, B, common + [
        dict(dx=None, db=None), dict(dy=None), dict(dy=P(0)), dict(dx=P(0)), dict(db=P(0)), dict(ds=15), dict(os=15),
        dict(ws=None), dict(ws=8 * BASE + 8), dict(wb=63), dict(dx=P(BASE + 4)), dict(db=P(2 * BASE)), dict(ws=2 * BASE),
        dict(ws=BASE), dict(step=3 * BASE), dict(dx=P(BASE), os=20)])
    # nothing to do
    assert drop(B, rows=N(0), x=None, y=None) == B.arSuccess
    assert drop(B, rows=N(0), first=Q((1 << 64) - 1)) == B.arSuccess
    assert drop_back(B, rows=N(0), dy=None, db=None) == B.arSuccess


def test_logprob_refusals(B):
    common = [dict(cols=None), dict(nranks=0), dict(nranks=129), dict(cols=N(0)), dict(cols=N((1 << 30) + 1)),
              dict(strides=N(15)), dict(strides=N((1 << 48) + 1)), dict(strides=N(1 << 47)), dict(rows=1 << 31),
              dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(scale=1.8e38), dict(dtype=B.arInt32),
              dict(dtype=7), dict(x=None), dict(x=P(0)), dict(x=P(BASE + 2)), dict(t=None), dict(t=2 * BASE + 4)]
    refused(logprob, B, common + [
        dict(logp=None), dict(logp=3 * BASE + 2), dict(top=4 * BASE + 1), dict(ls=5 * BASE + 3), dict(ws=None),
        dict(ws=8 * BASE + 8), dict(wb=31), dict(logp=BASE), dict(top=3 * BASE), dict(ls=2 * BASE), dict(ws=BASE),
        dict(ws=3 * BASE)])
    refused(logprob_back, B, common + [
        dict(d=None), dict(d=6 * BASE + 1), dict(top=None), dict(ls=None), dict(dx=None), dict(dx=P(0)), dict(ds=N(15)),
        dict(dx=P(BASE + 4)), dict(dx=P(2 * BASE)), dict(dx=P(4 * BASE)), dict(dx=P(BASE), ds=N(20)),
        dict(x=P(BASE, 9 * BASE), dx=P(7 * BASE, 7 * BASE + 64), cols=N(16, 16), nranks=2),
        dict(x=P(BASE, 9 * BASE), dx=P(9 * BASE, BASE), cols=N(16, 16), nranks=2)])
    assert logprob(B, rows=0, x=None, t=None, logp=None, ws=None) == B.arSuccess
    assert logprob_back(B, rows=0, x=None, t=None, dx=None) == B.arSuccess


def test_policy_refusals(B):
    refused(policy, B, [
        dict(tokens=None), dict(nranks=0), dict(nranks=129), dict(tokens=N(1 << 31)), dict(stats=None), dict(stats=7 * BASE + 2),
        dict(low=-0.1), dict(low=1.1), dict(low=math.nan), dict(high=-0.1), dict(high=math.nan), dict(kl=-1.0),
        dict(kl=math.inf), dict(kl=math.nan), dict(ref=None), dict(den=-1.0), dict(den=math.inf), dict(den=math.nan),
        dict(scale=math.inf), dict(scale=math.nan), dict(logp=None), dict(old=None), dict(adv=None), dict(logp=P(0)),
        dict(old=P(0)), dict(ref=P(0)), dict(adv=P(2)), dict(w=P(0)), dict(d=P(0)), dict(ws=None), dict(ws=8 * BASE + 8),
        dict(wb=100), dict(d=P(BASE + 4)), dict(d=P(2 * BASE)), dict(stats=BASE), dict(ws=BASE), dict(ws=6 * BASE),
        dict(d=P(4 * BASE)), dict(stats=6 * BASE + 16)])


def test_workspaces(B):
    L, b = B.lib(), ctypes.c_size_t()
    r = ctypes.byref(b)
    for args in ((None, 1, 16, r), (N(4), 1, 16, None), (N(4), 0, 16, r), (N(4), 1, 0, r)):
        assert L.arDropoutAddBackwardWorkspace(*args) == B.arInvalidArgument
    for args in ((4, None, 1, r), (4, N(16), 1, None), (4, N(16), 0, r), (4, N(0), 1, r), (1 << 31, N(16), 1, r)):
        assert L.arTokenLogprobWorkspace(*args) == B.arInvalidArgument
    for args in ((None, 1, r), (N(4), 1, None), (N(4), 0, r), (N(1 << 31), 1, r)):
        assert L.arPolicyLossWorkspace(*args) == B.arInvalidArgument
    for rows in ([0], [1], [100], [1 << 30], [5] * 72):
        for cols in (1, 33, 4096, 1 << 20, (1 << 26) + 1):
            n = B.arDropoutAddBackwardWorkspace(rows, cols)
            # at most 512 partial sums a column, or 16 a launch
            assert n % 16 == 0 and 4 * cols <= n <= 4 * (cols + 8) * max(512, 5 * 16)
    assert B.arTokenLogprobWorkspace(0, [5]) == 0
    for rows, cols in ((1, [16000] * 8), (1000, [9]), (1 << 20, [7] * 17), (3, [1 << 30] * 128)):
        n = B.arTokenLogprobWorkspace(rows, cols)
        assert n % 16 == 0 and n <= 8 * rows * 4096 + 16
    assert B.arPolicyLossWorkspace([0] * 128) == 0 and B.arPolicyLossWorkspace([1]) == 0
    assert 0 < B.arPolicyLossWorkspace([1 << 20] * 128) < 1 << 20


def test_an_open_group_refuses_them(B):
    L = B.lib()
    for call in (drop, drop_back, logprob, logprob_back, policy):
        assert L.arGroupStart() == B.arSuccess
        assert call(B) == B.arInvalidUsage
        assert L.arGroupEnd() == B.arInvalidUsage
    assert L.arGroupStart() == B.arSuccess
    assert L.arGroupEnd() == B.arSuccess


def test_binding_refusals(B):
    """CPU tensors stand in: shape and type checks come before the one for the device."""
    x, w, t, f = torch.zeros(4, 8), torch.zeros(8), torch.zeros(4, dtype=torch.int64), torch.zeros(4)

    def bad(match, call, *args, error=ValueError, **kw):
        with pytest.raises(error, match=match):
            call(*args, **kw)

    bad("at least one rank", B.arDropoutAdd, [], [], 0.1, 0)
    bad("got one tensor", B.arDropoutAdd, x, [x], 0.1, 0)
    bad("need 1 output", B.arDropoutAdd, [x], [x, x], 0.1, 0)
    bad("expected rows of 8", B.arDropoutAdd, [x], [x], 0.1, 0, residuals=[torch.zeros(4, 9)])
    bad("like the others", B.arDropoutAdd, [x], [x], 0.1, 0, residuals=[x.half()])
    bad("bias buffer 0 must hold 8", B.arDropoutAdd, [x], [x], 0.1, 0, biases=[w[:5]])
    bad("weights must be", B.arDropoutAdd, [x], [x], 0.1, 0, biases=[w.half()])
    bad("step must be an int64", B.arDropoutAdd, [x], [x], 0.1, 0, step=f)
    bad("step must be an int64", B.arDropoutAdd, [x], [x], 0.1, 0, step=t)
    bad("need 1 first rows", B.arDropoutAdd, [x], [x], 0.1, 0, firstRows=[1, 2])
    bad(".", B.arDropoutAdd, [x], [x], 0.1, -1, error=OverflowError)
    bad(".", B.arDropoutAdd, [x], [x], 0.1, 1 << 64, error=OverflowError)
    bad(".", B.arDropoutAdd, [x], [x], 0.1, 0, 1.5, error=TypeError)
    bad(".", B.arDropoutAdd, [x], [x], 0.1, 0, firstRows=[-1], error=OverflowError)
    bad("device tensors", B.arDropoutAdd, [x], [x], 0.1, 0, 3, t[:1], [w], [x], [7])
    bad("need 1 input gradient", B.arDropoutAddBackward, [x], [], 0.1, 0)
    bad("bias gradient buffer 0", B.arDropoutAddBackward, [x], [x], 0.1, 0, dbiases=[w[:3]])
    bad("device tensors", B.arDropoutAddBackward, [x], [x], 0.1, 0, dbiases=[w])
    bad("at least one rank", B.arTokenLogprob, [], t, f)
    bad("got one tensor", B.arTokenLogprob, x, t, f)
    bad("float32, float16 or bfloat16", B.arTokenLogprob, [x.double()], t, f)
    bad("like the others", B.arTokenLogprob, [x, x.half()], t, f)
    bad("has 3 rows, expected 4", B.arTokenLogprob, [x, x[:3]], t, f)
    bad("contiguous rows", B.arTokenLogprob, [torch.zeros(8, 4).t()], t, f)
    bad("targets is", B.arTokenLogprob, [x], t.int(), f)
    bad("targets must hold 4", B.arTokenLogprob, [x], t[:3], f)
    bad("logp must hold 4", B.arTokenLogprob, [x], t, w)
    bad("expected a tensor", B.arTokenLogprob, [x], t, None)
    bad("top is", B.arTokenLogprob, [x], t, f, f.half(), f)
    bad("device tensors", B.arTokenLogprob, [x, x], t, f, f, f)
    bad("need 1 logits gradient", B.arTokenLogprobBackward, f, [x], t, f, f, [x, x])
    bad("has 7 columns, expected 8", B.arTokenLogprobBackward, f, [x], t, f, f, [x[:, :7]])
    bad("has 3 rows, expected 4", B.arTokenLogprobBackward, f, [x], t, f, f, [x[:3]])
    bad("expected torch.float32 like", B.arTokenLogprobBackward, f, [x], t, f, f, [x.half()])
    bad("expected a tensor", B.arTokenLogprobBackward, f, [x], t, None, f, [x])
    bad("device tensors", B.arTokenLogprobBackward, f, [x], t, f, f, [x])
    s = torch.zeros(5)
    bad("at least one rank", B.arPolicyLoss, [], [], [], s)
    bad("got one tensor", B.arPolicyLoss, f, [f], [f], s)
    bad("need 1 old logp buffers", B.arPolicyLoss, [f], [f, f], [f], s)
    bad("list of tensors", B.arPolicyLoss, [f], None, [f], s, error=TypeError)
    bad("old logp buffer 0 must hold 4", B.arPolicyLoss, [f], [w], [f], s)
    bad("advantage buffer 0 is", B.arPolicyLoss, [f], [f], [f.half()], s)
    bad("weight buffer 0 is torch.bool|weight buffer 0 is Bool", B.arPolicyLoss, [f], [f], [f], s, weights=[f.bool()])
    bad("stats must hold 5", B.arPolicyLoss, [f], [f], [f], f)
    bad("device tensors", B.arPolicyLoss, [f], [f], [f], s, [f], [f], [f], klCoef=0.1)


def test_the_plain_generator():
    """Known answers of Philox4x32-10: zeros, ones and digits of pi."""
    def words(c, k):
        return [int(w) for w in su.philox(c, k)]
    assert words([0] * 4, (0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert words([0xFFFFFFFF] * 4, (0xFFFFFFFF, 0xFFFFFFFF)) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert words([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], (0xA4093822, 0x299F31D0)) == [
        0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]
