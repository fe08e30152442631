"""Arguments of the operators at the ends of their documented ranges, without a GPU."""
import pytest
import test_operators_cpu as ops


@pytest.fixture(scope="module")
def B():
    from ring_allreduce_reduction_amd import binding
    binding.lib()
    return binding


def test_every_finite_eps_is_taken(B):
    """The largest float too.  Without rows nothing is launched."""
    for eps in (0.0, 2.0 ** -149, 3.4e38, (2.0 - 2.0 ** -23) * 2.0 ** 127):
        assert ops.forward(B, eps=eps, rows=ops.N(0)) == B.arSuccess
    for eps in (float("inf"), float("-inf"), float("nan"), -2.0 ** -149):
        assert ops.forward(B, eps=eps, rows=ops.N(0)) == B.arInvalidArgument


@pytest.mark.parametrize("version", ["2.9.1+rocm7.0", "2.10.0+rocm9.9"])
def test_a_module_built_for_another_torch_is_not_used(B, monkeypatch, version):
    """The extension module reads torch's C++ objects: another torch lays them out differently."""
    import torch
    module = B._torch_calls()
    assert "torch " + torch.__version__ in module.built_for
    monkeypatch.setattr(B, "_torch_calls_module", None)
    monkeypatch.setattr(torch, "__version__", version)
    with pytest.raises(ImportError, match="was built for"):
        B.arLayerNorm([torch.zeros(4, 8)], [torch.zeros(4, 8)])
    monkeypatch.undo()
    assert B._torch_calls() is module


def test_row_strides(B):
    """At least the row's width, and no limit but that a rank's rows stay inside 2^48 elements."""
    for stride in (16, (1 << 32) + 1, 1 << 48):
        assert ops.forward(B, xs=stride, ys=stride, rows=ops.N(0)) == B.arSuccess
    for stride in (15, (1 << 48) + 1, 1 << 63):
        assert ops.forward(B, xs=stride, ys=stride, rows=ops.N(0)) == B.arInvalidArgument
    far = dict(x=ops.P(1 << 20), y=ops.P((1 << 20) + 64), xs=1 << 47, ys=1 << 47)
    assert ops.forward(B, rows=ops.N(3), **far) == B.arInvalidArgument
