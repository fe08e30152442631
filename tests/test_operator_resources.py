"""The operators' kernels in the built code object: none spills or uses scratch memory, and those of the headline
widths keep the wavefronts their comments count on.  CPU only."""
import pytest
from test_kernel_resources import kernels  # noqa: F401  (a fixture)

FAMILIES = {"layerNormInRegisters": 65, "layerNormRows": 10, "layerNormBackwardInRegisters": 42,
            "layerNormBackwardRows": 20, "layerNormBackwardColumns": 10, "layerNormBackwardFew": 5,
            "layerNormWeightGrads": 3, "normTiles": 2, "normFinish": 2, "clipTiles": 2, "smallList": 4}


@pytest.mark.parametrize("family", FAMILIES)
def test_operator_kernels_do_not_spill(kernels, family):  # noqa: F811
    hits = {n: k for n, k in kernels.items() if "%d%sI" % (len(family), family) in n}
    assert len(hits) == FAMILIES[family], sorted(hits)
    bad = {n: k for n, k in hits.items() if k["private_segment_fixed_size"] or k["vgpr_spill_count"]}
    assert not bad, bad


def test_registers_of_the_widest_launches(kernels):  # noqa: F811
    """8192 columns of 16 bits: 6 wavefronts a SIMD forward (80 registers), 4 backward (128)."""
    for name, most in (("layerNormInRegistersILi3ELi3ELi512ELi2ELi2E", 80),
                       ("layerNormBackwardInRegistersILi3ELi3ELi1024ELi1ELi3ELi4E", 128)):
        hits = [k for n, k in kernels.items() if name in n]
        assert len(hits) == 1 and hits[0]["vgpr_count"] <= most, hits
