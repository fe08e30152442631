"""The kernels of dropout, token log-probabilities and the policy loss in the built code object: none spills or uses
scratch memory, and the wide ones keep the wavefronts their launches count on.  CPU only."""
import pytest
from test_kernel_resources import kernels  # noqa: F401  (a fixture)

FAMILIES = {"dropoutAddI": 20, "dropoutAddBackwardI": 24, "dropoutAddBackwardFewI": 10, "dropoutBiasGradsI": 3,
            "tokenLogprobRowsI": 54, "tokenLogprobPiecesI": 6, "tokenLogprobJoinE": 1, "tokenLogprobBackwardI": 60,
            "policySumsI": 2, "policyGradI": 2, "policyFewI": 2}


@pytest.mark.parametrize("family", FAMILIES)
def test_kernels_do_not_spill(kernels, family):  # noqa: F811
    hits = {n: k for n, k in kernels.items() if "%d%s" % (len(family) - 1, family) in n}
    assert len(hits) == FAMILIES[family], sorted(hits)
    bad = {n: k for n, k in hits.items() if k["private_segment_fixed_size"] or k["vgpr_spill_count"]}
    assert not bad, bad


def test_registers_leave_wavefronts_enough(kernels):  # noqa: F811
    """Memory-bound kernels with one step a wavefront in flight: 8 wavefronts a SIMD (64 registers), 7 for rows of
    narrow shards, whose threads look their shards up one by one."""
    for name, most in (("dropoutAddI", 64), ("dropoutAddBackwardI", 64), ("tokenLogprobRowsI", 72), ("tokenLogprobBackwardI", 64)):
        for n, k in kernels.items():
            if "%d%s" % (len(name) - 1, name) in n:
                assert k["vgpr_count"] <= (64 if "ELi512E" in n else most), (n, k)
