"""Host-side tests of the sizes at which the grouped planner stops.  Nothing
here launches GPU work."""
import pytest

import tiled_gemm_amd as tg

BF, F32O = tg.GEMM_BF16_OUT_BF16, tg.GEMM_BF16_OUT_F32
BT, PRE, BN, AT_BN = (tg.LAYOUTS[k] for k in ("bt", "bt_preshuffled", "bn", "at_bn"))


@pytest.mark.parametrize("code", [BF, F32O])
@pytest.mark.parametrize("M", [1 << 24, 17_043_520, (1 << 25) - 8])
def test_inner_groups_refuse_rows_a_step_cannot_reach(code, M):
    """One step of the weight gradient loads 64 K-rows of A from one base with
    offsets below 2^31: 64 * M * 2 bytes must stay below that."""
    with pytest.raises(tg.GemmError, match="64 rows of A"):
        tg.GroupPlan(2, M, 16, 1000, code, AT_BN)


def test_inner_groups_take_the_largest_rows():
    with tg.GroupPlan(2, (1 << 24) - 8, 16, 1000, BF, AT_BN) as p:
        assert p.info()["grid"] == 2 * 65536
