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


@pytest.mark.parametrize("M,N,tile", [(1 << 24, 1 << 16, 32), (1024, (1 << 22) - 16, 32), (1024, (1 << 22) - 16, 256),
                                      (1 << 24, 1 << 18, 256), (1 << 24, 1 << 16, 256),   # 66556 x 256 tiles of 512 threads
                                      (512, (1 << 22) - 16, 32)])                         # 512 x 32768 of 256: 2^32
def test_more_threads_than_a_launch_has_are_refused(M, N, tile):
    with pytest.raises(tg.GemmError, match="2\\^32 threads"):
        tg.GroupPlan(1024, M, N, 32, BF, BT, tile_rows=tile)


def test_the_largest_launches():
    for M, N, tile in ((1 << 24, 16, 0), (1 << 24, 1 << 14, 256), (511, (1 << 22) - 16, 32)):
        with tg.GroupPlan(1024, M, N, 32, BF, BT, tile_rows=tile) as p:
            info = p.info()
        assert 0 < info["grid"] * info["threads"] < 1 << 32
