"""Refusals of the adapters and of the few-token expert layer that come before anything is launched, on the CPU."""
import pytest

import tiled_gemm_amd as tg

BF, BT, PRE = tg.GEMM_BF16_OUT_BF16, tg.LAYOUTS["bt"], tg.LAYOUTS["bt_preshuffled"]
P = 1 << 40                     # an aligned address that is never read
AT = [P + (i << 34) for i in range(12)]


@pytest.mark.parametrize("M", [5, 300])
@pytest.mark.parametrize("change", [dict(workspace=AT[10]), dict(C=AT[10]), dict(preact=AT[10]),
                                    dict(workspace=AT[10] + 240), dict(C=AT[10] + 240)])
def test_adapters_bias_overlaps_an_output(M, change):
    """The bias is read behind the first launch, which has written the workspace by then."""
    a = dict(A=AT[0], B=AT[1], C=AT[2], adapter=AT[3], adapters=4, rank=16, down=AT[4], up=AT[5], scale=AT[6],
             residual=AT[7], preact=AT[8], workspace=AT[9], workspace_bytes=1 << 33, bias=AT[10],
             epilogue=tg.GEMM_EPI_BIAS)
    a.update(change)
    with tg.Plan(M, 64, 128, BF, BT) as p, pytest.raises(tg.GemmError, match="overlap"):
        p.run_lora(**a)


@pytest.mark.parametrize("change,why", [
    (dict(down=0), "NULL"), (dict(down_image=0), "NULL"), (dict(down=AT[2] + 8), "16-byte"),
    (dict(down_image=AT[3] + 4), "16-byte"), (dict(down_image=AT[2] + 16), "overlap"), (dict(down_image=AT[1]), "overlap"),
    (dict(down_image=AT[0]), "overlap"), (dict(up_image=AT[2]), "overlap"), (dict(up_image=AT[3] + 4096), "overlap")])
def test_preshuffle_checks_both_matrices_first(change, why):
    """Nothing is launched for one matrix where the other is refused, and no image lies on what is still to be read."""
    a = dict(up=AT[0], up_image=AT[1], down=AT[2], down_image=AT[3])
    a.update(change)
    with tg.GroupMlpPlan(8, 4, 2, 128, 64, tg.GEMM_TYPE_BF16, PRE, True, tg.GEMM_EPI_BIAS_SILU) as p, \
            pytest.raises(tg.GemmError, match=why):
        p.preshuffle(**a)


@pytest.mark.parametrize("gated,weight_type", [(True, tg.GEMM_TYPE_BF16), (False, tg.GEMM_TYPE_BF16),
                                               (True, tg.GEMM_TYPE_E4M3), (False, tg.GEMM_TYPE_E4M3)])
def test_more_tokens_than_the_layer_takes(gated, weight_type):
    """The refusal names the single products only as what they are: without the gate, and with rows of the weights' type."""
    with pytest.raises(tg.GemmError) as e:
        tg.GroupMlpPlan(8, 65, 2, 128, 64, weight_type, BT, gated, tg.GEMM_EPI_BIAS_SILU)
    text = str(e.value)
    assert "gemm_group_run" in text
    assert ("gate" in text) == gated and ("e4m3 rows" in text) == (weight_type == tg.GEMM_TYPE_E4M3)
