"""Host-side tests of the mixture-of-experts layer for a few tokens: planning
and every documented refusal.  Nothing here launches GPU work (each bad call is
refused before the device is touched)."""
import pytest

import tiled_gemm_amd as tg

BF, E4, F32 = tg.GEMM_TYPE_BF16, tg.GEMM_TYPE_E4M3, tg.GEMM_TYPE_F32
BT, PRE = tg.LAYOUTS["bt"], tg.LAYOUTS["bt_preshuffled"]
SILU = tg.GEMM_EPI_BIAS_SILU
P = 1 << 40                     # an aligned address that is never read
AT = [P + (i << 34) for i in range(12)]


def plan(groups=8, tokens=4, topk=2, K=128, N=64, weight_type=BF, layout=BT, gated=True, epilogue=SILU):
    return tg.GroupMlpPlan(groups, tokens, topk, K, N, weight_type, layout, gated, epilogue)


@pytest.mark.parametrize("change,why", [
    (dict(groups=0), "groups"), (dict(groups=1025), "groups"), (dict(tokens=-1), "tokens"), (dict(tokens=65), "tokens"),
    (dict(topk=0), "topk"), (dict(topk=65), "topk"), (dict(weight_type=F32), "bf16 or e4m3"),
    (dict(weight_type=3), "weight_type"), (dict(weight_type=-1), "weight_type"), (dict(layout=9), "unknown layout"),
    (dict(layout=tg.LAYOUTS["bn"]), "GEMM_LAYOUT_BT"), (dict(gated=2), "gated"), (dict(epilogue=5), "epilogue"),
    (dict(epilogue=-1), "epilogue"), (dict(K=0), "positive"), (dict(N=0), "positive"), (dict(K=-32), "positive"),
    (dict(K=48), "multiple of 64"), (dict(N=48), "multiple of 64"), (dict(N=40), "multiple"),
    (dict(weight_type=E4, K=96), "multiple of 64"), (dict(weight_type=E4, N=96), "multiple of 64"),
    (dict(N=1 << 21), "2\\^20"), (dict(K=1 << 21), "2\\^20"),
    (dict(tokens=64, topk=64, N=1 << 18), "2\\^30")])
def test_plan_refusals(change, why):
    with pytest.raises(tg.GemmError, match=why):
        plan(**change)


def test_query_and_workspace():
    with plan(tokens=5, topk=3, K=160, N=96, gated=False) as p:
        assert p.info() == dict(tokens=5, K=160, N=96, groups=8, topk=3, weight_type=BF, layout=BT, gated=0,
                                epilogue=SILU)
        # the slots' hidden rows (bf16), their sums (fp32), one counter per 32 output columns
        up = lambda n: -(-n // 256) * 256
        assert p.workspace_bytes() == up(15 * 96 * 2) + up(15 * 160 * 4) + 5 * 4
    with plan(tokens=0) as p:
        assert p.workspace_bytes() == 0
        p.run(0, 0, 0, 0, 0)                                   # no tokens: nothing to do
    assert tg.gemm_group_mlp_workspace_bytes(0) == 0


def run(p, **kw):
    a = dict(x=AT[0], ids=AT[1], up=AT[2], down=AT[3], out=AT[4], weights=AT[5], up_scale=AT[6], down_scale=AT[7],
             up_bias=AT[8], down_bias=AT[9], residual=AT[10], workspace=AT[11], workspace_bytes=1 << 30)
    a.update(kw)
    p.run(**a)


@pytest.mark.parametrize("change,why", [
    (dict(x=0), "NULL"), (dict(ids=0), "NULL"), (dict(up=0), "NULL"), (dict(down=0), "NULL"), (dict(out=0), "NULL"),
    (dict(workspace=0), "workspace"), (dict(workspace_bytes=64), "workspace"), (dict(x=AT[0] + 8), "16-byte"),
    (dict(up=AT[2] + 8), "16-byte"), (dict(down=AT[3] + 2), "16-byte"), (dict(out=AT[4] + 4), "16-byte"),
    (dict(residual=AT[10] + 4), "16-byte"), (dict(workspace=AT[11] + 4), "16-byte"), (dict(ids=AT[1] + 2), "4-byte"),
    (dict(weights=AT[5] + 1), "4-byte"), (dict(up_bias=AT[8] + 2), "4-byte"), (dict(out=AT[0]), "overlap"),
    (dict(out=AT[1]), "overlap"), (dict(out=AT[2] + 16), "overlap"), (dict(out=AT[9]), "overlap"),
    (dict(residual=AT[4] + 16), "overlap"), (dict(residual=AT[11]), "overlap"), (dict(out=AT[11]), "overlap"),
    (dict(workspace=AT[3]), "overlap"), (dict(workspace=AT[5]), "overlap")])
def test_run_refusals(change, why):
    with plan() as p, pytest.raises(tg.GemmError, match=why):
        run(p, **change)


def test_preshuffle_refusals():
    with plan(layout=PRE) as p:
        with pytest.raises(tg.GemmError, match="NULL"):
            p.preshuffle(0, AT[0], AT[1], AT[2])
        with pytest.raises(tg.GemmError, match="overlap"):
            p.preshuffle(AT[0], AT[0], AT[1], AT[2])
    with pytest.raises(tg.GemmError, match="NULL plan"):
        tg.gemm_group_mlp_preshuffle(0, AT[0], AT[1], AT[2], AT[3])
    with pytest.raises(tg.GemmError, match="NULL plan"):
        tg.gemm_group_mlp_run(0, AT[0], AT[1], AT[2], AT[3], AT[4])
