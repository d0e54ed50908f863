"""Host-side tests of the low-rank adapters: every documented refusal and the
workspace.  Nothing here launches GPU work (each bad call is refused before the
device is touched)."""
import pytest

import tiled_gemm_amd as tg

BF, F32O = tg.GEMM_BF16_OUT_BF16, tg.GEMM_BF16_OUT_F32
BT, PRE, BN = (tg.LAYOUTS[k] for k in ("bt", "bt_preshuffled", "bn"))
P = 1 << 40                     # an aligned address that is never read
AT = [P + (i << 34) for i in range(12)]


def run(p, **kw):
    a = dict(A=AT[0], B=AT[1], C=AT[2], adapter=AT[3], adapters=4, rank=16, down=AT[4], up=AT[5], scale=AT[6],
             residual=AT[7], preact=AT[8], workspace=AT[9], workspace_bytes=1 << 33)
    a.update(kw)
    p.run_lora(**a)


@pytest.mark.parametrize("change,why", [
    (dict(adapters=0), "adapters"), (dict(adapters=65537), "adapters"), (dict(adapters=-1), "adapters"),
    (dict(rank=0), "rank"), (dict(rank=12), "rank"), (dict(rank=264), "rank"), (dict(rank=-8), "rank"),
    (dict(adapter=0), "NULL"), (dict(down=0), "NULL"), (dict(up=0), "NULL"), (dict(A=0), "NULL"), (dict(C=0), "NULL"),
    (dict(adapter=AT[3] + 2), "4-byte"), (dict(scale=AT[6] + 1), "4-byte"), (dict(down=AT[4] + 8), "4-byte"),
    (dict(up=AT[5] + 2), "4-byte"), (dict(A=AT[0] + 8), "16-byte"), (dict(C=AT[2] + 4), "16-byte"),
    (dict(residual=AT[7] + 4), "16-byte"), (dict(preact=AT[8] + 4), "16-byte"), (dict(workspace=AT[9] + 4), "workspace"),
    (dict(workspace=0), "workspace"), (dict(workspace_bytes=100), "workspace"), (dict(workspace=AT[4]), "overlap"),
    (dict(workspace=AT[3]), "overlap"), (dict(workspace=AT[2]), "overlap"), (dict(workspace=AT[8]), "overlap"),
    (dict(workspace=AT[7]), "overlap"), (dict(C=AT[5]), "overlap"), (dict(C=AT[3]), "overlap"),
    (dict(preact=AT[6]), "overlap"), (dict(preact=AT[2] + 16), "preact"), (dict(residual=AT[2] + 16), "residual"),
    (dict(scale_a=AT[10]), "scale"), (dict(scale_b=AT[10]), "scale"), (dict(epilogue=7), "epilogue"),
    (dict(epilogue=tg.GEMM_EPI_BIAS), "bias")])
@pytest.mark.parametrize("M", [5, 300])
def test_run_refusals(M, change, why):
    with tg.Plan(M, 64, 128, BF, BT) as p, pytest.raises(tg.GemmError, match=why):
        run(p, **change)


@pytest.mark.parametrize("dtype,layout,why", [
    (tg.GEMM_E4M3_OUT_BF16, BT, "bf16 plans"), (BF, BN, "bf16 plans"), (tg.GEMM_I8_OUT_BF16, BT, "bf16 plans"),
    (tg.GEMM_MXFP8_OUT_BF16, BT, "MX plans"), (BF, tg.LAYOUTS["at"], "bf16 plans")])
def test_plans_without_adapters(dtype, layout, why):
    with tg.Plan(64, 64, 128, dtype, layout) as p, pytest.raises(tg.GemmError, match=why):
        run(p)


@pytest.mark.parametrize("kernel", ["pipe4", "generic256"])
def test_kernel_choices_without_adapters(kernel):
    with tg.Plan(300, 256, 128, BF, PRE, kernel=tg.KERNELS[kernel]) as p, \
            pytest.raises(tg.GemmError, match="kernel choice"):
        run(p, residual=0, preact=0)


def test_null_descriptions():
    with tg.Plan(4, 64, 128, BF, BT) as p:
        assert tg.load().gemm_run_lora(p.handle, AT[0], AT[1], AT[2], None, None, None, None, AT[9], 1 << 30, 0) == \
            tg.GEMM_ERR_INVALID_ARG
    with pytest.raises(tg.GemmError, match="NULL plan"):
        tg.gemm_run_lora(0, AT[0], AT[1], AT[2], AT[3], 4, 16, AT[4], AT[5])


def test_workspace():
    pad = lambda n: -(-n // 256) * 256
    with tg.Plan(5, 64, 128, BF, BT) as p:
        assert p.lora_workspace_bytes(16) == pad(5 * 32 * 4)
        assert p.lora_workspace_bytes(40) == pad(5 * 64 * 4)
        assert [p.lora_workspace_bytes(r) for r in (0, 4, 20, 264, -16)] == [0] * 5
    with tg.Plan(7, 64, 8192, BF, BT) as p:                    # decode: K in 4 parts of 16 ranks x 4 KiB
        assert p.lora_workspace_bytes(16) == pad(4 * 7 * 32 * 4)
    with tg.Plan(256, 4096, 16384, BF, PRE) as p:              # partial tiles behind v
        assert p.workspace_bytes() > 0
        assert p.lora_workspace_bytes(32) == pad(4 * 256 * 32 * 4) + p.workspace_bytes()
    with tg.Plan(256, 4096, 8192, BF, PRE) as p:               # adapters split K above 8192 only
        assert p.workspace_bytes() > 0
        assert p.lora_workspace_bytes(32) == pad(4 * 256 * 32 * 4)
    with tg.Plan(256, 4096, 8192, BF, PRE, splits=3) as p:     # or where the caller says so
        assert p.lora_workspace_bytes(32) == pad(4 * 256 * 32 * 4) + p.workspace_bytes()
    with tg.Plan(0, 64, 128, BF, BT) as p:
        assert p.lora_workspace_bytes(16) == 0
        run(p, A=0, B=0, C=0, adapter=0, down=0, up=0, scale=0, residual=0, preact=0, workspace=0)      # nothing to do
    assert tg.gemm_lora_workspace_bytes(0, 16) == 0


def test_sizes():
    with tg.Plan((1 << 24) + 1, 16, 32, BF, BT) as p, pytest.raises(tg.GemmError, match="2\\^24"):
        run(p)
