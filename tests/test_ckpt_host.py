"""Host-side tests of the 8-bit checkpoint: every documented refusal, and calls
of no rows.  Nothing here launches GPU work (each bad call is refused before
the device is touched)."""
import pytest

import tiled_gemm_amd as tg

P = 1 << 40                     # an aligned address that is never read
Q, R, S, T, U = (P + (i << 34) for i in range(1, 6))
BF, F32 = tg.GEMM_TYPE_BF16, tg.GEMM_TYPE_F32


def pack(**kw):
    a = dict(M=64, N=96, type=BF, src=P, q=Q, scales=R)
    a.update(kw)
    tg.gemm_ckpt_pack(**a)


def unpack(**kw):
    a = dict(M=64, N=96, type=BF, epilogue=tg.GEMM_EPI_BIAS_SILU, q=Q, scales=R, out=P)
    a.update(kw)
    tg.gemm_ckpt_unpack(**a)


def grad(**kw):
    a = dict(M=64, N=96, type=BF, epilogue=tg.GEMM_EPI_BIAS_SILU, d_c=P, q=Q, scales=R, d_z=S, d_bias=T, workspace=U,
             workspace_bytes=1 << 20)
    a.update(kw)
    tg.gemm_act_grad_ckpt(**a)


SIZES = [(dict(M=-1), "negative"), (dict(N=-16), "negative"), (dict(N=24), "multiple of 16"),
         (dict(N=1 << 21), "2\\^21"), (dict(M=(1 << 24) + 1), "2\\^24"), (dict(type=7), "type"),
         (dict(type=tg.GEMM_TYPE_BF16 + 1), "type")]


@pytest.mark.parametrize("change,why", SIZES + [
    (dict(src=0), "NULL src"), (dict(q=0), "NULL"), (dict(scales=0), "NULL"), (dict(src=P + 8), "aligned"),
    (dict(q=Q + 8), "aligned"), (dict(q=P), "overlap"), (dict(q=P + 64 * 96 * 2 - 16), "overlap"),
    (dict(scales=P + 3), "overlap"), (dict(scales=Q + 64 * 96 - 1), "overlap"), (dict(scales=Q - 64 * 3 + 1), "overlap"),
    (dict(M=1 << 24, N=(1 << 21) - 16), "too large")])
def test_pack_refusals(change, why):
    with pytest.raises(tg.GemmError, match=why):
        pack(**change)


@pytest.mark.parametrize("change,why", SIZES + [
    (dict(out=0), "NULL out"), (dict(q=0), "NULL"), (dict(scales=0), "NULL"), (dict(out=P + 8), "aligned"),
    (dict(epilogue=5), "epilogue"), (dict(epilogue=-1), "epilogue"), (dict(out=Q + 16), "overlap"),
    (dict(out=R - 16), "overlap")])
def test_unpack_refusals(change, why):
    with pytest.raises(tg.GemmError, match=why):
        unpack(**change)


@pytest.mark.parametrize("change,why", SIZES + [
    (dict(q=0), "NULL"), (dict(scales=0), "NULL scales"), (dict(d_c=0), "NULL"), (dict(d_z=0), "NULL"),
    (dict(d_z=Q), "d_z must be"), (dict(d_z=P + 16), "d_z must be"), (dict(d_z=R), "overlap"),
    (dict(scales=T), "overlap"), (dict(scales=U + 5), "workspace"), (dict(workspace=0), "workspace"),
    (dict(workspace_bytes=16), "workspace"), (dict(groups=2), "offsets"), (dict(groups=0), "groups"),
    (dict(epilogue=5), "epilogue"), (dict(q=Q + 4), "aligned"), (dict(d_bias=Q), "overlap")])
def test_grad_refusals(change, why):
    with pytest.raises(tg.GemmError, match=why):
        grad(**change)


def test_no_rows_or_columns():
    for size in (dict(M=0), dict(N=0), dict(M=0, N=0)):
        pack(src=0, q=0, scales=0, **size)
        unpack(out=0, q=0, scales=0, **size)
    grad(M=0, d_c=0, q=0, scales=0, d_z=0, d_bias=0)
    grad(N=0, d_c=0, q=0, scales=0, d_z=0, d_bias=0)
