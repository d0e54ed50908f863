"""Which kernel choices have the residual epilogue, as the header lists them.
Nothing here launches GPU work: A is NULL, which every plan that has the
epilogue refuses next."""
import pytest

import tiled_gemm_amd as tg

P = 1 << 40                     # aligned addresses that are never read
Q, R, S, T = (P + (i << 36) for i in range(1, 5))
MX = (tg.GEMM_MXFP8_OUT_BF16, tg.GEMM_MXFP4_OUT_BF16)
CODES = range(7)


def plans(kernel, M):
    for code in CODES:
        for layout in tg.LAYOUTS:
            try:
                p = tg.Plan(M, 528, 256, code, tg.LAYOUTS[layout], kernel=tg.KERNELS[kernel])
            except tg.GemmError:
                continue
            with p:
                yield p, code, layout


def why(p, code, **kw):
    with pytest.raises(tg.GemmError) as e:
        p.run_mx_res(0, P, Q, T, R, **kw) if code in MX else p.run_res(0, Q, R, **kw)
    return str(e.value)


@pytest.mark.parametrize("kw", [dict(residual=S), dict(preact=S)])
@pytest.mark.parametrize("kernel", sorted(tg.KERNELS))
def test_choices_with_a_residual_epilogue(kernel, kw):
    seen = 0
    for M in (16, 64, 304, 4096):
        for p, code, layout in plans(kernel, M):
            has = kernel in ("auto", "tile256", "generic128") or (
                kernel == "pipe" and (layout == "bt_preshuffled" or code == tg.GEMM_W4A8_OUT_BF16))
            assert ("NULL A" if has else "kernel choice") in why(p, code, **kw), (M, code, layout)
            assert "NULL A" in why(p, code)                  # neither: gemm_run_ws
            seen += 1
    assert seen


@pytest.mark.parametrize("per_row,why", [(True, "below 2\\^30"), (False, "NULL A")])
def test_a_scale_per_row_of_the_most_rows(per_row, why):
    """2^30 scales are 2^32 bytes: their record count in 32 bits would be 0."""
    with tg.Plan(1 << 30, 16, 32, tg.GEMM_BF16_OUT_BF16, tg.GEMM_LAYOUT_BT) as p:
        for call in (lambda **kw: p.run_ex(0, Q, R, **kw), lambda **kw: p.run_res(0, Q, R, residual=R, **kw)):
            with pytest.raises(tg.GemmError, match=why):
                call(scale_a=S, scale_a_per_row=per_row)
    with tg.Plan((1 << 30) - 1, 16, 32, tg.GEMM_BF16_OUT_BF16, tg.GEMM_LAYOUT_BT) as p:
        with pytest.raises(tg.GemmError, match="NULL A"):
            p.run_ex(0, Q, R, scale_a=S, scale_a_per_row=True)
