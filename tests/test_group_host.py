"""Host-side tests of the grouped-row operators and of the residual epilogue:
planning and every documented refusal.  Nothing here launches GPU work (each
bad call is refused before the device is touched)."""
import pytest

import tiled_gemm_amd as tg

BF, F32O, E4 = tg.GEMM_BF16_OUT_BF16, tg.GEMM_BF16_OUT_F32, tg.GEMM_E4M3_OUT_BF16
BT, PRE, BN, AT, AT_BN = (tg.LAYOUTS[k] for k in ("bt", "bt_preshuffled", "bn", "at", "at_bn"))
P = 1 << 40                     # an aligned address that is never read
Q, R, S, T, U, V = (P + (i << 34) for i in range(1, 7))


@pytest.mark.parametrize("groups,M,layout,tile", [(64, 64, PRE, 32), (64, 24 * 64, BT, 32), (8, 25 * 8, BT, 64),
                                                  (8, 96 * 8, PRE, 64), (8, 97 * 8, BT, 128), (4, 4 * 192, BT, 128),
                                                  (4, 4 * 193, BT, 256), (4, 1, BN, 32), (4, 4096, BN, 256)])
def test_tile_rule_and_grid(groups, M, layout, tile):
    with tg.GroupPlan(groups, M, 528, 256, BF, layout) as p:
        info = p.info()
    assert info["tile_m"] == tile
    tiles_n = -(-528 // info["tile_n"])
    assert info["grid"] == min(M, (M + groups * (tile - 1)) // tile) * tiles_n


def test_grid_bounds_every_split_of_the_rows():
    import itertools
    for tile in (32, 128):
        for M in (0, 1, 15, 16, 17, 40, 130):
            with tg.GroupPlan(3, M, 16, 64, BF, BT, tile_rows=tile) as p:
                grid = p.info()["grid"]
            for a, b in itertools.combinations_with_replacement(range(0, M + 1, max(1, M // 17)), 2):
                sizes = (a, b - a, M - b)
                assert sum(-(-s // tile) for s in sizes) <= grid


def test_inner_grid():
    with tg.GroupPlan(5, 264, 528, 1001, F32O, AT_BN) as p:
        info = p.info()
    assert info["grid"] == 5 * 2 * 3 and info["tile_m"] == 256


@pytest.mark.parametrize("args,why", [
    ((0, 1, 16, 64, BF, BT), "groups"), ((1025, 1, 16, 64, BF, BT), "groups"),
    ((4, -1, 16, 64, BF, BT), "negative"), ((4, 1, 24, 64, BF, BT), "multiple of 16"),
    ((4, 1, 16, 33, BF, BT), "multiple of 64"), ((4, (1 << 24) + 1, 16, 64, BF, BT), "2\\^24"),
    ((4, 1, 16, 64, 9, BT), "dtype"), ((4, 1, 16, 64, BF, 9), "layout"), ((4, 1, 16, 64, BF, AT), "no grouped"),
    ((4, 1, 16, 64, E4, BN), "no grouped"), ((4, 16, 16, 64, E4, AT_BN), "no grouped"),
    ((4, 1, 16, 64, tg.GEMM_I8_OUT_BF16, BT), "bf16 and fp8"), ((4, 4, 16, 64, BF, AT_BN), "16-byte"),
    ((4, 16, 16, (1 << 24) + 1, BF, AT_BN), "2\\^24")])
def test_plan_refusals(args, why):
    with pytest.raises(tg.GemmError, match=why):
        tg.GroupPlan(*args)


@pytest.mark.parametrize("layout,tile,why", [(AT_BN, 64, "no grouped kernel"), (AT_BN, 128, "no grouped kernel"),
                                             (BT, 16, "none of")])
def test_tile_choice_refusals(layout, tile, why):
    with pytest.raises(tg.GemmError, match=why):
        tg.GroupPlan(4, 64, 64, 64, BF, layout, tile_rows=tile)


@pytest.mark.parametrize("kw,why", [
    (dict(A=0), "NULL"), (dict(C=0), "NULL"), (dict(offsets=0), "offsets"), (dict(A=P + 8), "16-byte"),
    (dict(offsets=S + 2), "4-byte"), (dict(C=P), "overlaps"), (dict(C=Q), "overlaps"), (dict(C=S), "overlaps"),
    (dict(preact=R), "preact overlaps"), (dict(preact=T + 8), "16-byte"),
    (dict(row_index=T, a_rows=-1), "a_rows"), (dict(row_index=T, a_rows=1 << 24), "2\\^31"),
    (dict(epilogue=tg.GEMM_EPI_BIAS), "bias"), (dict(epilogue=9), "unknown epilogue"), (dict(bias=U), "GEMM_EPI_NONE"),
    (dict(scale_b=U + 4, scale_b_per_col=True), "16-byte")])
def test_run_refusals(kw, why):
    args = dict(A=P, B=Q, C=R, offsets=S)
    args.update(kw)
    with tg.GroupPlan(4, 100, 64, 64, BF, BT) as p:
        with pytest.raises(tg.GemmError, match=why):
            p.run(**args)


def test_inner_refusals():
    with tg.GroupPlan(4, 64, 64, 100, BF, AT_BN) as p:
        for kw in (dict(row_index=T, a_rows=4), dict(preact=T), dict(bias=U, epilogue=tg.GEMM_EPI_BIAS),
                   dict(scale_a=U, scale_a_per_row=True), dict(scale_b=U, scale_b_per_col=True)):
            with pytest.raises(tg.GemmError, match="AT_BN"):
                p.run(P, Q, R, S, **kw)
        with pytest.raises(tg.GemmError, match="N x K"):
            p.preshuffle_b(P, Q)
        assert p.preshuffled_b_bytes() == 0
    with tg.GroupPlan(4, 64, 64, 128, BF, PRE) as p:
        assert p.preshuffled_b_bytes() == 4 * 64 * 128 * 2
        for a, b in ((0, Q), (P, P + 1024), (P, Q + 8)):
            with pytest.raises(tg.GemmError):
                p.preshuffle_b(a, b)


def test_nothing_to_do_needs_no_device():
    with tg.GroupPlan(4, 0, 64, 64, BF, BT) as p:
        p.run(0, 0, 0, 0)
    tg.gemm_group_combine(0, 2, 64, tg.GEMM_TYPE_BF16, 0, 0, 0, 0)
    tg.gemm_group_combine_grad(0, 2, 64, tg.GEMM_TYPE_BF16, 0, 0, 0, 0, None, 0)
    tg.gemm_act_grad(0, 64, tg.GEMM_TYPE_BF16, tg.GEMM_EPI_BIAS, 0, 0, 0)


@pytest.mark.parametrize("kw,why", [
    (dict(groups=0), "groups"), (dict(groups=1025), "groups"), (dict(slots=-2), "slots"), (dict(slots=7), "multiple"),
    (dict(slots=1 << 25), "slots"), (dict(topk=0), "multiple"), (dict(ids=0), "NULL"), (dict(offsets=0), "NULL"),
    (dict(ids=P + 1), "aligned"), (dict(row_token=S), "overlap"), (dict(slot_row=P), "overlap"),
    (dict(slots=8192), "workspace"), (dict(slots=8192, workspace=T, workspace_bytes=4), "workspace"),
    (dict(slots=8192, workspace=P, workspace_bytes=1 << 20), "overlap")])
def test_sort_refusals(kw, why):
    args = dict(ids=P, slots=8, topk=2, groups=4, offsets=Q, row_token=R, slot_row=S)
    args.update(kw)
    with pytest.raises(tg.GemmError, match=why):
        tg.gemm_group_sort(**args)


def test_sort_workspace_bytes():
    assert tg.gemm_group_sort_workspace_bytes(4096, 64) == 0
    assert tg.gemm_group_sort_workspace_bytes(4097, 64) > 0
    assert tg.gemm_group_sort_workspace_bytes(-1, 64) == tg.gemm_group_sort_workspace_bytes(64, 0) == 0


@pytest.mark.parametrize("kw,why", [
    (dict(tokens=-1), "tokens"), (dict(topk=0), "topk"), (dict(topk=65), "topk"), (dict(N=24), "multiple of 16"),
    (dict(type=2), "type"), (dict(src_rows=-1), "src_rows"), (dict(src=0), "NULL"), (dict(out=0), "NULL"),
    (dict(slot_row=0), "NULL"), (dict(src=P + 8), "aligned"), (dict(out=P), "overlaps"), (dict(out=Q), "overlaps"),
    (dict(weights=R), "overlaps"), (dict(residual=R + 16), "overlaps")])
def test_combine_refusals(kw, why):
    args = dict(tokens=8, topk=2, N=64, type=tg.GEMM_TYPE_BF16, src=P, src_rows=16, slot_row=Q, out=R)
    args.update(kw)
    with pytest.raises(tg.GemmError, match=why):
        tg.gemm_group_combine(**args)


@pytest.mark.parametrize("kw,why", [
    (dict(topk=0), "topk"), (dict(d_out=0), "NULL"), (dict(src=0, d_weights=T), "NULL"), (dict(d_src=0), "NULL"),
    (dict(d_src=P), "overlaps"), (dict(d_src=Q), "overlaps"), (dict(d_weights=P), "overlaps"),
    (dict(d_weights=S), "overlaps"), (dict(d_src=S + 4), "aligned")])
def test_combine_grad_refusals(kw, why):
    args = dict(tokens=8, topk=2, N=64, type=tg.GEMM_TYPE_BF16, d_out=P, src=Q, src_rows=16, slot_row=R, weights=None,
                d_src=S)
    args.update(kw)
    with pytest.raises(tg.GemmError, match=why):
        tg.gemm_group_combine_grad(**args)


@pytest.mark.parametrize("kw,why", [
    (dict(groups=0), "groups"), (dict(groups=2), "offsets"), (dict(M=-1), "negative"), (dict(N=8), "multiple of 16"),
    (dict(type=3), "type"), (dict(epilogue=7), "epilogue"), (dict(z=0), "NULL"), (dict(d_c=0), "NULL"),
    (dict(d_z=0), "NULL"), (dict(d_c=P + 4), "aligned"), (dict(d_z=P + 16), "d_z must be"),
    (dict(d_z=Q + 16), "d_z must be"), (dict(d_bias=S), "workspace"), (dict(d_bias=P), "overlap"),
    (dict(d_bias=S, workspace=P, workspace_bytes=1 << 20), "overlaps"),
    (dict(d_bias=S, workspace=T + 4, workspace_bytes=1 << 20), "workspace")])
def test_act_grad_refusals(kw, why):
    args = dict(M=8, N=64, type=tg.GEMM_TYPE_BF16, epilogue=tg.GEMM_EPI_BIAS_SILU, d_c=P, z=Q, d_z=R)
    args.update(kw)
    with pytest.raises(tg.GemmError, match=why):
        tg.gemm_act_grad(**args)


@pytest.mark.parametrize("kw,why", [
    (dict(residual=R + 16), "residual must be C"), (dict(residual=S + 8), "16-byte"), (dict(preact=S + 8), "16-byte"),
    (dict(preact=R), "preact overlaps"), (dict(preact=P), "preact overlaps"), (dict(preact=S, residual=S), "preact overlaps")])
def test_residual_refusals(kw, why):
    with tg.Plan(200, 64, 64, BF, BT) as p:
        with pytest.raises(tg.GemmError, match=why):
            p.run_res(P, Q, R, **kw)


def test_residual_refusals_by_plan():
    with tg.Plan(200, 64, 64, BF, BT, kernel=tg.GEMM_KERNEL_GENERIC_256) as p:
        with pytest.raises(tg.GemmError, match="kernel choice"):
            p.run_res(P, Q, R, residual=S)
    with tg.Plan(256, 2048, 4096, BF, BT) as p:
        need = p.workspace_bytes()
        with pytest.raises(tg.GemmError, match="workspace overlaps"):
            p.run_res(P, Q, R, residual=S, workspace=S, workspace_bytes=need)
        with pytest.raises(tg.GemmError, match="workspace overlaps"):
            p.run_res(P, Q, R, preact=S, workspace=S, workspace_bytes=need)
    with tg.Plan(200, 64, 64, tg.GEMM_MXFP8_OUT_BF16, BT) as p:
        with pytest.raises(tg.GemmError, match="gemm_run_mx"):
            p.run_res(P, Q, R, residual=S)
        with pytest.raises(tg.GemmError, match="block-scale"):
            p.run_mx_res(P, 0, Q, 0, R, residual=S)
