"""The grouped-row operators against plain 64-bit computations of their
definitions (numpy / torch float64 on the host).

Bit-exact wherever every intermediate is exact in the type that holds it:
integer inputs with sums below 2^24 (fp32) for the products, powers of two for
scales and weights.  Elsewhere the bounds are derived beside the test from:
fp32 accumulation (4e-6 of the sum of magnitudes, the library's GEMM bound),
fp32 elementwise arithmetic (2^-20 of the magnitudes involved), and the one
rounding to the output type (half a step: 2^-9 of the value in bf16, 2^-24 in
fp32, counted as 2^-8 and 2^-23).
"""
import numpy as np
import pytest
import torch

import tiled_gemm_amd as tg

pytestmark = pytest.mark.gpu

BF, F32O, E4 = tg.GEMM_BF16_OUT_BF16, tg.GEMM_BF16_OUT_F32, tg.GEMM_E4M3_OUT_BF16
CODE = {"bf16": BF, "f32": F32O, "e4m3": E4}
RHO = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -23}


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def stream():
    return torch.cuda.current_stream().cuda_stream


def ints(rng, shape, lo, hi):
    return rng.integers(lo, hi + 1, shape).astype(np.float64)


def dev(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dtype).cuda()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def f32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda()


def host(t):
    return t.to(torch.float64).cpu().numpy()


def cuts(rng, groups, rows, first=0, empty=0.3):
    """Random group offsets, some groups empty, the last up to `rows`."""
    sizes = rng.random(groups) * (rng.random(groups) > empty)
    if sizes.sum() == 0:
        sizes[-1] = 1.0
    at = first + np.floor(np.cumsum(sizes) / sizes.sum() * (rows - first)).astype(int)
    return np.concatenate([[first], at])


def act64(z, kind):
    t = torch.from_numpy(z)
    if kind == "relu":
        t = t.clamp(min=0)
    elif kind == "silu":
        t = t * torch.sigmoid(t)
    elif kind == "gelu":
        t = 0.5 * t * torch.erfc(-t / 2 ** 0.5)
    return t.numpy()


# ------------------------------------------------------------------ routing tables

def sort_ref(ids, topk, groups):
    flat = ids.reshape(-1)
    ok = (flat >= 0) & (flat < groups)
    order = np.argsort(np.where(ok, flat, groups), kind="stable")[:ok.sum()]
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[ok], minlength=groups))])
    slot_row = np.full(flat.size, -1)
    slot_row[order] = np.arange(order.size)
    return offsets, order // topk, slot_row


def run_sort(ids, topk, groups):
    n = ids.size
    d = i32(ids.reshape(-1)) if n else torch.empty(1, dtype=torch.int32, device="cuda")
    off, tok, row = (torch.full((m,), 77, dtype=torch.int32, device="cuda") for m in (groups + 1, max(n, 1), max(n, 1)))
    need = tg.gemm_group_sort_workspace_bytes(n, groups)
    ws = torch.full((max(4, need),), 0x55, dtype=torch.uint8, device="cuda")
    tg.gemm_group_sort(d.data_ptr(), n, topk, groups, off.data_ptr(), tok.data_ptr(), row.data_ptr(), ws.data_ptr(),
                       need, stream())
    torch.cuda.synchronize()
    return off, tok[:n], row[:n]


@pytest.mark.parametrize("tokens,topk,groups,lo,hi", [
    (0, 2, 5, 0, 4), (1, 1, 1, 0, 0), (1, 8, 8, 0, 7), (3, 2, 64, 0, 63), (64, 4, 7, 0, 6), (500, 8, 64, -3, 70),
    (4096, 1, 1024, 0, 1023), (4097, 1, 1024, 0, 1023), (1025, 4, 65, -1, 64), (20000, 8, 256, 0, 255),
    (777, 3, 33, 5, 5), (5000, 2, 16, -9, -1), (9999, 1, 3, 3, 9), (300000, 1, 129, 0, 200)])
def test_sort(tokens, topk, groups, lo, hi):
    print("case sort", tokens, topk, groups, flush=True)
    rng = np.random.default_rng(tokens + groups)
    ids = rng.integers(lo, hi + 1, (tokens, topk))
    if tokens > 10:
        ids[3, 0], ids[4, 0] = -2 ** 31, 2 ** 31 - 1      # far outside: slots that go nowhere
    off, tok, row = run_sort(ids, topk, groups)
    roff, rtok, rrow = sort_ref(ids, topk, groups)
    assert np.array_equal(off.cpu().numpy(), roff)
    assert np.array_equal(row.cpu().numpy(), rrow)
    assert np.array_equal(tok.cpu().numpy()[:rtok.size], rtok)
    assert bool((tok[rtok.size:] == 77).all())            # behind the last routed row: as it was


# ------------------------------------------------------------------ grouped products

# (type, layout, tile rows)
FAMILIES = ([(t, lay, tile) for t in ("bf16", "f32", "e4m3") for lay in ("bt", "bt_preshuffled")
             for tile in (32, 64, 128, 256)] + [(t, "bn", tile) for t in ("bf16", "f32") for tile in (32, 64, 128, 256)])


def grouped(plan, A, B, C, offsets, **kw):
    if plan.info()["layout"] == tg.GEMM_LAYOUT_BT_PRESHUFFLED:
        image = torch.empty(max(16, plan.preshuffled_b_bytes()), dtype=torch.uint8, device="cuda")
        plan.preshuffle_b(B.data_ptr(), image.data_ptr(), stream())
        B = image
    plan.run(A.data_ptr(), B.data_ptr(), C.data_ptr(), offsets.data_ptr(), stream=stream(), **kw)
    torch.cuda.synchronize()


@pytest.mark.parametrize("types,layout,tile", FAMILIES)
@pytest.mark.parametrize("groups,rows,gather", [(1, 1, False), (5, 300, False), (5, 300, True), (70, 333, True),
                                               (3, 700, False), (130, 77, True)])
def test_grouped_rows_bit_exact(types, layout, tile, groups, rows, gather):
    print("case grouped", types, layout, tile, groups, rows, gather, flush=True)
    N, K = 176, (352 if types != "e4m3" else 320)        # a half-filled last 128-byte step, ragged columns
    rng = np.random.default_rng(groups * 1000 + rows + tile)
    M = rows + 9                                          # room behind the last group
    off = cuts(rng, groups, rows, first=min(2, rows - 1))
    a_rows = 41 if gather else M
    a, b = ints(rng, (a_rows, K), -3, 3), ints(rng, (groups, N, K), -3, 3)
    sa, sb = 2.0 ** rng.integers(-1, 2, a_rows), 2.0 ** rng.integers(-1, 2, (groups, N))
    bias = ints(rng, (groups, N), -9, 9)
    index = rng.integers(0, a_rows, M)                    # the same row twice and more
    index[rng.random(M) < 0.1] = -1
    index[rng.random(M) < 0.05] = a_rows + 5
    et = torch.float8_e4m3fn if types == "e4m3" else torch.bfloat16
    ct = torch.float32 if types == "f32" else torch.bfloat16
    z = np.zeros((M, N))
    inside = np.zeros(M, bool)
    for g in range(groups):
        r = np.arange(off[g], off[g + 1])
        inside[r] = True
        src = index[r] if gather else r
        ok = (src >= 0) & (src < a_rows)
        src = np.where(ok, src, 0)
        z[r] = (a[src] @ b[g].T) * sa[src][:, None] * sb[g] * ok[:, None] + bias[g]
    A = dev(a, torch.float32)
    if not gather:
        A[torch.from_numpy(~inside).cuda()] = float("nan")    # rows of no group are never used
    A = A.to(et)
    B = dev(b.transpose(0, 2, 1) if layout == "bn" else b, torch.float32).to(et)
    C = torch.full((M, N), 5.0, dtype=ct, device="cuda")
    Z = torch.full_like(C, 6.0)
    dsa, dsb, dbias = f32(sa), f32(sb), f32(bias)
    with tg.GroupPlan(groups, M, N, K, CODE[types], tg.LAYOUTS[layout], tile_rows=tile) as p:
        assert p.info()["tile_m"] == tile
        grouped(p, A, B, C, i32(off), row_index=i32(index).data_ptr() if gather else None, a_rows=a_rows,
                preact=Z.data_ptr(), scale_a=dsa.data_ptr(), scale_a_per_row=True, scale_b=dsb.data_ptr(),
                scale_b_per_col=True, bias=dbias.data_ptr(), epilogue=tg.GEMM_EPI_BIAS_RELU)
    want_c = np.where(inside[:, None], np.maximum(z, 0.0), 5.0)
    want_z = np.where(inside[:, None], z, 6.0)
    assert torch.equal(C, dev(want_c, torch.float32).to(ct))
    assert torch.equal(Z, dev(want_z, torch.float32).to(ct))


@pytest.mark.parametrize("layout,tile", [("bt", 0), ("bt_preshuffled", 32), ("bt", 64), ("bt", 128), ("bt_preshuffled", 256),
                                         ("bn", 128), ("bn", 256)])
@pytest.mark.parametrize("kind", ["silu", "gelu", "none"])
def test_grouped_rows_random(layout, tile, kind):
    groups, rows, N, K = 6, 410, 400, 1056
    rng = np.random.default_rng(17)
    off = cuts(rng, groups, rows)
    a = host(dev(rng.normal(0, 1, (rows, K)), torch.float32).to(torch.bfloat16))
    b = host(dev(rng.normal(0, 1.5 * K ** -0.5, (groups, N, K)), torch.float32).to(torch.bfloat16))
    bias = rng.normal(0, 0.5, (groups, N)).astype(np.float32).astype(np.float64)
    acc, S = np.zeros((rows, N)), np.zeros((rows, N))
    for g in range(groups):
        r = slice(off[g], off[g + 1])
        acc[r], S[r] = a[r] @ b[g].T, np.abs(a[r]) @ np.abs(b[g].T)
    bz = np.concatenate([np.repeat(bias[g][None], off[g + 1] - off[g], 0) for g in range(groups)]) * (kind != "none")
    C = torch.zeros((rows, N), dtype=torch.bfloat16, device="cuda")
    B = b.transpose(0, 2, 1) if layout == "bn" else b
    dbias = f32(bias)
    with tg.GroupPlan(groups, rows, N, K, BF, tg.LAYOUTS[layout], tile_rows=tile) as p:
        grouped(p, dev(a, torch.bfloat16), dev(B, torch.bfloat16), C, i32(off),
                bias=dbias.data_ptr() if kind != "none" else None,
                epilogue=tg.EPILOGUES["none" if kind == "none" else "bias_" + kind])
    ref = act64(acc + bz, kind)
    # the pre-activation's error through the activation's slope (at most 1.13)
    bound = 1.13 * (4e-6 * S + 2.0 ** -20 * (np.abs(acc) + np.abs(bz))) + 2.0 ** -8 * np.abs(ref)
    assert np.all(np.abs(host(C) - ref) <= bound)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("groups,rows,M,N", [(1, 1, 8, 16), (4, 0, 264, 272), (5, 300, 264, 272), (3, 129, 520, 48),
                                             (40, 200, 24, 304), (2, 64, 256, 256)])
def test_weight_gradient_bit_exact(out, groups, rows, M, N):
    print("case weight gradient", out, groups, rows, M, N, flush=True)
    rng = np.random.default_rng(rows + M)
    cap = rows + 5
    off = cuts(rng, groups, rows, first=min(1, rows)) if rows else np.zeros(groups + 1, int)
    a, b = ints(rng, (cap, M), -3, 3), ints(rng, (cap, N), -3, 3)
    A, B = dev(a, torch.bfloat16), dev(b, torch.bfloat16)
    A[:off[0]], B[:off[0]], A[off[-1]:], B[off[-1]:] = (float("nan"),) * 4      # rows of no group
    C = torch.full((groups, M, N), 9.0, dtype=torch.float32 if out == "f32" else torch.bfloat16, device="cuda")
    s = torch.tensor([0.5, 4.0], device="cuda")
    with tg.GroupPlan(groups, M, N, cap, CODE[out], tg.GEMM_LAYOUT_AT_BN) as p:
        grouped(p, A, B, C, i32(off), scale_a=s.data_ptr(), scale_b=s.data_ptr() + 4)
    want = np.stack([2.0 * a[lo:hi].T @ b[lo:hi] for lo, hi in zip(off[:-1], off[1:])])
    assert torch.equal(C, dev(want, torch.float32).to(C.dtype))


def test_offsets_outside_the_rows_are_clamped():
    rng = np.random.default_rng(2)
    a, b = ints(rng, (40, 64), -3, 3), ints(rng, (3, 32, 64), -3, 3)
    for tile in (32, 128, 256):
        C = torch.full((40, 32), 5.0, dtype=torch.float32, device="cuda")
        with tg.GroupPlan(3, 40, 32, 64, F32O, tg.GEMM_LAYOUT_BT, tile_rows=tile) as p:
            grouped(p, dev(a, torch.bfloat16), dev(b, torch.bfloat16), C, i32([-7, 10, 2 ** 30, 2 ** 31 - 1]))
        want = np.concatenate([a[:10] @ b[0].T, a[10:] @ b[1].T])
        assert np.array_equal(host(C), want)


def test_rows_past_32_bits():
    """C, and in the weight gradient A, beyond 2^32 bytes: the far rows against
    the plain product of those rows."""
    M, N, K, groups = 300_001, 4096, 64, 3
    g = torch.Generator(device="cuda").manual_seed(1)
    A = torch.randint(-3, 4, (M, K), generator=g, device="cuda").to(torch.bfloat16)
    B = torch.randint(-3, 4, (groups, N, K), generator=g, device="cuda").to(torch.bfloat16)
    off = [0, 1000, 1001, M]
    C = torch.empty((M, N), dtype=torch.float32, device="cuda")
    with tg.GroupPlan(groups, M, N, K, F32O, tg.GEMM_LAYOUT_BT) as p:
        grouped(p, A, B, C, i32(off))
    for e, rows in ((0, slice(0, 300)), (1, slice(1000, 1001)), (2, slice(262_100, 262_300)), (2, slice(M - 200, M))):
        assert torch.equal(C[rows], A[rows].float() @ B[e].float().t())
    del C
    rows, M, N = 600_013, 4096, 16                        # A: 4.9e9 bytes
    A = torch.zeros((rows, M), dtype=torch.bfloat16, device="cuda")
    B = torch.zeros((rows, N), dtype=torch.bfloat16, device="cuda")
    for at in (0, 262_143, 262_144, 524_287, 524_288, rows - 1):
        A[at] = torch.randint(-3, 4, (M,), generator=g, device="cuda").to(torch.bfloat16)
        B[at] = torch.randint(-3, 4, (N,), generator=g, device="cuda").to(torch.bfloat16)
    C = torch.empty((2, M, N), dtype=torch.float32, device="cuda")
    with tg.GroupPlan(2, M, N, rows, F32O, tg.GEMM_LAYOUT_AT_BN) as p:
        grouped(p, A, B, C, i32([0, 5, rows]))
    live = torch.tensor([262_143, 262_144, 524_287, 524_288, rows - 1], device="cuda")
    assert torch.equal(C[0], A[:5].float().t() @ B[:5].float())
    assert torch.equal(C[1], A[live].float().t() @ B[live].float())


# ------------------------------------------------------------------ combine and its gradient

@pytest.mark.parametrize("tokens,topk,N", [(1, 1, 16), (1, 8, 2048), (33, 3, 272), (257, 5, 4112), (40, 64, 80), (7, 2, 8208)])
@pytest.mark.parametrize("kind,weights,residual", [("bf16", True, True), ("f32", True, False), ("bf16", False, False)])
def test_combine_and_gradient(tokens, topk, N, kind, weights, residual):
    print("case combine", tokens, topk, N, kind, flush=True)
    rng = np.random.default_rng(tokens * topk + N)
    t = torch.bfloat16 if kind == "bf16" else torch.float32
    code = tg.GEMM_TYPE_BF16 if kind == "bf16" else tg.GEMM_TYPE_F32
    rows = tokens * topk + 3
    perm = rng.permutation(rows)[:tokens * topk].reshape(tokens, topk)
    slot_row = np.where(rng.random((tokens, topk)) < 0.2, -1, perm)
    if topk > 1:
        slot_row[0, 0] = rows + 7                        # past src: contributes nothing
        slot_row[-1, :] = -1 if tokens > 1 else slot_row[-1, :]      # a token whose slots all went nowhere
    live = (slot_row >= 0) & (slot_row < rows)
    at = np.where(live, slot_row, 0)
    src, res, dout = (host(dev(rng.normal(0, 1, s), torch.float32).to(t)) for s in ((rows, N), (tokens, N), (tokens, N)))
    w = rng.normal(0, 1, (tokens, topk)).astype(np.float32)
    w64 = np.where(live, w.astype(np.float64) if weights else 1.0, 0.0)
    dw = f32(np.where(live, w, np.nan))                   # weights of dead slots are never used
    S, R = dev(src, t), dev(res, t)
    dead = np.setdiff1d(np.arange(rows), slot_row[live])
    S[torch.from_numpy(dead).cuda()] = float("nan")       # rows that no slot names are never read
    out = R.clone()
    tg.gemm_group_combine(tokens, topk, N, code, S.data_ptr(), rows, i32(slot_row).data_ptr(), out.data_ptr(),
                          weights=dw.data_ptr() if weights else None, residual=out.data_ptr() if residual else None,
                          stream=stream())
    ref = (w64[:, :, None] * src[at]).sum(1) + (res if residual else 0.0)
    mag = (np.abs(w64)[:, :, None] * np.abs(src[at])).sum(1) + (np.abs(res) if residual else 0.0)
    # fp32 sum of topk + 1 terms: at most topk + 1 roundings of 2^-24 of the magnitudes
    eps = (topk + 1) * 2.0 ** -24
    assert np.all(np.abs(host(out) - ref) <= eps * mag + RHO[t] * np.abs(ref))

    dsrc = torch.full((rows, N), 3.0, dtype=t, device="cuda")
    dwt = torch.full((tokens, topk), 3.0, device="cuda")
    D = dev(dout, t)
    tg.gemm_group_combine_grad(tokens, topk, N, code, D.data_ptr(), S.data_ptr(), rows, i32(slot_row).data_ptr(),
                               dw.data_ptr() if weights else None, dsrc.data_ptr(), dwt.data_ptr(), stream())
    want = np.full((rows, N), 3.0)
    want[slot_row[live]] = (w64[:, :, None] * dout[:, None, :])[live]
    assert np.all(np.abs(host(dsrc) - want) <= (RHO[t] + 2.0 ** -23) * np.abs(want))
    ref = (src[at] * dout[:, None, :]).sum(2) * live
    mag = (np.abs(src[at]) * np.abs(dout)[:, None, :]).sum(2) * live
    assert np.all(np.abs(host(dwt) - ref) <= N * 2.0 ** -24 * mag + 2.0 ** -23 * np.abs(ref))
    only = torch.full_like(dsrc, 3.0)                     # without the weights' gradient, src is not needed
    tg.gemm_group_combine_grad(tokens, topk, N, code, D.data_ptr(), None, rows, i32(slot_row).data_ptr(),
                               dw.data_ptr() if weights else None, only.data_ptr(), None, stream())
    assert torch.equal(only, dsrc)


# ------------------------------------------------------------------ gradient of the epilogue

def slope64(z, kind):
    t = torch.from_numpy(z)
    if kind == "bias_relu":
        return (t > 0).double().numpy()
    if kind == "bias_silu":
        s = torch.sigmoid(t)
        return (s + t * s * torch.sigmoid(-t)).numpy()
    if kind == "bias_gelu":
        return (0.5 * torch.erfc(-t / 2 ** 0.5) + t * torch.exp(-t * t / 2) / (2 * np.pi) ** 0.5).numpy()
    return np.ones_like(z)


@pytest.mark.parametrize("kind", ["none", "bias_relu", "bias_silu", "bias_gelu"])
def test_slope_is_the_derivative_of_the_epilogue(kind):
    """The formula above against central differences of the forward definition."""
    z = np.linspace(-9, 9, 2001) + 1e-3
    h = 1e-5
    act = kind.replace("bias_", "")
    diff = (act64(z + h, act) - act64(z - h, act)) / (2 * h)
    assert np.abs(slope64(z, kind) - diff).max() < 1e-8


@pytest.mark.parametrize("kind", ["none", "bias", "bias_relu", "bias_silu", "bias_gelu"])
@pytest.mark.parametrize("M,N,groups", [(1, 16, 1), (130, 528, 1), (300, 1040, 5), (77, 272, 200), (5000, 4112, 3)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_act_grad(kind, M, N, groups, dtype):
    rng = np.random.default_rng(M + N)
    code = tg.GEMM_TYPE_BF16 if dtype == torch.bfloat16 else tg.GEMM_TYPE_F32
    dc, z = (host(dev(rng.normal(0, s, (M, N)), torch.float32).to(dtype)) for s in (1.0, 2.0))
    off = cuts(rng, groups, max(1, M - 3)) if groups > 1 else np.array([0, M])
    D, Z = dev(dc, dtype), dev(z, dtype)
    out = torch.full_like(D, 4.0)
    db = torch.full((groups, N), 4.0, device="cuda")
    need = tg.gemm_act_grad_workspace_bytes(M, N, groups)
    ws = torch.full((need,), 0x7F, dtype=torch.uint8, device="cuda")
    offsets = i32(off) if groups > 1 else None
    args = dict(groups=groups, offsets=offsets.data_ptr() if groups > 1 else None, stream=stream())
    tg.gemm_act_grad(M, N, code, tg.EPILOGUES[kind], D.data_ptr(), Z.data_ptr(), out.data_ptr(), db.data_ptr(),
                     workspace=ws.data_ptr(), workspace_bytes=need, **args)
    full = dc * slope64(z, kind)
    inside = np.zeros(M, bool)
    inside[off[0]:off[-1]] = True
    want = np.where(inside[:, None], full, 4.0)
    # fp32 evaluation of the slope: within 2^-19 of its largest value (1.13) and of z times it
    mag = np.abs(dc) * (1.13 + np.abs(z) * slope64(-np.abs(z), "bias_silu").__abs__())
    tol = np.where(inside[:, None], 2.0 ** -19 * mag, 0.0)
    assert np.all(np.abs(host(out) - want) <= tol + RHO[dtype] * np.abs(want))
    for g in range(groups):
        r = slice(off[g], off[g + 1])
        n = off[g + 1] - off[g]
        bound = (2.0 ** -19 + n * 2.0 ** -24) * mag[r].sum(0)
        assert np.all(np.abs(host(db[g]) - full[r].sum(0)) <= bound)
    # in place over either operand, without the bias
    for target in ("d", "z"):
        D2, Z2 = D.clone(), Z.clone()
        t = D2 if target == "d" else Z2
        before = t.clone()
        tg.gemm_act_grad(M, N, code, tg.EPILOGUES[kind], D2.data_ptr(), Z2.data_ptr(), t.data_ptr(), **args)
        m = torch.from_numpy(inside).cuda()[:, None]
        assert torch.equal(t, torch.where(m, out, before))


def test_act_grad_at_the_ends():
    z = torch.tensor([float("-inf"), float("inf"), -3e38, 3e38, -0.0, 0.0, float("nan"), -90.0] * 2, device="cuda")[None]
    dc, out = torch.ones_like(z), torch.empty_like(z)
    want = {"bias_relu": [0, 1, 0, 1, 0, 0, 0, 0], "bias_silu": [0, 1, 0, 1, 0.5, 0.5, np.nan, 0],
            "bias_gelu": [0, 1, 0, 1, 0.5, 0.5, np.nan, 0]}
    for kind, w in want.items():
        tg.gemm_act_grad(1, 16, tg.GEMM_TYPE_F32, tg.EPILOGUES[kind], dc.data_ptr(), z.data_ptr(), out.data_ptr(),
                         stream=stream())
        np.testing.assert_allclose(host(out)[0, :8], w, rtol=0, atol=1e-30)


# ------------------------------------------------------------------ together

def sparse(rng, shape, n):
    """Matrices with n entries of +-1 in every row: products stay small integers."""
    w = np.zeros(shape)
    for i in np.ndindex(shape[:-1]):
        w[i][rng.choice(shape[-1], n, replace=False)] = rng.choice([-1.0, 1.0], n)
    return w


class Layer:
    """A mixture-of-experts layer y = x + sum_j w_j W2_e relu(W1_e x + b1_e), forward and backward."""

    def __init__(self, tokens, topk, experts, width, inner, layout):
        self.shape = tokens, topk, experts, width, inner
        rows, bf = tokens * topk, torch.bfloat16
        e = lambda *s, dtype=bf: torch.zeros(s, dtype=dtype, device="cuda")
        self.ids, self.w = e(tokens, topk, dtype=torch.int32), e(tokens, topk, dtype=torch.float32)
        self.off, self.tok, self.row = (e(n, dtype=torch.int32) for n in (experts + 1, rows, rows))
        self.x, self.y, self.dy, self.dx = (e(tokens, width) for _ in range(4))
        self.h, self.z, self.dh = (e(rows, inner) for _ in range(3))
        self.u, self.du, self.dxr = (e(rows, width) for _ in range(3))
        self.dw = e(tokens, topk, dtype=torch.float32)
        self.w1, self.w2 = e(experts, inner, width), e(experts, width, inner)
        self.b1, self.db1 = (e(experts, inner, dtype=torch.float32) for _ in range(2))
        self.dw1, self.dw2 = torch.zeros_like(self.w1), torch.zeros_like(self.w2)
        P, L = tg.GroupPlan, tg.LAYOUTS
        self.layout = layout
        self.up, self.down = P(experts, rows, inner, width, BF, L[layout]), P(experts, rows, width, inner, BF, L[layout])
        self.dup, self.ddown = P(experts, rows, width, inner, BF, L["bn"]), P(experts, rows, inner, width, BF, L["bn"])
        self.gup, self.gdown = P(experts, inner, width, rows, BF, L["at_bn"]), P(experts, width, inner, rows, BF, L["at_bn"])
        n = max(tg.gemm_group_sort_workspace_bytes(rows, experts), tg.gemm_act_grad_workspace_bytes(rows, inner, experts), 16)
        self.ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        self.i1, self.i2 = self.w1, self.w2

    def weights(self, w1, b1, w2):
        self.w1.copy_(dev(w1, torch.bfloat16)), self.w2.copy_(dev(w2, torch.bfloat16)), self.b1.copy_(f32(b1))
        if self.layout == "bt_preshuffled":
            self.i1, self.i2 = torch.empty_like(self.w1), torch.empty_like(self.w2)
            self.up.preshuffle_b(self.w1.data_ptr(), self.i1.data_ptr(), stream())
            self.down.preshuffle_b(self.w2.data_ptr(), self.i2.data_ptr(), stream())

    def forward(self):
        T, k, E, D, H = self.shape
        s, p = stream(), lambda t: t.data_ptr()
        tg.gemm_group_sort(p(self.ids), T * k, k, E, p(self.off), p(self.tok), p(self.row), p(self.ws), self.ws.numel(), s)
        self.up.run(p(self.x), p(self.i1), p(self.h), p(self.off), row_index=p(self.tok), a_rows=T, preact=p(self.z),
                    bias=p(self.b1), epilogue=tg.GEMM_EPI_BIAS_RELU, stream=s)
        self.down.run(p(self.h), p(self.i2), p(self.u), p(self.off), stream=s)
        tg.gemm_group_combine(T, k, D, tg.GEMM_TYPE_BF16, p(self.u), T * k, p(self.row), p(self.y), weights=p(self.w),
                              residual=p(self.x), stream=s)

    def backward(self):
        T, k, E, D, H = self.shape
        s, p, R = stream(), lambda t: t.data_ptr(), T * k
        tg.gemm_group_combine_grad(T, k, D, tg.GEMM_TYPE_BF16, p(self.dy), p(self.u), R, p(self.row), p(self.w), p(self.du),
                                   p(self.dw), s)
        self.gdown.run(p(self.du), p(self.h), p(self.dw2), p(self.off), stream=s)
        self.ddown.run(p(self.du), p(self.w2), p(self.dh), p(self.off), stream=s)
        tg.gemm_act_grad(R, H, tg.GEMM_TYPE_BF16, tg.GEMM_EPI_BIAS_RELU, p(self.dh), p(self.z), p(self.dh), p(self.db1), E,
                         p(self.off), p(self.ws), self.ws.numel(), s)
        self.xr = self.x[self.tok.long()]                # the weight gradient reads the gathered tokens
        self.gup.run(p(self.dh), p(self.xr), p(self.dw1), p(self.off), stream=s)
        self.dup.run(p(self.dh), p(self.w1), p(self.dxr), p(self.off), stream=s)
        tg.gemm_group_combine(T, k, D, tg.GEMM_TYPE_BF16, p(self.dxr), R, p(self.row), p(self.dx), residual=p(self.dy), stream=s)


def layer_inputs(rng, tokens, topk, experts, width):
    ids = np.stack([rng.choice(experts, topk, replace=False) for _ in range(tokens)])
    return (ids, 2.0 ** rng.integers(-1, 2, (tokens, topk)), ints(rng, (tokens, width), -2, 2),
            ints(rng, (tokens, width), -2, 2) * (rng.random((tokens, width)) < 0.05))


def layer_reference(ids, w, x, dy, w1, b1, w2):
    t = lambda v: torch.from_numpy(np.ascontiguousarray(v)).double().requires_grad_(True)
    x, w, w1, b1, w2 = map(t, (x, w, w1, b1, w2))
    rows = []
    for tok in range(x.shape[0]):
        y = x[tok]
        for j, e in enumerate(ids[tok]):
            y = y + w[tok, j] * (w2[e] @ torch.relu(w1[e] @ x[tok] + b1[e]))
        rows.append(y)
    y = torch.stack(rows)
    y.backward(torch.from_numpy(dy))
    return [v.detach().numpy() for v in (y, x.grad, w.grad, w1.grad, b1.grad, w2.grad)]


@pytest.mark.parametrize("tokens,topk,experts,layout", [(1, 2, 4, "bt_preshuffled"), (9, 2, 11, "bt"), (90, 3, 5, "bt")])
def test_expert_layer_forward_and_backward(tokens, topk, experts, layout):
    """Small integers and powers of two all the way: every value the layer
    rounds to bf16 is exact, so outputs and gradients equal autograd's in 64
    bits."""
    width, inner = 64, 96
    rng = np.random.default_rng(tokens)
    layer = Layer(tokens, topk, experts, width, inner, layout)
    w1, w2, b1 = sparse(rng, (experts, inner, width), 3), sparse(rng, (experts, width, inner), 3), ints(rng, (experts, inner), -2, 2)
    layer.weights(w1, b1, w2)
    for again in range(2):
        ids, w, x, dy = layer_inputs(rng, tokens, topk, experts, width)
        layer.ids.copy_(i32(ids)), layer.w.copy_(f32(w)), layer.x.copy_(dev(x, torch.float32)), layer.dy.copy_(dev(dy, torch.float32))
        layer.forward()
        layer.backward()
        torch.cuda.synchronize()
        want = layer_reference(ids, w, x, dy, w1, b1, w2)
        for name, got, ref in zip(("y", "dx", "dw", "dw1", "db1", "dw2"),
                                  (layer.y, layer.dx, layer.dw, layer.dw1, layer.db1, layer.dw2), want):
            exact = dev(ref, torch.float32).to(got.dtype)
            assert np.array_equal(host(exact), ref), name      # the reference itself is exact in the type
            assert torch.equal(got, exact), name


def test_expert_layer_in_a_graph():
    """Forward and backward captured once, replayed on other tokens, routes and
    weights with eager work between the replays."""
    shape = (37, 2, 6, 64, 96)
    rng = np.random.default_rng(8)
    a, b = Layer(*shape, "bt"), Layer(*shape, "bt")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                           # another stream than the default one
        a.forward(), a.backward()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.forward(), a.backward()
    for _ in range(3):
        w1, w2 = rng.normal(0, 0.3, (6, 96, 64)), rng.normal(0, 0.3, (6, 64, 96))
        ids, w, x, dy = layer_inputs(rng, *shape[:4])
        for m in (a, b):
            m.weights(w1, np.zeros((6, 96)), w2)
            m.ids.copy_(i32(ids)), m.w.copy_(f32(w)), m.x.copy_(dev(x, torch.float32)), m.dy.copy_(dev(dy, torch.float32))
        b.forward(), b.backward()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for name in ("off", "row", "y", "dx", "dw", "dw1", "db1", "dw2"):
            assert torch.equal(getattr(a, name), getattr(b, name)), name


@pytest.mark.parametrize("tile", [32, 64, 128, 256])
def test_capacity_far_above_the_rows(tile):
    """Room for 9000 rows, 0 to 70 of them used: what lies behind is left alone."""
    rng = np.random.default_rng(tile)
    a, b = ints(rng, (9000, 64), -3, 3), ints(rng, (4, 48, 64), -3, 3)
    A, B = dev(a, torch.bfloat16), dev(b, torch.bfloat16)
    with tg.GroupPlan(4, 9000, 48, 64, F32O, tg.GEMM_LAYOUT_BT, tile_rows=tile) as p:
        for off in ([0, 0, 0, 0, 0], [0, 0, 1, 1, 1], [0, 33, 33, 69, 70]):
            C = torch.full((9000, 48), 5.0, dtype=torch.float32, device="cuda")
            grouped(p, A, B, C, i32(off))
            want = np.full((9000, 48), 5.0)
            for g in range(4):
                want[off[g]:off[g + 1]] = a[off[g]:off[g + 1]] @ b[g].T
            assert np.array_equal(host(C), want)
