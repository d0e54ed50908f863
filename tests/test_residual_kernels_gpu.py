"""The kernel families behind the residual epilogue and the grouped products
that medium sizes, long inner sizes and MX plans reach, and the ends of K x N
and K x M operands.

Inputs are small integers and powers of two, so that every value up to the
one rounding to C's type is exact and the comparisons are equalities with a
computation in 64 bits.  SiLU alone has a tolerance: its argument is exact, so
|C - ref| <= 2^-20 (|z| + |act| + |r|) + eps / 2 |ref|: the activation and the
addition in fp32 (2^-20, the epilogue's bound) and one rounding to C's type
(half a step: 2^-8 of the value in bf16, 2^-24 in fp32).
"""
import numpy as np
import pytest
import torch

import tiled_gemm_amd as tg
import workloads as W
from gpu_util import to_dev

pytestmark = pytest.mark.gpu

BF, F32O, E4 = tg.GEMM_BF16_OUT_BF16, tg.GEMM_BF16_OUT_F32, tg.GEMM_E4M3_OUT_BF16
F64 = torch.float64


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def stream():
    return torch.cuda.current_stream().cuda_stream


def etype(code):
    return torch.float8_e4m3fn if code == E4 else torch.bfloat16


def ctype(code):
    return torch.float32 if code == F32O else torch.bfloat16


class Draw:
    """Small integers and powers of two on the device, in 64 bits."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(seed)

    def ints(self, lo, hi, *shape):
        return torch.randint(lo, hi + 1, shape, generator=self.g, device="cuda").to(F64)

    def powers(self, lo, hi, *shape):
        return torch.exp2(self.ints(lo, hi, *shape))


def image(plan, B, nbytes):
    out = torch.empty(max(16, nbytes), dtype=torch.uint8, device="cuda")
    plan.preshuffle_b(B.data_ptr(), out.data_ptr(), stream())
    return out


def exactly(x, dtype):
    """x (64 bits) in C's type; x itself has to be exact in fp32."""
    assert torch.equal(x.float().double(), x)
    return x.float().to(dtype)


# ------------------------------------------------------------------ medium sizes

# 64 x 64, 64 x 128 and 128 x 128 tiles with a ring of stages, 128 x 128 with
# two (the last two rows); the smallest tiles that number at most 256 are taken
MEDIUM = [(200, 528, "auto"), (1100, 1040, "auto"), (1990, 1552, "auto"), (2100, 2064, "auto"), (200, 272, "generic128")]


def tiles(M, N, bm, bn):
    return -(-M // bm) * -(-N // bn)


def test_medium_sizes_reach_every_tile():
    counts = [[tiles(M, N, *t) for t in ((64, 64), (64, 128), (128, 128), (256, 256))] for M, N, k in MEDIUM if k == "auto"]
    first = [next((i for i, c in enumerate(row[:3]) if c <= 256), 3) for row in counts]
    assert first == [0, 1, 2, 3] and all(row[3] < 128 for row in counts)


@pytest.mark.parametrize("M,N,kernel", MEDIUM)
@pytest.mark.parametrize("code,layout", [(BF, "bt"), (F32O, "bt"), (E4, "bt"), (BF, "bt_preshuffled"), (F32O, "bt_preshuffled"),
                                         (E4, "bt_preshuffled"), (BF, "bn"), (F32O, "bn")])
@pytest.mark.parametrize("half", [False, True])
def test_medium_sizes_bit_exact(M, N, kernel, code, layout, half):
    K = (1024 if code == E4 else 512) + (64 if code == E4 else 32) * half      # whole steps, or a half-filled last one
    print("case medium", M, N, K, kernel, code, layout, flush=True)
    d = Draw(M + N + K)
    a, b, r = d.ints(-3, 3, M, K), d.ints(-3, 3, N, K), d.ints(-64, 64, M, N)
    sa, sb, bias = d.powers(-2, 0, M), d.powers(-1, 1, N), d.ints(-9, 9, N)
    A, B = a.to(etype(code)), (b.t().contiguous() if layout == "bn" else b).to(etype(code))
    R, dsa, dsb, dbias = r.to(ctype(code)), sa.float(), sb.float(), bias.float()
    z = (a @ b.t()) * sa[:, None] * sb + bias
    C, Z, D = torch.full_like(R, 7.0), torch.full_like(R, 7.0), R.clone()
    with tg.Plan(M, N, K, code, tg.LAYOUTS[layout], kernel=tg.KERNELS[kernel]) as p:
        assert p.info()["tile_m"] == 128
        if layout == "bt_preshuffled":
            B = image(p, B, tg.gemm_preshuffled_b_bytes(p.handle))
        kw = dict(scale_a=dsa.data_ptr(), scale_a_per_row=True, scale_b=dsb.data_ptr(), scale_b_per_col=True,
                  bias=dbias.data_ptr(), epilogue=tg.GEMM_EPI_BIAS_RELU, stream=stream())
        p.run_res(A.data_ptr(), B.data_ptr(), C.data_ptr(), residual=R.data_ptr(), preact=Z.data_ptr(), **kw)
        p.run_res(A.data_ptr(), B.data_ptr(), D.data_ptr(), residual=D.data_ptr(), **kw)      # in place
    assert torch.equal(Z, exactly(z, Z.dtype))
    want = exactly(z.clamp(min=0) + r, C.dtype)
    assert torch.equal(C, want) and torch.equal(D, want)


# ------------------------------------------------------------------ grouped rows: long inner sizes, several column tiles

FAMILIES = ([(c, lay, t) for c in (BF, F32O, E4) for lay in ("bt", "bt_preshuffled") for t in (32, 64, 128, 256)] +
            [(c, "bn", t) for c in (BF, F32O) for t in (32, 64, 128, 256)])


@pytest.mark.parametrize("code,layout,tile", FAMILIES)
@pytest.mark.parametrize("steps", [8, 8.5, 9])
def test_grouped_rows_long_inner_size(code, layout, tile, steps):
    K = int(steps * (128 if code == E4 else 64))
    groups, N, off = 4, 656, [3, 420, 420, 425, 690]
    M = off[-1] + 5
    print("case grouped, long K", code, layout, tile, K, flush=True)
    d = Draw(K + tile)
    a, b, bias = d.ints(-3, 3, 300, K), d.ints(-3, 3, groups, N, K), d.ints(-9, 9, groups, N)
    sa, sb = d.powers(-1, 1, 300), d.powers(-1, 1, groups, N)
    index = d.ints(0, 299, M).to(torch.int32)
    A, B = a.to(etype(code)), (b.transpose(1, 2).contiguous() if layout == "bn" else b).to(etype(code))
    z = torch.full((M, N), 6.0, dtype=F64, device="cuda")
    y = torch.full_like(z, 5.0)
    for g in range(groups):
        s = slice(off[g], off[g + 1])
        at = index[s].long()
        z[s] = (a[at] @ b[g].t()) * sa[at][:, None] * sb[g] + bias[g]
        y[s] = z[s].clamp(min=0)
    C, Z = torch.full((M, N), 5.0, dtype=ctype(code), device="cuda"), torch.full((M, N), 6.0, dtype=ctype(code), device="cuda")
    dsa, dsb, dbias, offsets = sa.float(), sb.float(), bias.float(), torch.tensor(off, dtype=torch.int32, device="cuda")
    with tg.GroupPlan(groups, M, N, K, code, tg.LAYOUTS[layout], tile_rows=tile) as p:
        if layout == "bt_preshuffled":
            B = image(p, B, p.preshuffled_b_bytes())
        p.run(A.data_ptr(), B.data_ptr(), C.data_ptr(), offsets.data_ptr(), row_index=index.data_ptr(), a_rows=300,
              preact=Z.data_ptr(), scale_a=dsa.data_ptr(), scale_a_per_row=True, scale_b=dsb.data_ptr(),
              scale_b_per_col=True, bias=dbias.data_ptr(), epilogue=tg.GEMM_EPI_BIAS_RELU, stream=stream())
    assert torch.equal(Z, exactly(z, Z.dtype)) and torch.equal(C, exactly(y, C.dtype))


@pytest.mark.parametrize("code", [BF, F32O])
def test_weight_gradient_of_many_rows(code):
    M, N, off = 520, 528, [0, 1500, 1500, 2135]
    d = Draw(11)
    a, b = d.ints(-2, 2, off[-1], M), d.ints(-2, 2, off[-1], N)
    A, B, C = a.to(torch.bfloat16), b.to(torch.bfloat16), torch.empty((3, M, N), dtype=ctype(code), device="cuda")
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    with tg.GroupPlan(3, M, N, off[-1], code, tg.GEMM_LAYOUT_AT_BN) as p:
        p.run(A.data_ptr(), B.data_ptr(), C.data_ptr(), offsets.data_ptr(), stream=stream())
    for g in range(3):
        s = slice(off[g], off[g + 1])
        assert torch.equal(C[g], exactly(a[s].t().contiguous() @ b[s], C.dtype))


# ------------------------------------------------------------------ what lies behind an operand is not used

@pytest.mark.parametrize("tile", [32, 64, 128, 256])
def test_grouped_k_by_n_ends_with_its_own_matrix(tile):
    """A last step that is half filled reads 64 K-rows where the matrix has 32
    left; the next expert's rows, all NaN here, do not reach the sums."""
    groups, N, K, off = 4, 272, 352, [0, 70, 140, 300, 301]
    d = Draw(tile)
    a, b = d.ints(-3, 3, off[-1], K), d.ints(-3, 3, groups, K, N)
    A, B = a.to(torch.bfloat16), b.to(torch.bfloat16)
    B[1], B[3] = float("nan"), float("nan")
    C = torch.empty((off[-1], N), dtype=torch.float32, device="cuda")
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    with tg.GroupPlan(groups, off[-1], N, K, F32O, tg.GEMM_LAYOUT_BN, tile_rows=tile) as p:
        p.run(A.data_ptr(), B.data_ptr(), C.data_ptr(), offsets.data_ptr(), stream=stream())
    for g in (0, 2):
        s = slice(off[g], off[g + 1])
        assert torch.equal(C[s].double(), a[s] @ b[g])
    assert bool(C[off[1]:off[2]].isnan().all()) and bool(C[off[3]:].isnan().all())


@pytest.mark.parametrize("layout", ["bn", "at", "at_bn"])
@pytest.mark.parametrize("code,kernel", [(BF, "auto"), (F32O, "tile256"), (E4, "auto")])
def test_transposed_operands_end_with_their_rows(layout, code, kernel):
    """Both operands lie at the start of larger buffers filled with NaN."""
    M, N, K = 272, 304, (352 if code != E4 else 320)       # a half-filled last step
    d = Draw(M + K)
    a, b, r = d.ints(-3, 3, M, K), d.ints(-3, 3, N, K), d.ints(-64, 64, M, N)

    def at_the_start(x):
        big = torch.full((2 * x.numel(),), float("nan"), device="cuda")
        big[:x.numel()] = x.reshape(-1)
        return big.to(etype(code))
    A, B = at_the_start(a.t() if layout.startswith("at") else a), at_the_start(b.t() if layout.endswith("bn") else b)
    R = r.to(ctype(code))
    C = torch.empty_like(R)
    with tg.Plan(M, N, K, code, tg.LAYOUTS[layout], kernel=tg.KERNELS[kernel]) as p:
        p.run_res(A.data_ptr(), B.data_ptr(), C.data_ptr(), residual=R.data_ptr(), stream=stream())
    assert torch.equal(C, exactly(a @ b.t() + r, C.dtype))


# ------------------------------------------------------------------ MX plans

@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("M,layout", [(300, "bt"), (300, "bt_preshuffled"), (33, "bt_preshuffled"), (16, "bt_preshuffled"),
                                      (33, "bt")])
@pytest.mark.parametrize("kind", ["bias", "bias_relu", "bias_silu"])
def test_mx_scales_bias_activation_in_place(oracle_mod, fmt, M, layout, kind):
    N, K = 272, 1152
    print("case mx", fmt, M, layout, kind, flush=True)
    inp = W.mx_int_inputs(M, N, K, fmt, seed=M + N)
    acc, _ = oracle_mod.gemm_bt_mx(inp.A, inp.sa_blocks, inp.B, inp.sb_blocks, K, fmt=fmt)
    acc = torch.from_numpy(np.asarray(acc, np.float64)).cuda()
    assert torch.equal(acc.float().double(), acc)
    d = Draw(M)
    sa, sb, bias, r = d.powers(-6, -4, M), d.powers(-5, -3, N), d.ints(-4, 4, N), d.ints(-8, 8, M, N)
    z = acc * sa[:, None] * sb + bias
    z32 = ((acc.float() * sa.float()[:, None]) * sb.float() + bias.float())     # the one fp32 addition, rounded
    y = {"bias": lambda: z, "bias_relu": lambda: z.clamp(min=0), "bias_silu": lambda: z * torch.sigmoid(z)}[kind]()
    R, dsa, dsb, dbias = r.to(torch.bfloat16), sa.float(), sb.float(), bias.float()
    C, Z, D = torch.empty_like(R), torch.empty_like(R), R.clone()
    code = {"mxfp8": tg.GEMM_MXFP8_OUT_BF16, "mxfp4": tg.GEMM_MXFP4_OUT_BF16}[fmt]
    with tg.Plan(M, N, K, code, tg.LAYOUTS[layout]) as p:
        A, B, imgs = to_dev(inp.A), to_dev(inp.B), []
        if layout == "bt_preshuffled":
            B = image(p, B, tg.gemm_preshuffled_b_bytes(p.handle))
        for operand, blocks in ((0, inp.sa_blocks), (1, inp.sb_blocks)):
            src = torch.from_numpy(np.ascontiguousarray(blocks, np.uint8)).cuda()
            img = torch.empty(p.bscale_image_bytes(operand), dtype=torch.uint8, device="cuda")
            p.preshuffle_bscale(operand, src.data_ptr(), img.data_ptr(), stream())
            imgs.append(img)
        kw = dict(scale_a=dsa.data_ptr(), scale_a_per_row=True, scale_b=dsb.data_ptr(), scale_b_per_col=True,
                  bias=dbias.data_ptr(), epilogue=tg.EPILOGUES[kind], stream=stream())
        p.run_mx_res(A.data_ptr(), imgs[0].data_ptr(), B.data_ptr(), imgs[1].data_ptr(), C.data_ptr(),
                     residual=R.data_ptr(), preact=Z.data_ptr(), **kw)
        p.run_mx_res(A.data_ptr(), imgs[0].data_ptr(), B.data_ptr(), imgs[1].data_ptr(), D.data_ptr(),
                     residual=D.data_ptr(), **kw)
        torch.cuda.synchronize()
    assert torch.equal(Z, z32.to(torch.bfloat16))
    assert torch.equal(C, D)
    ref = y + r
    # 2^-20 also covers the roundings of z and of the last addition (2^-24 each)
    bound = 2.0 ** -20 * (z.abs() + bias.abs() + y.abs() + r.abs()) + 2.0 ** -8 * ref.abs()
    assert bool(((C.double() - ref).abs() <= bound).all())


# ------------------------------------------------------------------ two calls at once

def test_one_plan_on_two_streams():
    groups, M, N, K = 6, 1500, 528, 512
    d = Draw(3)
    B = d.ints(-3, 3, groups, N, K).to(torch.bfloat16)
    off = torch.tensor([0, 200, 200, 700, 900, 1400, 1500], dtype=torch.int32, device="cuda")
    a = [d.ints(-3, 3, M, K).to(torch.bfloat16) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    with tg.GroupPlan(groups, M, N, K, BF, tg.GEMM_LAYOUT_BT) as p:
        want = [torch.empty((M, N), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        got = [torch.empty_like(w) for w in want]
        for x, c in zip(a, want):
            p.run(x.data_ptr(), B.data_ptr(), c.data_ptr(), off.data_ptr(), stream=stream())
        torch.cuda.synchronize()
        for _ in range(5):
            for x, c, s in zip(a, got, streams):
                p.run(x.data_ptr(), B.data_ptr(), c.data_ptr(), off.data_ptr(), stream=s.cuda_stream)
        torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want))
