"""Sizes at the ends of what the residual epilogue and the grouped operators
accept: an empty inner size, and the largest ones.  Every expected value is
exact (small integers, powers of two), so the comparisons are equalities."""
import numpy as np
import pytest
import torch

import tiled_gemm_amd as tg

pytestmark = pytest.mark.gpu

BF, F32O, E4, I8 = tg.GEMM_BF16_OUT_BF16, tg.GEMM_BF16_OUT_F32, tg.GEMM_E4M3_OUT_BF16, tg.GEMM_I8_OUT_BF16


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def stream():
    return torch.cuda.current_stream().cuda_stream


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def ctype(code):
    return torch.float32 if code == F32O else torch.bfloat16


def small_ints(shape, lo, hi, seed, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda").to(dtype)


# ------------------------------------------------------------------ K = 0
# C = act(bias) (+ residual), and nothing of A or B is read.  N gives several
# column tiles of every family.

GROUPED = ([(code, lay, tile) for code in (BF, F32O) for lay in ("bt", "bt_preshuffled", "bn") for tile in (32, 64, 128, 256)] +
           [(E4, lay, tile) for lay in ("bt", "bt_preshuffled") for tile in (32, 64, 128, 256)])


@pytest.mark.parametrize("code,layout,tile", GROUPED)
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_product_with_no_inner_size(code, layout, tile, gather):
    print("case K=0 grouped", code, layout, tile, gather, flush=True)
    groups, M, N, off = 3, 400, 528, [1, 300, 300, 390]
    dt = ctype(code)
    C = torch.full((M, N), 5.0, dtype=dt, device="cuda")
    Z = torch.full((M, N), 6.0, dtype=dt, device="cuda")
    bias = small_ints((groups, N), -9, 9, 1)
    A, B = torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda")
    index, offsets = i32(np.arange(M) % 7), i32(off)
    with tg.GroupPlan(groups, M, N, 0, code, tg.LAYOUTS[layout], tile_rows=tile) as p:
        p.run(A.data_ptr(), B.data_ptr(), C.data_ptr(), offsets.data_ptr(),
              row_index=index.data_ptr() if gather else None, a_rows=7, preact=Z.data_ptr(), bias=bias.data_ptr(),
              epilogue=tg.GEMM_EPI_BIAS_RELU, stream=stream())
    want = torch.full_like(Z, 6.0)
    for g in range(groups):
        want[off[g]:off[g + 1]] = bias[g].to(dt)
    inside = (torch.arange(M, device="cuda") >= off[0]) & (torch.arange(M, device="cuda") < off[-1])
    assert torch.equal(Z, want)
    assert torch.equal(C, torch.where(inside[:, None], want.clamp(min=0), torch.full_like(C, 5.0)))


DENSE = ([(code, lay, k) for code in (BF, F32O) for lay in ("bt", "bt_preshuffled", "bn") for k in ("auto", "tile256")] +
         [(code, lay, "auto") for code in (BF, F32O) for lay in ("at", "at_bn")] +
         [(code, lay, "auto") for code in (E4, I8) for lay in ("bt", "bt_preshuffled", "bn", "at", "at_bn")])


@pytest.mark.parametrize("code,layout,kernel", DENSE)
@pytest.mark.parametrize("M", [304, 48])
def test_product_with_no_inner_size(code, layout, kernel, M):
    print("case K=0", code, layout, kernel, M, flush=True)
    N = 528
    dt = ctype(code)
    bias = small_ints((N,), -9, 9, 2)
    R = small_ints((M, N), -64, 64, 3, dt)
    A, B = torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda")
    C, C0, Z = torch.full_like(R, 5.0), torch.full_like(R, 5.0), torch.full_like(R, 6.0)
    with tg.Plan(M, N, 0, code, tg.LAYOUTS[layout], kernel=tg.KERNELS[kernel]) as p:
        p.run_res(A.data_ptr(), B.data_ptr(), C.data_ptr(), residual=R.data_ptr(), preact=Z.data_ptr(),
                  bias=bias.data_ptr(), epilogue=tg.GEMM_EPI_BIAS_RELU, stream=stream())
        p.run_ex(A.data_ptr(), B.data_ptr(), C0.data_ptr(), bias=bias.data_ptr(), epilogue=tg.GEMM_EPI_BIAS_RELU,
                 stream=stream())
    z = bias.expand(M, N)
    assert torch.equal(Z, z.to(dt)) and torch.equal(C0, z.clamp(min=0).to(dt))
    assert torch.equal(C, (z.clamp(min=0) + R.float()).to(dt))


# ------------------------------------------------------------------ the largest rows of a weight gradient

def test_weight_gradient_with_the_longest_rows():
    """M just below 2^24: the last of a step's 64 K-rows lies 2^31 bytes behind the first."""
    M, N, rows = (1 << 24) - 8, 16, 70
    print("case weight gradient, longest rows", M, flush=True)
    A, B = small_ints((rows, M), -3, 3, 4, torch.bfloat16), small_ints((rows, N), -3, 3, 5, torch.bfloat16)
    C = torch.empty((2, M, N), dtype=torch.bfloat16, device="cuda")
    off = i32([0, 3, rows])
    with tg.GroupPlan(2, M, N, rows, BF, tg.GEMM_LAYOUT_AT_BN) as p:
        p.run(A.data_ptr(), B.data_ptr(), C.data_ptr(), off.data_ptr(), stream=stream())
    for cols in (slice(0, 4096), slice(M // 2 - 100, M // 2 + 2000), slice(M - 4000, M)):
        for g, r in enumerate((slice(0, 3), slice(3, rows))):
            want = A[r, cols].float().t().contiguous() @ B[r].float()
            assert torch.equal(C[g, cols], want.to(torch.bfloat16))


# ------------------------------------------------------------------ the most tokens

def test_combine_and_gradient_of_the_most_tokens():
    """2^24 tokens: workgroups of 256 threads for each would be 2^32 threads."""
    T, N = tg.GEMM_GROUP_MAX_ROWS, 16
    print("case most tokens", T, flush=True)
    src, dout = small_ints((T, N), -3, 3, 6, torch.bfloat16), small_ints((T, N), -3, 3, 7, torch.bfloat16)
    row = torch.randperm(T, device="cuda").to(torch.int32)
    row[::1001] = -1
    w = torch.full((T,), 2.0, device="cuda")
    out, dsrc = torch.full_like(src, 5.0), torch.full_like(src, 5.0)
    dw = torch.full((T,), 5.0, device="cuda")
    tg.gemm_group_combine(T, 1, N, tg.GEMM_TYPE_BF16, src.data_ptr(), T, row.data_ptr(), out.data_ptr(),
                          weights=w.data_ptr(), stream=stream())
    tg.gemm_group_combine_grad(T, 1, N, tg.GEMM_TYPE_BF16, dout.data_ptr(), src.data_ptr(), T, row.data_ptr(),
                               w.data_ptr(), dsrc.data_ptr(), dw.data_ptr(), stream())
    live = row >= 0
    at = row.clamp(min=0).long()
    assert torch.equal(out, torch.where(live[:, None], 2 * src[at], 0))
    want = torch.full_like(src, 5.0)
    want[at[live]] = 2 * dout[live]
    assert torch.equal(dsrc, want)
    assert torch.equal(dw, (src[at].float() * dout.float()).sum(1) * live)


def test_combine_past_the_largest_grid():
    """64 GiB of output: a workgroup for every 256 items of 8 columns would be 2^32 threads."""
    T, N = tg.GEMM_GROUP_MAX_ROWS, 2048
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GiB of device memory")
    print("case largest grid of combine", T, N, flush=True)
    src = small_ints((997, N), -3, 3, 8, torch.bfloat16)
    row = (torch.arange(T, device="cuda") % 1000).to(torch.int32)       # 997, 998, 999: rows that src does not have
    out = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    tg.gemm_group_combine(T, 1, N, tg.GEMM_TYPE_BF16, src.data_ptr(), 997, row.data_ptr(), out.data_ptr(), stream=stream())
    table = torch.cat([src, torch.zeros((3, N), dtype=torch.bfloat16, device="cuda")])
    for lo in (0, 1 << 20, (1 << 23) - 5000, (1 << 23) + 77, T - 8000):
        at = torch.arange(lo, lo + 8000, device="cuda")
        assert torch.equal(out[lo:lo + 8000], table[at % 1000])
    del out
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ no rows at all

@pytest.mark.parametrize("code", [BF, F32O])
def test_weight_gradient_without_room_for_rows(code):
    print("case weight gradient, K = 0", code, flush=True)
    A, off = torch.zeros(64, device="cuda"), i32([0, 0, 0, 0])
    C = torch.full((3, 264, 528), 9.0, dtype=ctype(code), device="cuda")
    with tg.GroupPlan(3, 264, 528, 0, code, tg.GEMM_LAYOUT_AT_BN) as p:
        p.run(A.data_ptr(), A.data_ptr(), C.data_ptr(), off.data_ptr(), stream=stream())
    assert not C.any()


@pytest.mark.parametrize("groups", [1, 3])
def test_bias_gradient_of_no_rows(groups):
    db, off = torch.full((groups, 272), 4.0, device="cuda"), i32([0] * (groups + 1))
    tg.gemm_act_grad(0, 272, tg.GEMM_TYPE_BF16, tg.GEMM_EPI_BIAS_SILU, 0, None, 0, db.data_ptr(), groups=groups,
                     offsets=off.data_ptr() if groups > 1 else None, stream=stream())
    assert not db.any()
