"""GELU and its slope behind the 8-bit checkpoint: fp32 results as exact as the library's own GELU, bf16 ones from the
shorter form of the normal distribution within the bound it states."""
import numpy as np
import pytest
import torch

import tiled_gemm_amd as tg
from test_ckpt_gpu import CODE, e4m3_table

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def stream():
    return torch.cuda.current_stream().cuda_stream


def every_code():
    """All finite e4m3 numbers under 32 scales, 2^-26 .. 2^5, one row: q, scales and their values."""
    codes = np.array([c for c in range(256) if c & 127 != 127] + [0, 0], np.uint8)
    q = np.tile(codes, 32)[None]
    scales = np.repeat(np.arange(101, 133, dtype=np.uint8), 8)[None]
    z = e4m3_table()[q] * np.repeat(2.0 ** (scales.astype(float) - 127), 32, axis=1)
    assert not np.isnan(z).any()
    return torch.from_numpy(q).cuda(), torch.from_numpy(scales).cuda(), torch.from_numpy(z).cuda()


def phi64(z):
    return 0.5 * torch.erfc(-z / 2.0 ** 0.5)


def slope64(z):
    return phi64(z) + z * torch.exp(-z * z / 2) / (2 * np.pi) ** 0.5


def test_fp32_gelu():
    """erff within 2 ulp (2^-23, halved), its argument and 1 + erf rounded: Phi within 2^-24 + 2 2^-25; one more rounding
    makes the product with z."""
    q, s, z = every_code()
    out = torch.empty(z.shape, dtype=F32, device="cuda")
    tg.gemm_ckpt_unpack(1, z.shape[1], tg.GEMM_TYPE_F32, tg.GEMM_EPI_BIAS_GELU, q.data_ptr(), s.data_ptr(), out.data_ptr(),
                        stream())
    want = z * phi64(z)
    assert bool(((out.double() - want).abs() <= z.abs() * 2.0 ** -23 + want.abs() * 2.0 ** -24).all())


@pytest.mark.parametrize("kind", ["bias_relu", "bias_silu", "bias_gelu"])
def test_fp32_gradient_equals_that_of_the_values(kind):
    """gemm_act_grad_ckpt and gemm_act_grad on the decoded values: one evaluation, the same bits."""
    q, s, z = every_code()
    z = z.clamp(-100, 100)
    keep = z.abs() < 100
    n = z.shape[1]
    d = torch.empty((1, n), device="cuda").normal_(0, 1, generator=torch.Generator(device="cuda").manual_seed(3))
    a, b = torch.empty_like(d), torch.empty_like(d)
    z32 = z.float()
    epi = tg.EPILOGUES[kind]
    tg.gemm_act_grad_ckpt(1, n, tg.GEMM_TYPE_F32, epi, d.data_ptr(), q.data_ptr(), s.data_ptr(), a.data_ptr(),
                          stream=stream())
    tg.gemm_act_grad(1, n, tg.GEMM_TYPE_F32, epi, d.data_ptr(), z32.data_ptr(), b.data_ptr(), stream=stream())
    assert torch.equal(a[keep], b[keep])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_slope_within_its_bound(dtype):
    """The bias gradient of one row of ones is the slope in fp32.  Phi within 2^-21 (bf16), z phi(z) within 2^-23 (its
    exponent's three roundings, the exponential's and the two products'), their sum rounded to 2^-24."""
    q, s, z = every_code()
    n = z.shape[1]
    d, out = torch.ones((1, n), dtype=dtype, device="cuda"), torch.empty((1, n), dtype=dtype, device="cuda")
    bias = torch.empty(n, device="cuda")
    need = tg.gemm_act_grad_workspace_bytes(1, n, 1)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    tg.gemm_act_grad_ckpt(1, n, CODE[dtype], tg.GEMM_EPI_BIAS_GELU, d.data_ptr(), q.data_ptr(), s.data_ptr(),
                          out.data_ptr(), d_bias=bias.data_ptr(), workspace=ws.data_ptr(), workspace_bytes=need,
                          stream=stream())
    err = (bias.double() - slope64(z)[0]).abs().max().item()
    print("largest error 2^%.2f" % np.log2(err))
    assert err <= (2.0 ** -21 if dtype is BF16 else 2.0 ** -23) + 2.0 ** -23 + 2.0 ** -24
