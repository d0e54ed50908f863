"""Edges of the few-token expert layer, the adapters and the 8-bit checkpoint on the GPU: operands past 2^32 bytes,
two calls at once, infinities and NaN behind the checkpoint, every form of the adapters' first half.

Operands past 2^32 bytes are compared with the same numbers in small operands, bit for bit: where an expert or an
adapter lies does not change its sums."""
import numpy as np
import pytest
import torch

import tiled_gemm_amd as tg
from test_ckpt_gpu import CODE, e4m3_table
from test_lora_gpu import Case as LoraCase
from test_mlp_gpu import Case as MlpCase

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.empty_cache()


def stream():
    return torch.cuda.current_stream().cuda_stream


def spread(small, count):
    """`small`'s two matrices as the first and the last of `count` (the others are never read)."""
    big = torch.empty((count,) + tuple(small.shape[1:]), dtype=small.dtype, device="cuda")
    big[0], big[-1] = small[0], small[1]
    assert big.numel() * big.element_size() > 2 ** 32
    return big


def test_layer_weights_past_32_bits():
    c = MlpCase(2, 3, 2, 4096, 4096, gated=False)
    c.ids.copy_(torch.tensor([[0, 1], [1, 0], [1, -1]], dtype=torch.int32))
    c.run()
    torch.cuda.synchronize()
    ref = c.out.clone()
    n = 130
    up, down = spread(c.up, n), spread(c.down, n)
    c.ids[c.ids == 1] = n - 1
    with tg.GroupMlpPlan(n, 3, 2, 4096, 4096, tg.GEMM_TYPE_BF16, tg.GEMM_LAYOUT_BT, False,
                         tg.EPILOGUES["bias_silu"]) as p:
        need = p.workspace_bytes()
        ws = torch.full((need,), 0x7F, dtype=torch.uint8, device="cuda")
        c.out.fill_(7.0)
        p.run(c.x.data_ptr(), c.ids.data_ptr(), up.data_ptr(), down.data_ptr(), c.out.data_ptr(), stream=stream(),
              weights=c.w.data_ptr(), residual=c.residual.data_ptr(), workspace=ws.data_ptr(), workspace_bytes=need)
        torch.cuda.synchronize()
    assert torch.equal(c.out, ref)


@pytest.mark.parametrize("M", [5, 200, 300])
def test_adapters_past_32_bits(M):
    c = LoraCase(M, 32768, 8192, 256, 2)
    c.adapter.random_(0, 2, generator=c.g)
    n = 1100
    c.scale = torch.ones(2, device="cuda")
    # (the first half's parts of K depend on whether there are several adapters, not on how many)
    c.run()
    torch.cuda.synchronize()
    ref = c.c.clone()
    c.down, c.up = spread(c.down, n), spread(c.up, n)
    c.scale = torch.ones(n, device="cuda")
    c.adapter[c.adapter == 1] = n - 1
    c.shape = c.shape[:4] + (n,)
    c.c.fill_(7.0)
    c.run()
    torch.cuda.synchronize()
    assert torch.equal(c.c, ref)


def test_checkpoint_past_32_bits():
    M, N, last = 65601, 65552, 3
    B = (N + 31) // 32
    assert M * N > 2 ** 32
    g = torch.Generator(device="cuda").manual_seed(1)
    src = torch.zeros((M, N), dtype=BF16, device="cuda")
    src[-last:].normal_(0, 3, generator=g)
    tail = src[-last:].clone()
    q, s = (torch.empty((M, n), dtype=torch.uint8, device="cuda") for n in (N, B))
    tq, ts = torch.empty_like(q[:last]), torch.empty_like(s[:last])
    t = tg.GEMM_TYPE_BF16
    tg.gemm_ckpt_pack(M, N, t, src.data_ptr(), q.data_ptr(), s.data_ptr(), stream())
    tg.gemm_ckpt_pack(last, N, t, tail.data_ptr(), tq.data_ptr(), ts.data_ptr(), stream())
    assert torch.equal(q[-last:], tq) and torch.equal(s[-last:], ts) and not bool(q[0].any())
    silu = tg.GEMM_EPI_BIAS_SILU
    out, want = torch.empty_like(src), torch.empty_like(tail)
    tg.gemm_ckpt_unpack(M, N, t, silu, q.data_ptr(), s.data_ptr(), out.data_ptr(), stream())
    tg.gemm_ckpt_unpack(last, N, t, silu, tq.data_ptr(), ts.data_ptr(), want.data_ptr(), stream())
    assert torch.equal(out[-last:], want)
    tg.gemm_act_grad_ckpt(M, N, t, silu, src.data_ptr(), q.data_ptr(), s.data_ptr(), out.data_ptr(), stream=stream())
    tg.gemm_act_grad_ckpt(last, N, t, silu, tail.data_ptr(), tq.data_ptr(), ts.data_ptr(), want.data_ptr(),
                          stream=stream())
    assert torch.equal(out[-last:], want) and not bool(out[0].any())


@pytest.mark.parametrize("kind", ["mlp", "lora"])
def test_two_calls_at_once(kind):
    """Two layers on two streams, each with its own workspace: the results of one after the other."""
    if kind == "mlp":
        cases = [MlpCase(16, 16, 4, 512, 256, seed=1), MlpCase(16, 64, 2, 512, 256, wtype="e4m3", seed=2)]
        got = lambda c: c.out
    else:
        cases = [LoraCase(300, 512, 1024, 64, 9, seed=1), LoraCase(32, 1024, 1024, 16, 9, seed=2)]
        got = lambda c: c.c
    refs = []
    for c in cases:
        c.run()
        torch.cuda.synchronize()
        c.check()
        refs.append(got(c).clone())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for r in range(4):
        for c in cases:
            got(c)[:c.shape[1 if kind == "mlp" else 0]] = 3.0
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        for _ in range(6):
            for c, s in zip(cases, streams):
                with torch.cuda.stream(s):
                    c.run()
        torch.cuda.synchronize()
        for c, ref in zip(cases, refs):
            assert torch.equal(got(c), ref)


@pytest.mark.parametrize("M,adapters,rank,mix", [(256, 20, 40, "any"), (257, 20, 40, "any"), (257, 3, 32, "runs"),
                                                 (1100, 20, 72, "any"), (1100, 20, 32, "runs"), (2100, 9, 40, "any"),
                                                 (2100, 9, 256, "runs"), (2100, 1, 40, "one"), (4500, 5, 96, "runs")])
def test_first_half_forms(M, adapters, rank, mix):
    c = LoraCase(M, 64, 1056, rank, adapters, mix=mix, preact=True)
    c.run()
    torch.cuda.synchronize()
    c.check()


@pytest.mark.parametrize("layout", ["bt", "bt_preshuffled"])
@pytest.mark.parametrize("M,kernel,splits", [(5, "auto", 0), (30, "auto", 0), (60, "auto", 0), (100, "auto", 0),
                                             (700, "auto", 0), (2100, "auto", 0), (300, "generic128", 0),
                                             (300, "tile256", 0), (300, "tile256", 2)])
def test_fp32_outputs_get_all_of_v(M, kernel, splits, layout):
    """Nothing but one product of x and one rank behind each output: v = s (x d), rounded once to fp32, bit for bit."""
    N, K, rank = 400, 512, 16
    c = LoraCase(M, N, K, rank, 3, layout=layout, out=torch.float32, kernel=kernel, splits=splits)
    c.image.zero_()
    m = torch.arange(M, device="cuda")
    x = c.a[m, m % K].clone()
    c.a.zero_()
    c.a[m, m % K] = x
    c.up.zero_()
    n = torch.arange(N, device="cuda")
    c.up[:, n, n % rank] = 1.0
    c.run()
    there = (c.adapter >= 0) & (c.adapter < 3)
    e = torch.where(there, c.adapter, 0).long()
    v = c.scale[e][:, None] * (x.float()[:, None] * c.down[e, :, m % K].float())      # (the product of two bf16 is exact)
    want = torch.where(there[:, None], v, 0.0)[:, n % rank]
    assert torch.equal(c.c[:M], want) and bool((c.c[M] == 7.0).all())


def test_adapters_with_the_planners_split():
    """K above 8192 is split where the plan splits: partial tiles behind v."""
    c = LoraCase(200, 528, 9216, 40, 4, kind="bias_silu", residual=True, preact=True)
    assert c.need > 4 * 200 * 64 * 4 + 255
    c.run()
    torch.cuda.synchronize()
    c.check()


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
@pytest.mark.parametrize("kind", ["bias_relu", "bias_silu", "bias_gelu"])
def test_grad_behind_every_code(kind, dtype):
    """All elements under the smallest, ordinary and largest scales and NaN: slopes at zero, far out, at infinity
    (448 2^127 leaves fp32) and NaN, against the formula; NaN and infinities stay in their own columns."""
    scales = np.array([[0, 100, 125, 127, 129, 131, 254, 255]], np.uint8)
    q = np.arange(256, dtype=np.uint8)[None]
    with np.errstate(invalid="ignore", over="ignore"):
        step = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(float) - 127))
        z = (e4m3_table()[q] * np.repeat(step, 32, axis=1)).astype(np.float32).astype(np.float64)
    Q, S = torch.from_numpy(q).cuda(), torch.from_numpy(scales).cuda()
    d = torch.full((1, 256), 2.0, dtype=dtype, device="cuda")
    out = torch.empty_like(d)
    tg.gemm_act_grad_ckpt(1, 256, CODE[dtype], tg.EPILOGUES[kind], d.data_ptr(), Q.data_ptr(), S.data_ptr(),
                          out.data_ptr(), stream=stream())
    got = out.double().cpu().numpy()
    t = torch.from_numpy(np.clip(z, -1e4, 1e4))            # (the slopes are 0 and 1 to fp64 from there on)
    if kind == "bias_relu":
        want = (t > 0).double()
        want[torch.isnan(t)] = 0.0                         # as gemm_act_grad: NaN is not above zero
    elif kind == "bias_silu":
        p = torch.sigmoid(t)
        want = p * (1 + t * (1 - p))
    else:
        want = 0.5 * torch.erfc(-t / 2 ** 0.5) + t * torch.exp(-t * t / 2) / (2 * np.pi) ** 0.5
    want = 2.0 * want.numpy()
    half = {BF16: 2.0 ** -8, torch.float32: 2.0 ** -24}[dtype]
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    # the slope in fp32: within 2^-19 of its largest value and of z times the logistic factor, which is below 0.28
    assert np.all(np.abs(got - want)[ok] <= (2.0 ** -18 * (1.13 + 0.28) + half * np.abs(want))[ok])
    # the other gradient, from the decoded values, agrees on what is NaN
    Z = torch.from_numpy(z).float().to(dtype).cuda()
    ref = torch.empty_like(d)
    tg.gemm_act_grad(1, 256, CODE[dtype], tg.EPILOGUES[kind], d.data_ptr(), Z.data_ptr(), ref.data_ptr(),
                     stream=stream())
    assert bool((torch.isnan(ref) == torch.isnan(out)).all())


def test_the_largest_numbers_round_to_infinity():
    """2^128 (1 - 2^-5) is the border: below, the checkpoint stays finite."""
    edge = np.float32(2.0 ** 127 * 1.9375)
    x = np.zeros((4, 32), np.float32)
    x[0, 0], x[1, 0], x[2, 0], x[3, 0] = edge, np.nextafter(edge, np.float32(0)), -edge, 3.4028235e38
    src = torch.from_numpy(x).cuda()
    q, s = torch.empty((4, 32), dtype=torch.uint8, device="cuda"), torch.empty((4, 1), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(src)
    tg.gemm_ckpt_pack(4, 32, tg.GEMM_TYPE_F32, src.data_ptr(), q.data_ptr(), s.data_ptr(), stream())
    tg.gemm_ckpt_unpack(4, 32, tg.GEMM_TYPE_F32, tg.GEMM_EPI_NONE, q.data_ptr(), s.data_ptr(), out.data_ptr(), stream())
    got = out[:, 0].tolist()
    assert got == [float("inf"), 2.0 ** 127 * 1.875, float("-inf"), float("inf")]
