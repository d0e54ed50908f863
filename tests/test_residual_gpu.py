"""gemm_run_res / gemm_run_mx_res: bias, activation, residual and the saved
pre-activation in one epilogue, on every kernel a planner's choice reaches.

* Integer inputs, power-of-two scales, integer bias and residual: every value
  is exact in fp32, so C and the pre-activation match the definition (computed
  here in 64 bits) bit for bit.
* SiLU and GELU: |C - ref| <= L * (4e-6 S + 2^-20 (|z| + |bias|)) + 2^-20 (|act| + |r|)
  + 2^-8 |ref|: the pre-activation's bound through the activation's slope (L <=
  1.13), the fp32 addition of the residual (2^-24 of each term, inside the
  2^-20), and one rounding to bf16 (half a step, 2^-9 relative, inside the 2^-8).
* In place (the residual is C itself), captured into a graph, on another
  stream, and next to the refusals.
"""
import numpy as np
import pytest
import torch

import tiled_gemm_amd as tg
import workloads as W
from gpu_util import to_dev

pytestmark = pytest.mark.gpu

CODE = {("bf16", "f32"): tg.GEMM_BF16_OUT_F32, ("bf16", "bf16"): tg.GEMM_BF16_OUT_BF16,
        ("e4m3", "bf16"): tg.GEMM_E4M3_OUT_BF16, ("i8", "bf16"): tg.GEMM_I8_OUT_BF16,
        ("w4a8", "bf16"): tg.GEMM_W4A8_OUT_BF16}


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def as_c(x, out):
    """Values on the device in C's type."""
    t = torch.from_numpy(np.asarray(x, np.float32)).cuda()
    return t if out == "f32" else t.to(torch.bfloat16)


def sums(oracle_mod, inp, dtype, K):
    if dtype in ("i8", "w4a8"):
        return oracle_mod.gemm_bt_int(inp.A, inp.B, K, fmt=dtype)[0].astype(np.float64)
    return oracle_mod.gemm_bt(inp.A, inp.B, dtype=dtype)[0]


def call(plan, layout, A, B, C, **kw):
    s = torch.cuda.current_stream().cuda_stream
    if layout == "bt_preshuffled":
        image = torch.empty(tg.gemm_preshuffled_b_bytes(plan.handle), dtype=torch.uint8, device="cuda")
        plan.preshuffle_b(B.data_ptr(), image.data_ptr(), s)
        B = image
    plan.run_res(A.data_ptr(), B.data_ptr(), C.data_ptr(), stream=s, **kw)
    torch.cuda.synchronize()


# (dtype, out, layout, M, N, K, kernel choice): 128 x 128 tiles, skinny, the
# LDS-staged and the pipelined 256 x 256 kernels
SHAPES = [("bf16", "bf16", "bt", 130, 272, 1056, "auto"), ("bf16", "f32", "bt_preshuffled", 129, 144, 544, "auto"),
          ("e4m3", "bf16", "bt", 300, 272, 1088, "auto"), ("e4m3", "bf16", "bt_preshuffled", 65, 272, 1088, "auto"),
          ("bf16", "bf16", "bt", 1, 272, 1056, "auto"), ("bf16", "f32", "bt", 17, 48, 96, "auto"),
          ("bf16", "bf16", "bt_preshuffled", 33, 272, 1056, "auto"), ("e4m3", "bf16", "bt_preshuffled", 16, 80, 192, "auto"),
          ("i8", "bf16", "bt", 40, 272, 1088, "auto"), ("w4a8", "bf16", "bt_preshuffled", 7, 272, 1152, "auto"),
          ("bf16", "bf16", "bt", 300, 528, 1056, "tile256"), ("bf16", "f32", "bt", 257, 272, 96, "tile256"),
          ("bf16", "bf16", "bt_preshuffled", 300, 528, 1056, "tile256"),
          ("bf16", "f32", "bt_preshuffled", 300, 272, 1056, "tile256"),
          ("e4m3", "bf16", "bt", 300, 528, 1088, "tile256"), ("e4m3", "bf16", "bt_preshuffled", 300, 272, 1088, "tile256"),
          ("i8", "bf16", "bt", 300, 272, 1088, "tile256"), ("i8", "bf16", "bt_preshuffled", 300, 272, 1088, "tile256"),
          ("w4a8", "bf16", "bt", 300, 272, 1152, "tile256"), ("w4a8", "bf16", "bt_preshuffled", 300, 272, 1152, "tile256")]


@pytest.mark.parametrize("dtype,out,layout,M,N,K,kernel", SHAPES)
@pytest.mark.parametrize("kind,res,pre", [("none", True, False), ("bias_relu", True, True), ("bias", False, True)])
def test_bit_exact(oracle_mod, dtype, out, layout, M, N, K, kernel, kind, res, pre):
    print("case", dtype, out, layout, M, N, K, kernel, kind, res, pre, flush=True)
    inp = W.int_inputs(M, N, K, dtype, seed=M + N + K)
    rng = np.random.default_rng(M * 7 + N)
    acc = sums(oracle_mod, inp, dtype, K)
    sa, sb = 2.0 ** rng.integers(-2, 1, M), 2.0 ** rng.integers(-1, 2, N)
    bias = rng.integers(-8, 9, N).astype(np.float64)
    r = rng.integers(-64, 65, (M, N)).astype(np.float64)
    z = acc * sa[:, None] * sb[None, :] + (bias if kind != "none" else 0.0)
    y = (np.maximum(z, 0.0) if kind == "bias_relu" else z) + (r if res else 0.0)
    assert np.array_equal(y.astype(np.float32).astype(np.float64), y)
    R, dsa, dsb, dbias = as_c(r, out), *(torch.tensor(v, dtype=torch.float32, device="cuda") for v in (sa, sb, bias))
    C, Z = torch.full_like(R, 7.0), torch.full_like(R, 7.0)
    with tg.Plan(M, N, K, CODE[dtype, out], tg.LAYOUTS[layout], kernel=tg.KERNELS[kernel]) as p:
        call(p, layout, to_dev(inp.A), to_dev(inp.B), C, residual=R.data_ptr() if res else None,
             preact=Z.data_ptr() if pre else None, scale_a=dsa.data_ptr(), scale_a_per_row=True,
             scale_b=dsb.data_ptr(), scale_b_per_col=True, bias=dbias.data_ptr() if kind != "none" else None,
             epilogue=tg.EPILOGUES[kind])
    assert torch.equal(C, as_c(y, out))
    assert torch.equal(Z, as_c(z, out) if pre else torch.full_like(Z, 7.0))
    # in place: the residual is C itself
    if res:
        C.copy_(R)
        with tg.Plan(M, N, K, CODE[dtype, out], tg.LAYOUTS[layout], kernel=tg.KERNELS[kernel]) as p:
            call(p, layout, to_dev(inp.A), to_dev(inp.B), C, residual=C.data_ptr(), scale_a=dsa.data_ptr(),
                 scale_a_per_row=True, scale_b=dsb.data_ptr(), scale_b_per_col=True,
                 bias=dbias.data_ptr() if kind != "none" else None, epilogue=tg.EPILOGUES[kind])
        assert torch.equal(C, as_c(y, out))


@pytest.mark.parametrize("layout,kernel", [("bn", "auto"), ("bn", "tile256"), ("at", "auto"), ("at_bn", "auto")])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_bit_exact_transposed_layouts(layout, kernel, out):
    M, N, K = 136, 272, 1056
    rng = np.random.default_rng(5)
    a, b = rng.integers(-4, 5, (M, K)).astype(np.float64), rng.integers(-4, 5, (N, K)).astype(np.float64)
    r, bias = rng.integers(-64, 65, (M, N)).astype(np.float64), rng.integers(-8, 9, N).astype(np.float64)
    A = as_c(a.T if layout.startswith("at") else a, "bf16").contiguous()
    B = as_c(b.T if layout.endswith("bn") else b, "bf16").contiguous()
    R, dbias = as_c(r, out), torch.tensor(bias, dtype=torch.float32, device="cuda")
    C, Z = torch.empty_like(R), torch.empty_like(R)
    with tg.Plan(M, N, K, CODE["bf16", out], tg.LAYOUTS[layout], kernel=tg.KERNELS[kernel]) as p:
        call(p, layout, A, B, C, residual=R.data_ptr(), preact=Z.data_ptr(), bias=dbias.data_ptr(),
             epilogue=tg.GEMM_EPI_BIAS_RELU)
    z = a @ b.T + bias
    assert torch.equal(C, as_c(np.maximum(z, 0.0) + r, out)) and torch.equal(Z, as_c(z, out))


@pytest.mark.parametrize("layout", ["bn", "at", "at_bn"])
@pytest.mark.parametrize("dtype", ["e4m3", "i8"])
def test_bit_exact_transposed_8bit(layout, dtype):
    M, N, K = 272, 304, 1088
    rng = np.random.default_rng(9)
    a, b = rng.integers(-4, 5, (M, K)).astype(np.float64), rng.integers(-4, 5, (N, K)).astype(np.float64)
    r, bias = rng.integers(-64, 65, (M, N)).astype(np.float64), rng.integers(-8, 9, N).astype(np.float64)
    et = torch.float8_e4m3fn if dtype == "e4m3" else torch.int8
    A = as_c(a.T if layout.startswith("at") else a, "f32").contiguous().to(et)
    B = as_c(b.T if layout.endswith("bn") else b, "f32").contiguous().to(et)
    R, dbias = as_c(r, "bf16"), torch.tensor(bias, dtype=torch.float32, device="cuda")
    C, Z = torch.empty_like(R), torch.empty_like(R)
    with tg.Plan(M, N, K, CODE[dtype, "bf16"], tg.LAYOUTS[layout]) as p:
        call(p, layout, A, B, C, residual=R.data_ptr(), preact=Z.data_ptr(), bias=dbias.data_ptr(),
             epilogue=tg.GEMM_EPI_BIAS_RELU)
    z = a @ b.T + bias
    assert torch.equal(C, as_c(np.maximum(z, 0.0) + r, "bf16")) and torch.equal(Z, as_c(z, "bf16"))


@pytest.mark.parametrize("kind", ["bias_silu", "bias_gelu"])
@pytest.mark.parametrize("M,layout,kernel,split", [(300, "bt", "auto", 0), (300, "bt", "tile256", 0),
                                                  (20, "bt_preshuffled", "auto", 0), (300, "bt", "auto", 4),
                                                  (300, "bt_preshuffled", "tile256", 3)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_smooth_activations(oracle_mod, kind, M, layout, kernel, split, out):
    N, K = 784, 1472
    w = W.WORKLOADS["bf16_4096"]
    inp = W.make_inputs(w, M=M, N=N, K=K, seed=31)
    acc, S = oracle_mod.gemm_bt(inp.A, inp.B, dtype="bf16")
    rng = np.random.default_rng(6)
    scale = float(np.float32(2.0 / np.abs(acc).std()))
    bias = rng.normal(0, 0.5, N).astype(np.float32)
    R = as_c(rng.normal(0, 1, (M, N)), out)
    r = R.float().cpu().numpy().astype(np.float64)
    z = acc * scale + bias
    act = oracle_mod.epilogue(acc, scale, None, bias.astype(np.float64), kind)
    ds, dbias = torch.tensor([scale], device="cuda"), torch.from_numpy(bias).cuda()
    C, Z = torch.empty_like(R), torch.empty_like(R)
    with tg.Plan(M, N, K, CODE["bf16", out], tg.LAYOUTS[layout], kernel=tg.KERNELS[kernel], splits=split) as p:
        need = p.workspace_bytes()
        assert (need > 0) == (split > 0 or p.info()["ws_splits"] > 1)
        ws = torch.full((max(16, need),), 0x7F, dtype=torch.uint8, device="cuda")
        call(p, layout, to_dev(inp.A), to_dev(inp.B), C, residual=R.data_ptr(), preact=Z.data_ptr(),
             workspace=ws.data_ptr(), workspace_bytes=need, scale_a=ds.data_ptr(), bias=dbias.data_ptr(),
             epilogue=tg.EPILOGUES[kind])
        C2 = R.clone()                             # the same in place, without the workspace's split
        call(p, layout, to_dev(inp.A), to_dev(inp.B), C2, residual=C2.data_ptr(), scale_a=ds.data_ptr(),
             bias=dbias.data_ptr(), epilogue=tg.EPILOGUES[kind])
    rho = 2.0 ** -8 if out == "bf16" else 2.0 ** -24
    zb = 4e-6 * scale * S + 2.0 ** -20 * (np.abs(acc * scale) + np.abs(bias))
    ref = act + r
    bound = 1.13 * zb + 2.0 ** -20 * (np.abs(act) + np.abs(r)) + rho * np.abs(ref)
    for got in (C, C2):
        g = got.float().cpu().numpy().astype(np.float64)
        assert np.all(np.isfinite(g)) and np.all(np.abs(g - ref) <= bound)
    gz = Z.float().cpu().numpy().astype(np.float64)
    assert np.all(np.abs(gz - z) <= zb + rho * np.abs(z))


@pytest.mark.parametrize("dtype", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("M,layout", [(300, "bt"), (300, "bt_preshuffled"), (33, "bt_preshuffled")])
def test_mx(oracle_mod, dtype, M, layout):
    """The MX product's own bound (4e-6 S, products exact in fp32), the fp32
    addition of the residual, and one rounding to bf16."""
    N, K = 272, 1152
    inp = W.make_inputs(W.WORKLOADS[dtype + "_8192"], M=M, N=N, K=K, seed=3)
    acc, S = oracle_mod.gemm_bt_mx(inp.A, inp.sa_blocks, inp.B, inp.sb_blocks, K, fmt=dtype)
    code = {"mxfp8": tg.GEMM_MXFP8_OUT_BF16, "mxfp4": tg.GEMM_MXFP4_OUT_BF16}[dtype]
    s = torch.cuda.current_stream().cuda_stream
    R = as_c(np.random.default_rng(1).normal(0, np.abs(acc).std(), (M, N)), "bf16")
    C, Z = torch.empty_like(R), torch.empty_like(R)
    with tg.Plan(M, N, K, code, tg.LAYOUTS[layout]) as p:
        A, B, imgs = to_dev(inp.A), to_dev(inp.B), []
        if layout == "bt_preshuffled":
            image = torch.empty(tg.gemm_preshuffled_b_bytes(p.handle), dtype=torch.uint8, device="cuda")
            p.preshuffle_b(B.data_ptr(), image.data_ptr(), s)
            B = image
        for operand, blocks in ((0, inp.sa_blocks), (1, inp.sb_blocks)):
            src = torch.from_numpy(np.ascontiguousarray(blocks, np.uint8)).cuda()
            img = torch.empty(p.bscale_image_bytes(operand), dtype=torch.uint8, device="cuda")
            p.preshuffle_bscale(operand, src.data_ptr(), img.data_ptr(), s)
            imgs.append((src, img))
        p.run_mx_res(A.data_ptr(), imgs[0][1].data_ptr(), B.data_ptr(), imgs[1][1].data_ptr(), C.data_ptr(),
                     residual=R.data_ptr(), preact=Z.data_ptr(), stream=s)
        torch.cuda.synchronize()
    r = R.float().cpu().numpy().astype(np.float64)
    for got, ref in ((C, acc + r), (Z, acc)):
        g = got.float().cpu().numpy().astype(np.float64)
        assert np.all(np.abs(g - ref) <= 4e-6 * S + 2.0 ** -20 * (np.abs(acc) + np.abs(r)) + 2.0 ** -8 * np.abs(ref))


def test_non_finite_residual_stays_in_its_place():
    M, N, K = 70, 64, 64
    A = torch.ones((M, K), dtype=torch.bfloat16, device="cuda")
    B = torch.ones((N, K), dtype=torch.bfloat16, device="cuda")
    R = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    R[3, 5], R[69, 63], R[0, 0] = float("inf"), float("nan"), float("-inf")
    C = torch.empty_like(R)
    with tg.Plan(M, N, K, tg.GEMM_BF16_OUT_BF16, tg.GEMM_LAYOUT_BT) as p:
        call(p, "bt", A, B, C, residual=R.data_ptr())
    want = (R.float() + K).to(torch.bfloat16)
    assert torch.equal(torch.nan_to_num(C, nan=-7.0), torch.nan_to_num(want, nan=-7.0))


def test_graph_and_other_stream():
    M, N, K = 256, 2048, 4096
    g = torch.Generator(device="cuda").manual_seed(4)
    A, B, R = (torch.randn(s, generator=g, device="cuda").to(torch.bfloat16) for s in ((M, K), (N, K), (M, N)))
    C, C_eager, Z = torch.empty_like(R), torch.empty_like(R), torch.empty_like(R)
    with tg.Plan(M, N, K, tg.GEMM_BF16_OUT_BF16, tg.GEMM_LAYOUT_BT) as p:
        need = p.workspace_bytes()
        assert need > 0
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")

        def launch(C, z=None):
            p.run_res(A.data_ptr(), B.data_ptr(), C.data_ptr(), residual=R.data_ptr(),
                      preact=z.data_ptr() if z is not None else None, workspace=ws.data_ptr(), workspace_bytes=need,
                      stream=torch.cuda.current_stream().cuda_stream)
        launch(C_eager)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            launch(C, Z)
        torch.cuda.synchronize()
        assert torch.equal(C, C_eager)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            launch(C, Z)
        for _ in range(3):
            C.fill_(0.0)
            A.mul_(-1.0)                       # eager work between the replays: another input
            launch(C_eager)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(C, C_eager)
