"""The 8-bit checkpoint on the GPU against its definition in 64 bits.

Packing is exact arithmetic followed by one rounding, so its bytes must equal
those of a table search over all e4m3 numbers; an unpacked value is a number of
4 significant bits times a power of two, so it is exact in bf16 and fp32.
"""
import numpy as np
import pytest
import torch

import tiled_gemm_amd as tg

pytestmark = pytest.mark.gpu

CODE = {torch.bfloat16: tg.GEMM_TYPE_BF16, torch.float32: tg.GEMM_TYPE_F32}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}        # half a step, relative


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def stream():
    return torch.cuda.current_stream().cuda_stream


def e4m3_table():
    """The 256 e4m3 numbers: sign, 4 exponent bits (bias 7), 3 fraction bits; 0x7F and 0xFF are NaN."""
    v = np.zeros(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        x = f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        v[c] = np.nan if (c & 127) == 127 else (-x if c & 128 else x)
    return v


TABLE = e4m3_table()


def encode(x):
    """Nearest e4m3 code of each x (|x| <= 448, NaN -> 0x7F), ties to the even code."""
    mags = TABLE[:127]
    a = np.abs(x)
    hi = np.clip(np.searchsorted(mags, np.where(np.isnan(a), 0, a)), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - mags[lo], mags[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    code = code | (np.signbit(x).astype(int) << 7)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8)


def pack64(x):
    """Bytes of the checkpoint of x (fp64 holding the input's values)."""
    M, N = x.shape
    B = -(-N // 32)
    full = np.zeros((M, B * 32))
    full[:, :N] = x
    blocks = full.reshape(M, B, 32)
    top = np.where(np.isfinite(blocks), np.abs(blocks), 0.0).max(axis=2)
    s = np.full(top.shape, -127)
    for _ in range(260):                                  # the smallest s that fits, by trying
        s = np.where(top > 448.0 * 2.0 ** s.astype(float), s + 1, s)
    y = np.where(np.isfinite(blocks), blocks, np.nan) / 2.0 ** s.astype(float)[:, :, None]
    return encode(y.reshape(M, -1)[:, :N]), (s + 127).astype(np.uint8)


def value64(q, scales):
    N = q.shape[1]
    step = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(float) - 127.0))
    with np.errstate(invalid="ignore"):
        return TABLE[q] * np.repeat(step, 32, axis=1)[:, :N]


def gpu_pack(x, guard=64):
    """Packs x; q and scales sit in larger buffers whose surplus must stay as it was."""
    M, N = x.shape
    B = -(-N // 32)
    q = torch.full((M * N + guard,), 0xA5, dtype=torch.uint8, device="cuda")
    s = torch.full((M * B + guard,), 0xA5, dtype=torch.uint8, device="cuda")
    tg.gemm_ckpt_pack(M, N, CODE[x.dtype], x.data_ptr(), q.data_ptr(), s.data_ptr(), stream())
    assert bool((q[M * N:] == 0xA5).all()) and bool((s[M * B:] == 0xA5).all())
    return q[:M * N].view(M, N), s[:M * B].view(M, B)


def codes(q):
    """Elements as they compare: NaN has two codes (0x7F and 0xFF), either stands for it."""
    q = q.cpu().numpy()
    return np.where((q & 127) == 127, 127, q)


def awkward(rng, M, N):
    x = rng.normal(0, 1, (M, N)) * 2.0 ** rng.integers(-30, 30, (M, 1))
    flat = x.reshape(-1)
    at = rng.integers(0, M * N, 12)
    flat[at] = [0.0, -0.0, 448.0, np.nextafter(np.float32(448.0), np.float32(1e9)), 1.75 * 2.0 ** -40, 3.3e38,
                1e-40, np.inf, -np.inf, np.nan, 464.0, -1.0]
    x[M // 2] = 0.0                                        # blocks of nothing
    return x


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N", [(1, 16), (1, 32), (3, 48), (5, 2064), (77, 528), (130, 512), (2, 8192)])
def test_pack_bytes(M, N, dtype):
    rng = np.random.default_rng(M * 7 + N)
    x = torch.from_numpy(awkward(rng, M, N)).float().to(dtype).cuda()
    q, s = gpu_pack(x)
    wq, ws = pack64(x.double().cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), ws)
    assert np.array_equal(codes(q), wq)


def test_pack_borders():
    """One block per row whose largest magnitude sits at, below and above every border 448 2^k."""
    k = np.arange(-125, 119)
    top = np.float32(1.75) * np.exp2(k).astype(np.float32)
    rows = np.concatenate([top, np.nextafter(top, np.float32(0)), np.nextafter(top, np.float32(np.inf)),
                           np.array([1e-45, 1.1754944e-38, 3.4028235e38], np.float32)])
    x = np.zeros((rows.size, 32), np.float32)
    x[:, 7] = -rows
    x[:, 20] = rows * np.float32(0.37)
    q, s = gpu_pack(torch.from_numpy(x).cuda())
    wq, ws = pack64(x.astype(np.float64))
    assert np.array_equal(s.cpu().numpy(), ws) and np.array_equal(codes(q), wq)


def act64(z, kind):
    t = torch.from_numpy(z)
    if kind == "bias_relu":
        return torch.where(t > 0, t, 0.0).numpy()
    if kind == "bias_silu":
        return (t * torch.sigmoid(t)).numpy()
    if kind == "bias_gelu":
        return (0.5 * t * torch.erfc(-t / 2.0 ** 0.5)).numpy()
    return z


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_unpack_every_code(dtype):
    """All 256 elements under scales from the smallest to the largest and NaN, without an activation: exact."""
    scales = np.array([[0, 1, 100, 127, 130, 200, 245, 255]] * 3, np.uint8)
    q = np.stack([np.arange(256), np.arange(256)[::-1], np.arange(256) ^ 85]).astype(np.uint8)
    out = torch.full((3, 256), 7.0, dtype=dtype, device="cuda")
    Q, S = torch.from_numpy(q).cuda(), torch.from_numpy(scales).cuda()
    for kind in ("none", "bias"):
        tg.gemm_ckpt_unpack(3, 256, CODE[dtype], tg.EPILOGUES[kind], Q.data_ptr(), S.data_ptr(), out.data_ptr(), stream())
        want = torch.from_numpy(value64(q, scales)).float().to(dtype)       # exact: 4 significant bits
        np.testing.assert_array_equal(out.float().cpu().numpy(), want.float().numpy())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["bias_relu", "bias_silu", "bias_gelu"])
@pytest.mark.parametrize("M,N", [(1, 16), (3, 48), (9, 1040), (66, 512)])
def test_unpack_activation(M, N, kind, dtype):
    rng = np.random.default_rng(N)
    x = torch.from_numpy(rng.normal(0, 2, (M, N)) * 2.0 ** rng.integers(-3, 3, (M, 1))).float().cuda()
    q, s = gpu_pack(x)
    out = torch.full((M + 1, N), 7.0, dtype=dtype, device="cuda")
    tg.gemm_ckpt_unpack(M, N, CODE[dtype], tg.EPILOGUES[kind], q.data_ptr(), s.data_ptr(), out.data_ptr(), stream())
    assert bool((out[M] == 7.0).all())
    z = value64(q.cpu().numpy(), s.cpu().numpy())
    want = act64(z, kind)
    # the activation's fp32 evaluation: within 2^-20 |z| (the epilogue's term); ReLU is exact
    tol = HALF[dtype] * np.abs(want) + (0.0 if kind == "bias_relu" else 2.0 ** -20 * np.abs(z))
    assert np.all(np.abs(out[:M].double().cpu().numpy() - want) <= tol)


def slope64(z, kind):
    t = torch.from_numpy(z)
    if kind == "bias_relu":
        return (t > 0).double().numpy()
    if kind == "bias_silu":
        s = torch.sigmoid(t)
        return (s * (1 + t * torch.sigmoid(-t))).numpy()
    if kind == "bias_gelu":
        return (0.5 * torch.erfc(-t / 2.0 ** 0.5) + t * torch.exp(-t * t / 2) / (2 * np.pi) ** 0.5).numpy()
    return np.ones_like(z)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["none", "bias_relu", "bias_silu", "bias_gelu"])
@pytest.mark.parametrize("M,N,groups", [(1, 16, 1), (70, 48, 1), (133, 560, 5), (40, 1040, 64)])
def test_grad(kind, M, N, groups, dtype):
    rng = np.random.default_rng(M + N)
    x = torch.from_numpy(rng.normal(0, 2, (M, N))).float().cuda()
    q, s = gpu_pack(x)
    z = value64(q.cpu().numpy(), s.cpu().numpy())
    D = torch.from_numpy(rng.normal(0, 1, (M, N))).float().to(dtype).cuda()
    dc = D.double().cpu().numpy()
    last = max(1, M - 3)
    off = np.array([0, M]) if groups == 1 else np.sort(np.concatenate([[2, last], rng.integers(2, last + 1, groups - 1)]))
    offsets = torch.from_numpy(off.astype(np.int32)).cuda()
    out = torch.full_like(D, 4.0)
    db = torch.full((groups, N), 4.0, device="cuda")
    need = tg.gemm_act_grad_workspace_bytes(M, N, groups)
    ws = torch.full((need,), 0x7F, dtype=torch.uint8, device="cuda")
    args = dict(groups=groups, offsets=offsets.data_ptr() if groups > 1 else None, stream=stream())
    tg.gemm_act_grad_ckpt(M, N, CODE[dtype], tg.EPILOGUES[kind], D.data_ptr(), q.data_ptr(), s.data_ptr(),
                          out.data_ptr(), db.data_ptr(), workspace=ws.data_ptr(), workspace_bytes=need, **args)
    full = dc * slope64(z, kind)
    inside = np.zeros(M, bool)
    inside[off[0]:off[-1]] = True
    want = np.where(inside[:, None], full, 4.0)
    # fp32 evaluation of the slope: within 2^-19 of its largest value (1.13) and of z times it
    mag = np.abs(dc) * (1.13 + np.abs(z) * np.abs(slope64(-np.abs(z), "bias_silu")))
    tol = np.where(inside[:, None], 2.0 ** -19 * mag, 0.0)
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= tol + HALF[dtype] * np.abs(want))
    for g in range(groups):
        r = slice(off[g], off[g + 1])
        bound = (2.0 ** -19 + (off[g + 1] - off[g]) * 2.0 ** -24) * mag[r].sum(0)
        assert np.all(np.abs(db[g].double().cpu().numpy() - full[r].sum(0)) <= bound)
    # the gradient from the decoded values: the same bits (GELU: another evaluation within the same tolerance)
    Z = torch.from_numpy(z).float().to(dtype).cuda()       # exact (4 significant bits)
    ref = torch.full_like(D, 4.0)
    tg.gemm_act_grad(M, N, CODE[dtype], tg.EPILOGUES[kind], D.data_ptr(), Z.data_ptr(), ref.data_ptr(), **args)
    if kind == "bias_gelu":
        assert np.all(np.abs((ref - out).double().cpu().numpy()) <= 2 * (tol + HALF[dtype] * np.abs(want)))
    else:
        assert torch.equal(ref, out)
    # in place over d_c
    tg.gemm_act_grad_ckpt(M, N, CODE[dtype], tg.EPILOGUES[kind], D.data_ptr(), q.data_ptr(), s.data_ptr(), D.data_ptr(),
                          **args)
    m = torch.from_numpy(inside).cuda()[:, None]
    assert torch.equal(torch.where(m, D, 4.0), out)


def test_grad_against_differences():
    """The gradient of sum(d_c act(z)) at the checkpoint's values, by central differences in fp64."""
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.normal(0, 2, (6, 48))).float().cuda()
    q, s = gpu_pack(x)
    z = value64(q.cpu().numpy(), s.cpu().numpy())
    D = torch.from_numpy(rng.normal(0, 1, (6, 48))).float().cuda()
    out = torch.empty_like(D)
    for kind in ("bias_silu", "bias_gelu"):
        tg.gemm_act_grad_ckpt(6, 48, tg.GEMM_TYPE_F32, tg.EPILOGUES[kind], D.data_ptr(), q.data_ptr(), s.data_ptr(),
                              out.data_ptr(), stream=stream())
        h = 1e-5
        slope = (act64(z + h, kind) - act64(z - h, kind)) / (2 * h)
        # differences: h^2 / 6 of a third derivative below 2, and 2^-52 |z| / h of rounding
        assert np.all(np.abs(out.double().cpu().numpy() - D.double().cpu().numpy() * slope) <=
                      np.abs(D.double().cpu().numpy()) * (1e-9 + 2.0 ** -19 * (1.13 + np.abs(z))))


@pytest.mark.parametrize("M", [33, 200])
def test_checkpoint_is_an_mxfp8_operand(M):
    """x packed, its scales into the image, times packed weights: the product of the decoded values."""
    N, K = 64, 512
    rng = np.random.default_rng(M)
    x, w = (torch.from_numpy(rng.normal(0, 1, (r, K))).float().to(torch.bfloat16).cuda() for r in (M, N))
    (xq, xs), (wq, wsc) = gpu_pack(x), gpu_pack(w)
    c = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    with tg.Plan(M, N, K, tg.GEMM_MXFP8_OUT_BF16, tg.LAYOUTS["bt"]) as p:
        imgs = []
        for operand, sc in ((0, xs), (1, wsc)):
            img = torch.empty(p.bscale_image_bytes(operand), dtype=torch.uint8, device="cuda")
            p.preshuffle_bscale(operand, sc.contiguous().data_ptr(), img.data_ptr(), stream())
            imgs.append(img)
        p.run_mx(xq.data_ptr(), imgs[0].data_ptr(), wq.data_ptr(), imgs[1].data_ptr(), c.data_ptr(), stream=stream())
        torch.cuda.synchronize()
    a, b = value64(xq.cpu().numpy(), xs.cpu().numpy()), value64(wq.cpu().numpy(), wsc.cpu().numpy())
    want, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    # e4m3 products: the matrix unit's sums, 5.7e-6 of the magnitudes' sum at K = 512
    assert np.all(np.abs(c.double().cpu().numpy() - want) <= 5.7e-6 * mag + 2.0 ** -8 * np.abs(want))


def test_layer_forward_backward_through_the_checkpoint():
    """z saved by gemm_run_res, packed; d_z, d_bias and the remade output from the checkpoint; replayed as a graph
    with other inputs between the replays."""
    M, N, K = 100, 544, 256
    g = torch.Generator(device="cuda").manual_seed(5)
    bf = torch.bfloat16
    e = lambda *s, t=bf: torch.zeros(s, dtype=t, device="cuda")
    x, w, dc = e(M, K), e(N, K), e(M, N)
    bias, c, z, dz, h, db = e(N, t=torch.float32), e(M, N), e(M, N), e(M, N), e(M, N), e(1, N, t=torch.float32)
    q, s = e(M, N, t=torch.uint8), e(M, N // 32, t=torch.uint8)
    ws = e(tg.gemm_act_grad_workspace_bytes(M, N, 1), t=torch.uint8)
    plan = tg.Plan(M, N, K, tg.GEMM_BF16_OUT_BF16, tg.LAYOUTS["bt"])
    p = lambda t: t.data_ptr()
    silu = tg.GEMM_EPI_BIAS_SILU

    def step():
        st = stream()
        plan.run_res(p(x), p(w), p(c), preact=p(z), bias=p(bias), epilogue=silu, stream=st)
        tg.gemm_ckpt_pack(M, N, tg.GEMM_TYPE_BF16, p(z), p(q), p(s), st)
        tg.gemm_act_grad_ckpt(M, N, tg.GEMM_TYPE_BF16, silu, p(dc), p(q), p(s), p(dz), p(db), workspace=p(ws),
                              workspace_bytes=ws.numel(), stream=st)
        tg.gemm_ckpt_unpack(M, N, tg.GEMM_TYPE_BF16, silu, p(q), p(s), p(h), st)

    def fill():
        x.normal_(0, 1, generator=g), w.normal_(0, K ** -0.5, generator=g), dc.normal_(0, 1, generator=g)
        bias.normal_(0, 0.5, generator=g)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fill()
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        fill()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (c, z, q, s, dz, db, h)]
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (c, z, q, s, dz, db, h)):
            assert torch.equal(a, b)
        zq = value64(q.cpu().numpy(), s.cpu().numpy())
        zz = z.double().cpu().numpy()
        # each value within half an e4m3 step (2^-4 of itself, 2^-10 of the block's scale)
        step64 = np.repeat(2.0 ** (s.cpu().numpy().astype(float) - 127), 32, axis=1)
        assert np.all(np.abs(zq - zz) <= np.maximum(2.0 ** -4 * np.abs(zz), 2.0 ** -10 * step64))
        d = dc.double().cpu().numpy()
        want = d * slope64(zq, "bias_silu")
        assert np.all(np.abs(dz.double().cpu().numpy() - want) <=
                      2.0 ** -8 * np.abs(want) + 2.0 ** -19 * np.abs(d) * (1.13 + np.abs(zq)))
    plan.close()
