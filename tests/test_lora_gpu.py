"""Low-rank adapters beside a shared projection on the GPU against their
definition in 64 bits.

Tolerance (derived): fp32 sums are within 4e-6 of the sum of the magnitudes (the
library's bound), for the projection, for v and for the second product; v enters
that as two bf16 numbers, within 2^-16 of it; the epilogue's terms are those of
the residual epilogue (slope 1.13, 2^-20 |z|) and the output is rounded once.
"""
import numpy as np
import pytest
import torch

import tiled_gemm_amd as tg

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def stream():
    return torch.cuda.current_stream().cuda_stream


def ptr(t):
    return None if t is None else t.data_ptr()


def act64(z, kind):
    if kind == "bias_relu":
        return z.clamp(min=0)
    if kind == "bias_silu":
        return z * torch.sigmoid(z)
    if kind == "bias_gelu":
        return 0.5 * z * torch.erfc(-z / 2.0 ** 0.5)
    return z


class Case:
    def __init__(self, M, N, K, rank, adapters, layout="bt", out=BF16, kind="none", residual=False, preact=False, seed=0,
                 integers=False, kernel="auto", splits=0, mix="any", scaled=True):
        g = self.g = torch.Generator(device="cuda").manual_seed(seed + M)
        self.shape, self.out, self.kind, self.layout = (M, N, K, rank, adapters), out, kind, layout
        f = lambda *s, std=1.0, t=BF16: torch.empty(s, device="cuda").normal_(0, std, generator=g).to(t)
        if integers:
            f = lambda *s, std=1.0, t=BF16: torch.randint(-1, 2, s, generator=g, device="cuda").to(t)
        self.a, self.b = f(M, K), f(N, K, std=K ** -0.5)
        self.down, self.up = f(adapters, rank, K, std=K ** -0.5), f(adapters, N, rank, std=rank ** -0.5)
        if integers:                                              # few entries, so that every sum stays small
            self.down *= torch.rand(self.down.shape, generator=g, device="cuda") < 0.05
            self.up *= torch.rand(self.up.shape, generator=g, device="cuda") < 0.3
        self.scale = None
        if scaled:
            self.scale = (2.0 ** torch.randint(-1, 2, (adapters,), generator=g, device="cuda")).float() if integers \
                else torch.rand(adapters, generator=g, device="cuda") + 0.5
        self.adapter = torch.randint(-1, adapters + 1, (M,), generator=g, device="cuda").to(torch.int32)
        if mix == "runs":
            self.adapter = self.adapter.sort().values.contiguous()
        elif mix == "one":
            self.adapter.fill_(adapters - 1)
        self.bias = f(N, t=F32) if kind != "none" else None
        self.residual = f(M, N, t=out) if residual else None
        self.c = torch.full((M + 1, N), 7.0, dtype=out, device="cuda")
        self.z = torch.full((M + 1, N), 7.0, dtype=out, device="cuda") if preact else None
        self.plan = tg.Plan(M, N, K, tg.GEMM_BF16_OUT_BF16 if out == BF16 else tg.GEMM_BF16_OUT_F32, tg.LAYOUTS[layout],
                            kernel=tg.KERNELS[kernel], splits=splits)
        self.image = self.b
        if layout == "bt_preshuffled":
            self.image = torch.empty_like(self.b)
            self.plan.preshuffle_b(ptr(self.b), ptr(self.image), stream())
        self.need = self.plan.lora_workspace_bytes(rank)
        self.ws = torch.full((self.need + 64,), 0xFF, dtype=torch.uint8, device="cuda")     # NaN: never read unwritten

    def run(self, c=None, residual=None):
        M, N, K, rank, adapters = self.shape
        self.plan.run_lora(ptr(self.a), ptr(self.image), ptr(self.c if c is None else c), ptr(self.adapter), adapters, rank,
                           ptr(self.down), ptr(self.up), stream=stream(), scale=ptr(self.scale),
                           residual=ptr(self.residual if residual is None else residual), preact=ptr(self.z),
                           workspace=ptr(self.ws), workspace_bytes=self.need, bias=ptr(self.bias),
                           epilogue=tg.EPILOGUES[self.kind])

    def want(self):
        """(z, y, tolerance of z, of y) in 64 bits."""
        d = torch.float64
        M, N, K, rank, adapters = self.shape
        a, b = self.a.to(d), self.b.to(d)
        z, mag = a @ b.t().contiguous(), a.abs() @ b.abs().t().contiguous()
        tol = 4e-6 * mag
        for e in sorted(set(self.adapter.tolist())):
            if not 0 <= e < adapters:
                continue
            rows = torch.nonzero(self.adapter == e).flatten()
            dn, up = self.down[e].to(d), self.up[e].to(d)
            s = 1.0 if self.scale is None else float(self.scale[e])
            v, vm = s * (a[rows] @ dn.t().contiguous()), abs(s) * (a[rows].abs() @ dn.abs().t().contiguous())
            ut = up.t().contiguous()
            z[rows] += v @ ut
            tol[rows] += (4e-6 * vm + (2.0 ** -16 + 2.0 ** -23) * v.abs()) @ ut.abs() + 4e-6 * (v.abs() @ ut.abs())
        if self.bias is not None:
            z = z + self.bias.to(d)
        y = act64(z, self.kind)
        ty = 1.13 * tol + 2.0 ** -20 * z.abs()
        if self.residual is not None:
            y = y + self.residual.to(d)
            ty = ty + 2.0 ** -23 * y.abs()
        h = HALF[self.out]
        return z, y, tol + 2.0 ** -22 * z.abs() + h * z.abs() + h * tol, ty * (1 + h) + h * y.abs()

    def check(self):
        M = self.shape[0]
        z, y, tz, ty = self.want()
        err = (self.c[:M].double() - y).abs()
        assert bool((err <= ty + 1e-30).all()), "worst %.3g of the tolerance" % float((err / (ty + 1e-30)).max())
        assert bool((self.c[M] == 7.0).all()) and bool((self.ws[self.need:] == 0xFF).all())
        if self.z is not None:
            assert bool(((self.z[:M].double() - z).abs() <= tz).all()) and bool((self.z[M] == 7.0).all())


@pytest.mark.parametrize("layout", ["bt", "bt_preshuffled"])
@pytest.mark.parametrize("M,N,K,rank,adapters", [
    (1, 48, 96, 8, 1), (1, 528, 2048, 16, 3), (16, 64, 160, 24, 20), (17, 272, 512, 40, 2), (40, 96, 4096, 16, 64),
    (64, 160, 8224, 128, 5), (64, 32, 64, 256, 64), (65, 144, 320, 16, 9), (100, 528, 1056, 64, 3), (128, 80, 64, 8, 128),
    (129, 208, 96, 32, 4), (300, 400, 544, 48, 7), (513, 304, 128, 136, 2)])
def test_adapters(M, N, K, rank, adapters, layout):
    c = Case(M, N, K, rank, adapters, layout, preact=M % 2 == 0)
    c.run()
    c.check()


@pytest.mark.parametrize("layout", ["bt", "bt_preshuffled"])
@pytest.mark.parametrize("kernel", ["tile256", "generic128"])
@pytest.mark.parametrize("mix", ["any", "runs", "one"])
def test_large_tiles(mix, kernel, layout):
    c = Case(430, 528, 608, 40, 3, layout, kernel=kernel, kind="bias_silu", residual=True, preact=True, mix=mix)
    c.run()
    c.check()


@pytest.mark.parametrize("layout", ["bt", "bt_preshuffled"])
def test_planner_large_tiles(layout):
    c = Case(2900, 3088, 192, 16, 6, layout, mix="runs", kind="bias_gelu")
    assert c.plan.info()["tile_m"] == 256
    c.run()
    c.check()


@pytest.mark.parametrize("layout", ["bt", "bt_preshuffled"])
@pytest.mark.parametrize("out", [BF16, F32])
def test_split_k(out, layout):
    c = Case(200, 1040, 2112, 32, 4, layout, out, kind="bias_silu", residual=True, preact=True, splits=3)
    assert c.plan.workspace_bytes() > 0
    c.run()
    c.check()
    assert Case(256, 4096, 8192, 16, 2, layout).plan.info()["ws_splits"] > 1     # the planner's own choice splits too


@pytest.mark.parametrize("kind", ["bias", "bias_relu", "bias_silu", "bias_gelu"])
@pytest.mark.parametrize("M", [5, 33, 70, 260])
def test_epilogues_fp32(M, kind):
    c = Case(M, 112, 352, 16, 4, "bt", F32, kind, residual=True, preact=True)
    c.run()
    c.check()


@pytest.mark.parametrize("layout", ["bt", "bt_preshuffled"])
@pytest.mark.parametrize("M", [1, 30, 64, 90, 200])
def test_small_integers_are_exact(M, layout):
    c = Case(M, 144, 512, 24, 5, layout, kind="bias_relu", residual=True, integers=True)
    c.run()
    _, y, _, _ = c.want()
    assert torch.equal(c.c[:M].double(), y.to(BF16).double())


@pytest.mark.parametrize("M", [3, 64, 100, 300])
def test_rows_without_an_adapter_equal_the_projection(M):
    """No adapter at all: the bits of gemm_run_res; some: those rows' values within its tolerance."""
    c = Case(M, 96, 256, 16, 4, "bt", F32, "bias_silu", residual=True)
    c.adapter.copy_(torch.tensor([-1, 4, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32).repeat(M)[:M])
    c.run()
    ref = torch.empty((M, 96), dtype=F32, device="cuda")
    c.plan.run_res(ptr(c.a), ptr(c.b), ptr(ref), residual=ptr(c.residual), bias=ptr(c.bias),
                   epilogue=tg.GEMM_EPI_BIAS_SILU, stream=stream())
    assert torch.equal(c.c[:M], ref)


@pytest.mark.parametrize("M,kernel", [(20, "auto"), (64, "auto"), (120, "auto"), (300, "auto"), (300, "tile256")])
def test_adapters_keep_to_their_rows(M, kernel):
    """Infinities and NaN in one adapter, or in one row, stay in its rows."""
    c = Case(M, 96, 256, 16, 3, "bt", kind="none", kernel=kernel)
    c.adapter.copy_((torch.arange(M, device="cuda") % 4 - 1).to(torch.int32))
    c.run()
    before = c.c.clone()
    c.down[1, 3, 5], c.up[1, 7, 2], c.up[1, 9] = float("inf"), float("nan"), float("-inf")
    c.run()
    other = torch.cat([c.adapter != 1, torch.ones(1, dtype=torch.bool, device="cuda")])
    assert torch.equal(c.c[other], before[other]) and bool(torch.isnan(c.c[:M][c.adapter == 1][:, 7].float()).all())
    c.scale[2], c.a[M // 2, 3] = float("nan"), float("inf")
    c.run()
    keep = other & torch.cat([c.adapter != 2, torch.ones(1, dtype=torch.bool, device="cuda")])
    keep[M // 2] = False
    assert torch.equal(c.c[keep], before[keep])


def test_scale_left_out():
    c = Case(30, 64, 128, 8, 3, scaled=False)
    c.run()
    c.check()


@pytest.mark.parametrize("M", [2, 70])
def test_no_inner_size(M):
    """K = 0: v is zero and C is the epilogue of nothing."""
    with tg.Plan(M, 64, 0, tg.GEMM_BF16_OUT_BF16, tg.LAYOUTS["bt"]) as p:
        bias = torch.arange(64, dtype=F32, device="cuda") - 20
        ids = torch.zeros(M, dtype=torch.int32, device="cuda")
        up = torch.ones((1, 64, 16), dtype=BF16, device="cuda")
        out = torch.full((M, 64), 7.0, dtype=BF16, device="cuda")
        need = p.lora_workspace_bytes(16)
        ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
        p.run_lora(0, 0, ptr(out), ptr(ids), 1, 16, 0, ptr(up), workspace=ptr(ws), workspace_bytes=need, bias=ptr(bias),
                   epilogue=tg.GEMM_EPI_BIAS_RELU, stream=stream())
        torch.cuda.synchronize()
    assert torch.equal(out, bias.clamp(min=0).to(BF16).expand(M, 64))


@pytest.mark.parametrize("M,splits", [(9, 0), (64, 0), (90, 0), (260, 3)])
def test_residual_in_place_other_stream_and_graphs(M, splits):
    c = Case(M, 272, 1120, 16, 6, "bt", kind="bias_silu", residual=True, splits=splits)
    c.run()
    torch.cuda.synchronize()
    c.check()
    ref = c.c[:M].clone()
    side = torch.cuda.Stream()
    buf = c.residual.clone()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.run(c=buf, residual=buf)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(buf, ref)
    # two graphs that share the workspace, replayed in turn with new inputs
    d = Case(M, 272, 1120, 16, 3, "bt", seed=5, splits=splits)
    d.ws = c.ws
    graphs = []
    for x in (c, d):
        x.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.run()
        graphs.append(g)
    for _ in range(3):
        for x, g in zip((c, d), graphs):
            x.a.normal_(0, 1, generator=x.g)
            x.adapter.random_(-1, 3, generator=x.g)
            g.replay()
            torch.cuda.synchronize()
            got = x.c.clone()
            x.c.fill_(7.0)
            x.run()
            torch.cuda.synchronize()
            assert torch.equal(got, x.c)
    c.check()
