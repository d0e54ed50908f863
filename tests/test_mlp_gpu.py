"""The mixture-of-experts layer for a few tokens on the GPU against its
definition in 64 bits.

Tolerance (derived): a product's fp32 sums are within 4e-6 of the sum of the
magnitudes (the library's bound); h is rounded once to bf16 (2^-8); activations
have slopes of at most 1.13 and are evaluated within 2^-20 |z|; the output is
rounded once (2^-8).  The errors of h go through the second product by the
magnitudes of its weights.
"""
import numpy as np
import pytest
import torch

import tiled_gemm_amd as tg

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


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
    if kind == "relu":
        return z.clamp(min=0)
    if kind == "silu":
        return z * torch.sigmoid(z)
    if kind == "gelu":
        return 0.5 * z * torch.erfc(-z / 2.0 ** 0.5)
    return z


def code(kind):
    return tg.EPILOGUES["bias" if kind == "none" else "bias_" + kind]


class Case:
    """A layer's operands on the GPU."""

    def __init__(self, groups, tokens, topk, K, N, wtype="bf16", layout="bt", gated=True, act="silu", vectors=False,
                 weighted=True, residual=True, seed=0, integers=False):
        g = self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.shape = groups, tokens, topk, K, N
        self.e4, self.layout, self.gated, self.act = wtype == "e4m3", layout, gated, act
        inner = N * (2 if gated else 1)
        f = lambda *s, std=1.0: torch.empty(s, device="cuda").normal_(0, std, generator=g)
        if integers:
            f = lambda *s, std=1.0: torch.randint(-1, 2, s, generator=g, device="cuda").float() * (
                torch.rand(s, generator=g, device="cuda") < 0.1)
        cast = torch.float8_e4m3fn if self.e4 else BF16
        self.x = f(tokens, K).to(BF16)
        self.up, self.down = f(groups, inner, K, std=K ** -0.5).to(cast), f(groups, K, N, std=N ** -0.5).to(cast)
        vec = lambda *s: (torch.rand(s, generator=g, device="cuda") + 0.5) if vectors else None
        self.up_scale, self.down_scale = vec(groups, inner), vec(groups, K)
        self.up_bias, self.down_bias = (f(groups, inner) if vectors else None), (f(groups, K) if vectors else None)
        self.ids = torch.randint(0, groups, (tokens, topk), generator=g, device="cuda").to(torch.int32)
        self.w = f(tokens, topk) if weighted else None
        self.residual = f(tokens, K).to(BF16) if residual else None
        self.out = torch.full((tokens + 1, K), 7.0, dtype=BF16, device="cuda")
        self.plan = tg.GroupMlpPlan(groups, tokens, topk, K, N, tg.GEMM_TYPE_E4M3 if self.e4 else tg.GEMM_TYPE_BF16,
                                    tg.LAYOUTS[layout], gated, code(act))
        need = self.plan.workspace_bytes()
        self.ws = torch.full((need + 64,), 0x7F, dtype=torch.uint8, device="cuda")      # garbage: never read unwritten
        self.images()

    def images(self):
        self.iu, self.id = self.up, self.down
        if self.layout == "bt_preshuffled":
            self.iu, self.id = torch.empty_like(self.up), torch.empty_like(self.down)
            self.plan.preshuffle(ptr(self.up), ptr(self.iu), ptr(self.down), ptr(self.id), stream())

    def run(self, out=None, residual=None):
        out = self.out if out is None else out
        self.plan.run(ptr(self.x), ptr(self.ids), ptr(self.iu), ptr(self.id), ptr(out), weights=ptr(self.w),
                      up_scale=ptr(self.up_scale), down_scale=ptr(self.down_scale), up_bias=ptr(self.up_bias),
                      down_bias=ptr(self.down_bias), residual=ptr(self.residual if residual is None else residual),
                      workspace=ptr(self.ws), workspace_bytes=self.plan.workspace_bytes(), stream=stream())

    def want(self):
        """(the layer, its tolerance) in 64 bits."""
        groups, tokens, topk, K, N = self.shape
        d = torch.float64
        y, tol = torch.zeros((tokens, K), dtype=d, device="cuda"), torch.zeros((tokens, K), dtype=d, device="cuda")
        for t in range(tokens):
            for j in range(topk):
                e = int(self.ids[t, j])
                if not 0 <= e < groups:
                    continue
                x, u, dn = self.x[t].to(d), self.up[e].to(d), self.down[e].to(d)
                if self.up_scale is not None:
                    u, dn = u * self.up_scale[e].to(d)[:, None], dn * self.down_scale[e].to(d)[:, None]
                z, dz = u @ x, 4e-6 * (u.abs() @ x.abs())
                if self.up_bias is not None:
                    z = z + self.up_bias[e].to(d)
                dz = dz + 2.0 ** -22 * z.abs()                       # scale and bias in fp32
                a, da = act64(z[:N], self.act), 1.13 * dz[:N] + 2.0 ** -20 * z[:N].abs()
                if self.gated:
                    h, dh = a * z[N:], da * z[N:].abs() + a.abs() * dz[N:] + da * dz[N:]
                else:
                    h, dh = a, da
                dh = dh * (1 + 2.0 ** -8) + 2.0 ** -8 * h.abs()
                o, do = dn @ h, dn.abs() @ dh + 4e-6 * (dn.abs() @ (h.abs() + dh))
                if self.down_bias is not None:
                    o = o + self.down_bias[e].to(d)
                do = do + 2.0 ** -22 * o.abs()
                w = 1.0 if self.w is None else float(self.w[t, j])
                y[t] += w * o
                tol[t] += abs(w) * (do + topk * 2.0 ** -23 * o.abs())
        if self.residual is not None:
            y += self.residual.to(d)
        return y, tol * (1 + 2.0 ** -8) + 2.0 ** -8 * y.abs() + 1e-30

    def check(self):
        tokens = self.shape[1]
        y, tol = self.want()
        err = (self.out[:tokens].double() - y).abs()
        assert bool((err <= tol).all()), "worst %.3g of the tolerance" % float((err / tol).max())
        assert bool((self.out[tokens:] == 7.0).all()) and bool((self.ws[-64:] == 0x7F).all())


@pytest.mark.parametrize("layout", ["bt", "bt_preshuffled"])
@pytest.mark.parametrize("wtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("groups,tokens,topk,K,N", [(4, 1, 1, 64, 64), (8, 3, 2, 320, 192), (5, 16, 3, 512, 64),
                                                    (6, 17, 2, 64, 704), (3, 64, 2, 192, 320), (1024, 20, 4, 64, 64)])
def test_layer(groups, tokens, topk, K, N, wtype, layout):
    for gated in (True, False):
        c = Case(groups, tokens, topk, K, N, wtype, layout, gated, vectors=wtype == "e4m3", seed=tokens)
        c.run()
        c.check()


def test_bf16_widths_of_32():
    c = Case(3, 5, 2, 96, 160, "bf16", "bt_preshuffled", vectors=True)
    c.run()
    c.check()


@pytest.mark.parametrize("act", ["none", "relu", "gelu"])
def test_activations(act):
    for gated in (True, False):
        c = Case(4, 7, 2, 128, 128, gated=gated, act=act, vectors=True, weighted=False, residual=False)
        c.run()
        c.check()


@pytest.mark.parametrize("wtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("tokens,topk", [(1, 1), (9, 4), (40, 2), (64, 1)])
def test_small_integers_are_exact_and_equal_the_chain(tokens, topk, wtype):
    """ReLU on small integers is exact in every format, so the layer equals the chain of sort, products and sum."""
    groups, K, N = 6, 256, 128
    c = Case(groups, tokens, topk, K, N, wtype, gated=False, act="relu", weighted=False, seed=tokens, integers=True)
    c.run()
    y, _ = c.want()
    assert torch.equal(c.out[:tokens].double(), y.to(BF16).double())
    rows = tokens * topk
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")
    off, tok, row = i32(groups + 1), i32(rows), i32(rows)
    up, down = c.up.to(BF16), c.down.to(BF16)
    h, o = torch.zeros((rows, N), dtype=BF16, device="cuda"), torch.zeros((rows, K), dtype=BF16, device="cuda")
    zero, out = torch.zeros((groups, N), device="cuda"), torch.zeros((tokens, K), dtype=BF16, device="cuda")
    tg.gemm_group_sort(ptr(c.ids), rows, topk, groups, ptr(off), ptr(tok), ptr(row), stream=stream())
    with tg.GroupPlan(groups, rows, N, K, tg.GEMM_BF16_OUT_BF16, tg.LAYOUTS["bt"]) as a, \
            tg.GroupPlan(groups, rows, K, N, tg.GEMM_BF16_OUT_BF16, tg.LAYOUTS["bt"]) as b:
        a.run(ptr(c.x), ptr(up), ptr(h), ptr(off), row_index=ptr(tok), a_rows=tokens, bias=ptr(zero),
              epilogue=tg.GEMM_EPI_BIAS_RELU, stream=stream())
        b.run(ptr(h), ptr(down), ptr(o), ptr(off), stream=stream())
        tg.gemm_group_combine(tokens, topk, K, tg.GEMM_TYPE_BF16, ptr(o), rows, ptr(row), ptr(out),
                              residual=ptr(c.residual), stream=stream())
        torch.cuda.synchronize()
    assert torch.equal(out, c.out[:tokens])


def test_slots_that_go_nowhere():
    c = Case(7, 12, 3, 128, 64, vectors=True)
    c.ids[0] = -1
    c.ids[1, 1] = 7
    c.ids[2] = torch.tensor([2 ** 31 - 1, -2 ** 31, 3], dtype=torch.int32)
    c.w[0] = float("nan")                       # weights of such slots are not read as factors
    c.w[1, 1] = float("inf")
    c.ids[3:, 0] = 5
    c.run()
    c.w = torch.nan_to_num(c.w, 0.0, 0.0, 0.0)
    c.check()
    # nobody at all: the residual, or zeros
    c.ids.fill_(-1)
    c.run()
    assert torch.equal(c.out[:12], c.residual)
    c.residual = None
    c.run()
    assert bool((c.out[:12] == 0).all())


def test_experts_nobody_chose_are_not_read():
    c = Case(9, 10, 2, 64, 128, vectors=True)
    c.ids.copy_(torch.where(c.ids == 4, 3, c.ids))
    for t in (c.up, c.down, c.up_scale, c.down_bias):
        t[4] = float("nan")
    c.run()
    c.check()


@pytest.mark.parametrize("tokens,topk", [(3, 8), (64, 2), (50, 64)])
def test_one_expert_named_many_times(tokens, topk):
    """More rows than a pass holds: all slots on two experts, each named several times by a token."""
    c = Case(5, tokens, topk, 64, 64, seed=3)
    c.ids.copy_(torch.where(torch.rand(c.ids.shape, generator=c.g, device="cuda") < 0.7, 1, 4).to(torch.int32))
    c.run()
    c.check()


def test_one_row_leaves_the_others_alone():
    """Infinities and NaN in one token's row reach that token's output only."""
    c = Case(3, 20, 2, 128, 64, residual=False)
    c.run()
    before = c.out.clone()
    c.x[7, 3], c.x[7, 4] = float("inf"), float("nan")
    c.run()
    keep = torch.arange(21, device="cuda") != 7
    assert torch.equal(c.out[keep], before[keep]) and bool(torch.isnan(c.out[7].float()).all())


def test_same_bits_every_run_residual_in_place_other_stream():
    c = Case(16, 33, 4, 256, 192, seed=2)
    c.run()
    torch.cuda.synchronize()
    ref = c.out.clone()
    c.check()
    side = torch.cuda.Stream()
    for _ in range(5):
        buf = torch.cat([c.residual, torch.full((1, 256), 7.0, dtype=BF16, device="cuda")])
        c.ws.fill_(0x55)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            c.run(out=buf, residual=buf)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        assert torch.equal(buf, ref)


def test_graphs_that_share_a_workspace():
    a, b = Case(12, 9, 3, 128, 64, seed=1), Case(12, 40, 2, 128, 64, seed=2)
    shared = torch.empty(max(a.ws.numel(), b.ws.numel()), dtype=torch.uint8, device="cuda")
    a.ws = b.ws = shared
    graphs = []
    for c in (a, b):
        c.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run()
        graphs.append(g)
    for r in range(4):
        for c, g in ((a, graphs[0]), (b, graphs[1]), (a, graphs[0])):
            c.ids.random_(-1, 12, generator=c.g)
            c.x.normal_(0, 1, generator=c.g)
            g.replay()
            torch.cuda.synchronize()
            got = c.out.clone()
            c.run()
            torch.cuda.synchronize()
            assert torch.equal(got, c.out)
            shared.fill_(r * 37)
    a.ws = torch.full((a.plan.workspace_bytes() + 64,), 0x7F, dtype=torch.uint8, device="cuda")
    a.run()
    a.check()
