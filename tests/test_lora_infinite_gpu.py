"""Low-rank adapters whose sums leave the finite numbers: where the definition

    v = scale sum_k x down,   z = x B^T + sum_r v up

gives an infinity, z is that infinity and not NaN (which ReLU would turn into 0),
whatever the kernel makes of v on the way.
"""
import pytest
import torch

from test_lora_gpu import Case

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
INF = float("inf")

# (M, kernel, splits): the skinny kernels, small and large tiles, split K
FORMS = [(5, "auto", 0), (40, "auto", 0), (64, "auto", 0), (100, "auto", 0), (300, "auto", 0), (300, "generic128", 0),
         (300, "tile256", 0), (300, "tile256", 2)]


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def make(form, layout="bt", out=BF16, kind="none", rank=16, K=512, **kw):
    M, kernel, splits = form
    c = Case(M, 96, K, rank, 3, layout, out, kind, kernel=kernel, splits=splits, **kw)
    c.adapter.copy_((torch.arange(M, device="cuda") % 4 - 1).to(torch.int32))
    return c


def rows_of(c, e=1):
    return torch.nonzero(c.adapter == e).flatten()


def same(got, want):
    """Equal, infinities and NaN included."""
    got, want = got.double(), want.double()
    return torch.equal(torch.isnan(got), torch.isnan(want)) and \
        torch.equal(got[~torch.isnan(want)], want[~torch.isnan(want)])


@pytest.mark.parametrize("layout", ["bt", "bt_preshuffled"])
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("kind", ["none", "bias_relu"])
@pytest.mark.parametrize("form", FORMS)
def test_infinite_v(form, kind, out, layout):
    """One infinite element of down behind a nonzero x: z is an infinity of the sign of up."""
    c = make(form, layout, out, kind, preact=True)
    c.a[:, 5] = 1.0
    c.down[1, 3, 5] = INF
    sign = torch.where(torch.arange(96, device="cuda") % 3 == 0, -1.0, 1.0)
    c.up[1, :, 3] = (sign * 0.75).to(BF16)
    c.run()
    rows = rows_of(c)
    want = (sign * INF).expand(rows.numel(), 96)
    assert same(c.z[rows], want)
    assert same(c.c[rows], want.clamp(min=0) if kind == "bias_relu" else want)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("form", FORMS)
def test_infinite_up(form, out):
    """An infinite element of up: that column is an infinity of the sign of v."""
    c = make(form, out=out)
    c.a[:, 6:] = 0.0                                  # v of bf16 products: some have no lower bits at all
    c.down[1, 2] = 0.0
    c.a[:, 4] = torch.where(torch.arange(form[0], device="cuda") % 8 < 4, 1.0, -3.0).to(BF16)
    c.down[1, 2, 4] = 0.5
    c.up[1, 7, 2] = -INF
    c.run()
    rows = rows_of(c)
    assert same(c.c[rows, 7], -INF * c.a[rows, 4].double())
    assert bool(torch.isfinite(c.c[rows][:, torch.arange(96, device="cuda") != 7].float()).all())


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("form", FORMS)
def test_v_above_the_largest_bf16(form, out):
    """A finite v that a bf16 number cannot hold: z within the usual tolerance."""
    c = make(form, out=out)
    c.b[:, 5], c.down[:, :, 5], c.up[1, :, 3] = 0.0, 0.0, c.up[1, :, 3] * 2.0 ** -100
    c.a[:, 5], c.down[1, 3], c.down[1, 3, 5] = 2.0 ** 120, 0.0, 1.0
    c.scale[1] = (2.0 - 2.0 ** -12) * 2.0 ** 7        # v = (2 - 2^-12) 2^127; 2^128 in bf16
    c.scale[0] = c.scale[2] = 1.0
    c.up[1, :, [i for i in range(16) if i != 3]] = 0.0
    c.run()
    torch.cuda.synchronize()
    c.check()


@pytest.mark.parametrize("rank", [8, 40])
@pytest.mark.parametrize("form", FORMS)
def test_infinite_x_and_padded_ranks(form, rank):
    """Ranks that fill up a block of 32 have no part in z: an infinite x with positive weights gives an infinity."""
    c = make(form, rank=rank, kind="bias_relu")
    m = form[0] // 2
    e = max(int(c.adapter[m]), 0)
    c.adapter[m] = e
    c.a[m, 5] = INF
    c.b[:, 5], c.down[e, :, 5], c.up[e] = 0.5, 0.25, c.up[e].abs() + 0.125
    c.run()
    assert bool((c.c[m] == INF).all())


@pytest.mark.parametrize("form", FORMS + [(2100, "auto", 0)])
def test_infinite_scale_and_parts_of_k(form):
    """The scale multiplies the whole sum, not parts of it that differ in sign or are zero."""
    K = 8192
    c = make(form, K=K)
    c.a.zero_()
    c.a[:, 0], c.a[:, K // 2], c.a[:, K - 1] = 1.0, 1.0, 1.0
    c.down[1, :, 0], c.down[1, :, K // 2], c.down[1, :, K - 1] = -1.0, -1.0, 4.0       # sum 2
    c.up[1] = c.up[1].abs() + 0.125
    c.scale[1] = INF
    c.run()
    rows = rows_of(c)
    assert bool((c.c[rows] == INF).all())
    # and a finite scale whose products with the parts overflow: v = 2^111
    c.a[:, 0] = c.a[:, K - 1] = 2.0 ** 20
    c.b[:, 0] = c.b[:, K - 1] = 0.0
    c.down[:, :, 0], c.down[:, :, K - 1] = -1.0, 1.0
    c.down[:, :, K // 2] = 2.0
    c.scale.fill_(2.0 ** 110)
    c.up.copy_(torch.where(c.up == 0, 1.0, torch.sign(c.up.float())) * 2.0 ** -110)
    c.run()
    rows = torch.nonzero(c.adapter >= 0).flatten()
    e = c.adapter[rows].long()
    want = c.a[rows].double() @ c.b.double().t().contiguous() + 2.0 * 2.0 ** 110 * c.up.double().sum(dim=2)[e]
    # (sums of small integers and of x B's one product a column; one rounding of the output and of the sum)
    assert bool(((c.c[rows].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -20) * want.abs() + 2.0 ** -18).all())
