"""Every branch of the rule that splits K behind adapters, on the GPU, for both layouts: the workspace says which one a
plan takes (v alone, or the partial tiles behind it)."""
import pytest
import torch

from test_lora_gpu import Case

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


@pytest.mark.parametrize("layout", ["bt", "bt_preshuffled"])
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("M,N,K,parts,splits,split", [
    (600, 6656, 2432, 4, 0, True),      # the planner's split where no tiles with more steps in flight are
    (200, 528, 9216, 4, 0, True),       # its split above K = 8192
    (200, 2048, 4096, 2, 0, False),     # up to there the plan splits, adapters do not
    (200, 528, 1152, 1, 2, True)])      # the caller's
def test_the_rule(M, N, K, parts, splits, split, out, layout):
    c = Case(M, N, K, 24, 4, layout, out, kind="bias_silu", residual=True, preact=True, splits=splits)
    partial = c.plan.workspace_bytes()
    assert partial > 0
    v = -(-parts * M * 32 * 4 // 256) * 256              # parts of K x rows x ranks, fp32
    assert c.need == v + (partial if split else 0)
    c.run()
    torch.cuda.synchronize()
    c.check()
