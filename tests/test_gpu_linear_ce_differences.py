"""The linear cross entropy's gradients against differences of its own losses, along the gradients' signs."""
import pytest
import torch

from tests.gpu_common import DEV, build_lib
from tests.test_linear_ce_differences import STEP, agrees, both_ways, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    return build_lib()


@pytest.mark.parametrize("N,V,D", [(120, 600, 96), (40, 700, 96), (2100, 300, 96), (300, 600, 520)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_gradients(L, N, V, D, dt):
    """The joint call's, and the backward call's from the forward call's lse. A gradient in bf16 is off by 2^-8 of each element,
    mostly either way; its sum of products by far less."""
    h, w, t, wt = (x.to(DEV) for x in inputs(N, V, D))
    ws = torch.zeros(L.linear_cross_entropy_workspace_bytes(N, V, D, 2), dtype=torch.uint8, device=DEV)
    losses, lse = (torch.empty(N, device=DEV) for _ in range(2))

    def total(a, b):
        L.linear_cross_entropy_forward(a, b, t, wt, losses, lse, ws)
        return losses.double().sum().item()

    joint, alone = ([torch.empty(x.shape, dtype=dt, device=DEV) for x in (h, w)] for _ in range(2))
    L.linear_cross_entropy_forward_backward(h, w, t, wt, 1.0, losses, lse, *joint, ws)
    L.linear_cross_entropy_backward(h, w, t, wt, lse, None, *alone, ws)
    for dh, dw in (joint, alone):
        ahead, behind = both_ways(h, dh, STEP["h"])
        assert agrees(dh, total(ahead, w) - total(behind, w), ahead, behind)
        ahead, behind = both_ways(w, dw, STEP["w"] * min(1.0, (96 / D) ** 0.5 * (120 / N) ** 0.5))
        assert agrees(dw, total(h, ahead) - total(h, behind), ahead, behind)
    assert L.muon_check(ws) == L.MUON_OK
