"""w4a16_lora_linear refuses a workspace that holds one of its inputs: it would
write over it."""
import pytest

import oracle as O
from test_lora_gpu import L, LoraCase, torch
from gpu_util import note

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    note(f"[gpu] {request.node.nodeid}")


@pytest.mark.parametrize("M", [2, 40])
@pytest.mark.parametrize("name", ["x", "wq", "scales", "zp", "bias", "la", "lb", "ids", "alpha", "out"])
def test_inputs_inside(M, name):
    case = LoraCase(M, 64, 256, 32, O.BF16, False, True, 2, 16, "mixed")
    d = case.d
    a = dict(x=d.x, wq=d.wq, scales=d.s, la=case.t_la, lb=case.t_lb, ids=case.t_ids, zp=d.zp, bias=d.bias, alpha=case.t_alpha,
             out=torch.empty((M, 64), dtype=d.x.dtype, device="cuda"), group_size=32)
    want = L.w4a16_lora_linear(**a).clone()
    n = L.w4a16_lora_workspace_size(M, 64, 256, 32, L.W4A16_BF16, True, 16)
    ws = torch.zeros(n + 65536, dtype=torch.uint8, device="cuda")
    t = a[name]
    size = t.numel() * t.element_size()
    # the input at the workspace's last 64 bytes, running out of it
    inside = ws[n - 64:n - 64 + size].view(t.dtype).view(t.shape)
    inside.copy_(t)
    with pytest.raises(L.W4A16Error, match="workspace must not overlap"):
        L.w4a16_lora_linear(**{**a, name: inside}, workspace=ws[:n])
    # behind it: taken
    behind = ws[n:n + size].view(t.dtype).view(t.shape)
    behind.copy_(t)
    ws[:n].zero_()
    got = L.w4a16_lora_linear(**{**a, name: behind}, workspace=ws[:n])
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
