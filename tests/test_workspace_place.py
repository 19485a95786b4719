"""A caller's workspace is refused where its pointer and size are not those of
memory on the call's device.  Nothing is launched."""
import pytest

from int4_weight_only_linear_amd import _binding as B

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("call", ["_given_workspace", "_fp8_workspace"])
def test_host_memory_is_refused(call):
    device, ws = torch.device("cuda", 0), torch.zeros(1 << 17, dtype=torch.uint8)
    with pytest.raises(ValueError, match="workspace must be on cuda:0"):
        if call == "_given_workspace":
            B._given_workspace(device, ws)
        else:
            B._fp8_workspace(device, 0, ws, None)


@pytest.mark.gpu
def test_entry_points_refuse_other_memory():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import int4_weight_only_linear_amd as L
    M, N, K, dev = 40, 256, 1152, "cuda"
    x, dy = torch.zeros((M, K), dtype=torch.bfloat16, device=dev), torch.zeros((M, N), dtype=torch.bfloat16, device=dev)
    wq, s = torch.zeros((N, K // 8), dtype=torch.int32, device=dev), torch.ones((N, K // 128), dtype=torch.bfloat16, device=dev)
    la, lb = torch.zeros((2, 8, K), dtype=torch.bfloat16, device=dev), torch.zeros((2, N, 8), dtype=torch.bfloat16, device=dev)
    ids = torch.zeros(M, dtype=torch.int32, device=dev)
    u = torch.zeros((M, 8), device=dev)
    w = torch.zeros((N, K), device=dev).to(torch.float8_e4m3fn)
    ws = torch.ones((N // 128, K // 128), device=dev)
    calls = [
        lambda b: L.w4a16_linear(x, wq, s, group_size=128, workspace=b),
        lambda b: L.w4a16_linear_dense(x, torch.zeros((N, K), dtype=torch.bfloat16, device=dev), workspace=b),
        lambda b: L.w4a16_lora_linear(x, wq, s, la, lb, ids, group_size=128, workspace=b),
        lambda b: L.w4a16_lora_backward(dy, x, u, wq, s, la, lb, ids, group_size=128, workspace=b),
        lambda b: L.w4a16_minifloat_linear(x, w, ws, workspace=b),
        lambda b: L.w4a16_minifloat_moe_linear(x, w[None].contiguous(), ws[None], ids.view(M, 1), workspace=b),
    ]
    good = torch.zeros(32 << 20, dtype=torch.uint8, device=dev)
    for call in calls:
        with pytest.raises(ValueError, match="workspace must be on"):
            call(torch.zeros(32 << 20, dtype=torch.uint8))
        with pytest.raises(ValueError, match="workspace must be contiguous"):
            call(torch.zeros(1, dtype=torch.uint8, device=dev).expand(32 << 20))
        call(good)
    torch.cuda.synchronize()
