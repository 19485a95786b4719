"""Products far from 1 (test_lora_scales_gpu.py, with its tolerances) on the tall
tiles: adapters and tokens of all sizes, mixed, on 192- and 256-token tiles of the
forward product and on the input gradient's 128- and 256-token tiles."""
import pytest

from gpu_util import note
from test_lora_gpu import L, torch
from test_lora_scales_gpu import Scaled, run
from test_lora_tall_tiles_gpu import BACKWARD, tuned  # noqa: F401

pytestmark = pytest.mark.gpu

SIZES = ((-8, 0, 3), (0, 5, -4), (-8, 0, 0, 5), (0, -12, 3, -4, 0))


@pytest.fixture(autouse=True)
def _need_gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    note(f"[gpu] {request.node.nodeid}")


@pytest.mark.parametrize("R", [24, 128])
@pytest.mark.parametrize("mb,splits,two_pass,cb", [(4, 3, 1, 2), (6, 1, 0, 2), (6, 3, 0, 2), (8, 1, 0, 1), (8, 2, 0, 2)])
def test_forward_tiles(tuned, mb, splits, two_pass, cb, R):  # noqa: F811
    M, N, K = 64 * mb + 1, 333, 1184
    tuned("W4A16_GEMM_TILE", f"{mb},{splits},{two_pass},{cb}")
    p = L.w4a16_plan(M, N, K, 32, L.W4A16_F16, False)
    assert (p["tile_tokens"], p["tile_features"], p["splits"]) == (32 * mb, 128 * cb, splits)
    run(Scaled(M, N, K, 3, R, "mixed", *SIZES))


@pytest.mark.parametrize("shape,bm,split", BACKWARD)
def test_gradient_tiles(shape, bm, split):  # (the plans are asserted in test_lora_tall_tiles_gpu.py)
    M, N, K, R = shape
    run(Scaled(M, N, K, 3, R, "mixed", *SIZES))
