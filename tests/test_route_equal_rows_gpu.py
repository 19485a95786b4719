"""Rows of more equal keys than sixteen lanes settle, beside ordinary ones in the
same wave: each row is stored by one of the two forms, and by that alone.

Tolerances: those of test_route_gpu.py, fixed before the first run."""
import numpy as np
import pytest

from test_route_gpu import L, TYPES, check, torch
from gpu_util import note

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    note(f"[gpu] {request.node.nodeid}")


@pytest.mark.parametrize("M", [1, 2, 3, 5, 64, 1001])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,topk", [(32, 4), (100, 16), (256, 8), (512, 7)])
def test_equal_rows_beside_others(M, dtype, score, E, topk):
    rng = np.random.default_rng([M, E])
    l = rng.normal(0, 1.5, (M, E))
    kind = rng.integers(0, 5, M)
    for m in range(M):
        if kind[m] == 0:
            l[m] = 0.5                                   # all equal
        elif kind[m] == 1:
            l[m, rng.permutation(E)[:min(E, 20)]] = 9.0  # twenty are, in front
        elif kind[m] == 2:
            l[m, rng.permutation(E)[:E - 2]] = -np.inf   # two are left
        elif kind[m] == 3 and m % 2:
            l[m] = 0.5
            l[m, E // 2] = np.nan                        # equal, and NaN
    t = torch.from_numpy(l).to(TYPES[dtype])
    l = t.double().numpy()
    for bias in (None, np.full(E, 0.25, np.float32)):
        tb = None if bias is None else torch.from_numpy(bias).cuda()
        kw = dict(score=score, renormalize=True, scale=2.0)
        # more rows and slots than are written, whose values stay
        weights = torch.full((M + 2, topk), -7.0, device="cuda")
        ids = torch.full((M + 2, topk), -7, dtype=torch.int32, device="cuda")
        got = L.w4a16_route(t.cuda(), topk, tb, out=(weights[1:M + 1], ids[1:M + 1]), **kw)
        check(l, got, topk, bias, **kw)
        for edge in (weights[0], weights[-1], ids[0], ids[-1]):
            assert (edge == -7).all()
