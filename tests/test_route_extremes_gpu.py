"""Routing at the ends of its inputs' range: subnormal logits, biases that are
infinite or whose sums pass fp32's range.

Tolerances: those of test_route_gpu.py, fixed before the first run (ids equal)."""
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


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,kept", [(16, 1, 1), (64, 4, 2), (256, 8, 3), (512, 1, 1), (600, 4, 1)])
def test_subnormal_logits(dtype, score, E, groups, kept):
    rng = np.random.default_rng([E, groups])
    step = {"f16": 2.0 ** -24, "bf16": 2.0 ** -133, "f32": 2.0 ** -149}[dtype]
    l = rng.integers(-60, 61, (20, E)) * step
    l[::2, ::3] = rng.integers(-60, 61, (10, (E + 2) // 3)) * 2.0 ** -126
    t = torch.from_numpy(l).to(TYPES[dtype])
    kw = dict(score=score, groups=groups, topk_groups=kept, renormalize=True)
    check(t.double().numpy(), L.w4a16_route(t.cuda(), 7, **kw), 7, None, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,kept,top", [(16, 1, 1, 1), (64, 4, 2, 2), (256, 8, 3, 2), (256, 8, 3, 1), (512, 2, 1, 2), (640, 8, 3, 2)])
@pytest.mark.parametrize("kind", ["some infinite", "many infinite", "huge", "mixed"])
def test_biases_out_of_range(score, E, groups, kept, top, kind):
    rng = np.random.default_rng([E, groups, top])
    l = rng.normal(0, 1.5, (30, E)).astype(np.float32)
    l[5, ::2] = -np.inf
    b = rng.normal(0, 0.1, E).astype(np.float32)
    if kind in ("some infinite", "mixed"):
        b[rng.permutation(E)[:3]] = np.inf
        b[rng.permutation(E)[:5]] = -np.inf
    if kind == "many infinite":
        b[rng.permutation(E)[:E // 2]] = np.inf
    if kind in ("huge", "mixed"):
        # two of a group pass fp32's range together, and differ below fp32's step
        b[rng.permutation(E)[:E // 2]] = 3.0e38
        b[rng.permutation(E)[:E // 8]] = np.float32(3.4e38)
        b[rng.permutation(E)[:E // 8]] = -3.4e38
    if kind == "mixed":
        b[E // 2] = np.nan
    for renormalize in (False, True):
        kw = dict(score=score, groups=groups, topk_groups=kept, group_top=top, renormalize=renormalize)
        check(l.astype(np.float64), L.w4a16_route(torch.from_numpy(l).cuda(), 6, torch.from_numpy(b).cuda(), **kw), 6, b, **kw)
