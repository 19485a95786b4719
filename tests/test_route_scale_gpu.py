"""Scales of the routed weights that fp32 does not hold: weights are still rounded
once, and gradients meet the scale before they are rounded.

Tolerances, fixed before the first run: those of test_route_gpu.py (weights within
2^-24 of the value), and an infinity where fp32's range ends."""
import numpy as np
import pytest

from oracle import experts_ref as X
from test_route_gpu import L, TYPES, check, draw, gradient, torch
from gpu_util import note

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    note(f"[gpu] {request.node.nodeid}")


@pytest.mark.parametrize("scale", [0.1, 1.0 / 3.0, -2.6666666666666665, 1.0000000001, 7.3e-30, 0.0])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("E,topk", [(64, 6), (256, 8), (600, 20)])
def test_weights_are_rounded_once(scale, dtype, E, topk):
    t, l = draw(2000, E, dtype, seed=5)
    for score in ("softmax", "sigmoid"):
        for renormalize in (False, True):
            kw = dict(score=score, renormalize=renormalize, scale=scale)
            check(l[:40], tuple(v[:40] for v in L.w4a16_route(t.cuda(), topk, **kw)), topk, **kw)
            if scale == 0.1:
                # many weights, from the choice that the rows above confirm: each is the 64-bit product rounded once
                w, ids = (v.cpu().numpy() for v in L.w4a16_route(t.cuda(), topk, **kw))
                want = X.route_weights_ref(l, ids, **kw)
                assert (np.abs(w - want) <= 2.0 ** -24 * (1 + 1e-6) * np.abs(want)).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,topk", [(64, 6), (600, 20)])
def test_a_scale_past_fp32(score, E, topk):
    t, l = draw(9, E, "f32", seed=6)
    t[4, 3:] = float("-inf")
    w, ids = L.w4a16_route(t.cuda(), topk, score=score, renormalize=True, scale=1e39)
    want, ri = X.route_ref(t.double().numpy(), topk, score=score, renormalize=True, scale=1e39)
    assert np.array_equal(ids.cpu().numpy(), ri) and (ri[4, 3:] == -1).all()
    w, top = w.cpu().double().numpy(), float(np.finfo(np.float32).max)
    over = want > top * (1 + 2.0 ** -25)
    assert over.any() and (~over).any() and np.isinf(w[over]).all()
    assert (np.abs(w - want)[~over] <= 2.0 ** -24 * (1 + 1e-6) * want[~over]).all()
    assert not w[4, 3:].any()
    # gradients small enough to meet it
    dw = (np.random.default_rng(7).normal(size=(9, topk)) * 1e-30).astype(np.float32)
    for renormalize in (False, True):
        gradient(dw, t.double().numpy(), t, ri, "f32", score=score, renormalize=renormalize, scale=1e39)
