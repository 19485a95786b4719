"""The gradient of renormalised weights whose scores are all far below one: the
scores may lie outside fp32's range while their shares, and the gradient, are
ordinary numbers.

Tolerances, fixed before the first run.  The shares, the mean and their products
are formed in 64 bits and rounded once to fp32, after the product of a slot's
gradient and the scale was (2^-24 of the magnitudes that the formula adds, twice,
and 1e-6 of that for the 64-bit arithmetic), and once more to the logits' type.
Slots of one expert are added in fp32: 2^-24 for each."""
import numpy as np
import pytest

from oracle import experts_ref as X
from gpu_util import note

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import int4_weight_only_linear_amd as L  # noqa: E402

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _need_gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    note(f"[gpu] {request.node.nodeid}")


def check(dw, t, ids, score, scale=1.0):
    kw = dict(score=score, renormalize=True, scale=scale)
    got = L.w4a16_route_backward(torch.from_numpy(dw).cuda(), t.cuda(), torch.from_numpy(ids).cuda(), **kw).cpu().double().numpy()
    l = t.double().numpy()
    ref, bound = X.route_backward_ref(dw, l, ids, **kw)
    E, tiny = l.shape[1], 2.0 ** -25 if t.dtype == torch.float16 else 2.0 ** -134
    allowed = 2.0 ** -24 * (2 + ids.shape[1]) * (1 + 1e-6) * bound + torch.finfo(t.dtype).eps / 2 * np.abs(ref) + tiny
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= allowed).all(), float((np.abs(got - ref) / allowed).max())
    # experts that no slot names have none, whatever their scores
    named = np.zeros(l.shape, dtype=bool)
    for m in range(len(ids)):
        named[m, [e for e in ids[m] if 0 <= e < E]] = True
    assert not got[~named].any()
    return ref


@pytest.mark.parametrize("level", [-80, -88, -88.5, -95, -104, -110, -300, -700])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("E,topk", [(20, 1), (64, 4), (256, 8), (100, 16), (300, 17), (1000, 64)])
def test_sigmoid_of_far_negative_logits(level, dtype, E, topk):
    rng = np.random.default_rng([E, topk, -int(level * 2)])
    t = torch.from_numpy(level + rng.normal(0, 1, (9, E))).to(TYPES[dtype])
    t[3, ::2] = float("-inf")
    dw = rng.normal(size=(9, topk)).astype(np.float32)
    w, ids = L.w4a16_route(t.cuda(), topk, score="sigmoid", renormalize=True)
    assert (w.sum(1) - 1).abs().max() < 1e-5
    ref = check(dw, t, ids.cpu().numpy(), "sigmoid", 2.5)
    if topk > 1:
        assert (np.abs(ref).max(1) > 1e-3).all()


@pytest.mark.parametrize("level", [-80, -88, -95, -104, -110, -300, -700])
@pytest.mark.parametrize("E,topk", [(20, 1), (64, 4), (256, 8), (300, 17)])
def test_softmax_of_experts_far_below_the_largest(level, E, topk):
    # the bias takes experts whose scores are next to nothing beside the largest logit's
    rng = np.random.default_rng([E, topk, -level])
    l = rng.normal(0, 1, (9, E))
    bias = np.zeros(E, dtype=np.float32)
    low = rng.permutation(E)[:topk + 2]
    l[:, low] += level
    bias[low] = 10 + rng.normal(0, 1, len(low))
    t = torch.from_numpy(l.astype(np.float32))
    w, ids = L.w4a16_route(t.cuda(), topk, torch.from_numpy(bias).cuda(), renormalize=True)
    assert np.isin(ids.cpu().numpy(), low).all() and (w.sum(1) - 1).abs().max() < 1e-5
    ref = check(rng.normal(size=(9, topk)).astype(np.float32), t, ids.cpu().numpy(), "softmax")
    if topk > 1:
        assert (np.abs(ref).max(1) > 1e-3).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scores_that_are_zero_and_infinite_logits(score):
    rng = np.random.default_rng(1)
    l = rng.normal(0, 1, (7, 40)).astype(np.float32)
    ids = np.stack([rng.permutation(40)[:6] for _ in range(7)]).astype(np.int32)
    l[0] -= 800                              # sigmoid's 64-bit scores are zero, and so are the weights
    l[1, ids[1]] -= 800                      # softmax's chosen ones are
    l[2, [3, 30]] = np.inf
    ids[2, :2] = [3, 30]                     # two infinite ones, among others
    l[3, 5] = np.inf
    ids[3, ids[3] == 5] = 6                  # an infinite one that is not chosen
    ids[4] = [7, 7, 7, 8, -1, 40]
    l[5, ids[5, :5]] = -np.inf               # one is left
    l[6, ids[6]] = -np.inf                   # none is
    check(rng.normal(size=(7, 6)).astype(np.float32), torch.from_numpy(l), ids, score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_small_scores_against_differences_of_the_kernel(score):
    rng = np.random.default_rng(6)
    E, topk = 24, 4
    l = np.round(rng.normal(0, 1, (3, E)) * 256) / 256
    bias = np.zeros(E, dtype=np.float32)
    if score == "softmax":
        l[:, :8] -= 110
        bias[:8] = 10 + np.arange(8)
    else:
        l -= 110
        bias[:8] = np.arange(1, 9)
    t, tb = torch.from_numpy(l.astype(np.float32)).cuda(), torch.from_numpy(bias).cuda()
    dw = torch.from_numpy(rng.normal(size=(3, topk)).astype(np.float32)).cuda()
    kw = dict(score=score, renormalize=True, scale=2.0)
    _, ids = L.w4a16_route(t, topk, tb, **kw)
    got = L.w4a16_route_backward(dw, t, ids, **kw).double()
    assert got.abs().amax(1).min() > 1e-3
    h = 2.0 ** -6
    for e in range(E):
        both = []
        for sign in (1, -1):
            u = t.clone()
            u[:, e] += sign * h
            w, moved = L.w4a16_route(u, topk, tb, **kw)
            assert torch.equal(moved, ids)  # (the biases lie 1 apart)
            both.append((w.double() * dw).sum(1))
        # truncation h^2 / 6 times a third derivative below 4 * 2 * sum |dw|, rounding 2^-24 * 2 / h a term
        allowed = (h * h / 6 * 8 + 2.0 ** -23 / h) * dw.abs().sum(1).double()
        assert ((both[0] - both[1]) / (2 * h) - got[:, e]).abs().le(allowed).all()
