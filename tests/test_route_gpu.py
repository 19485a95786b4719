"""Routing and its gradient, through the C ABI, against the float64 oracle.

Tolerances, fixed before the first run: ids are equal.  Weights are formed in 64
bits and rounded once to fp32: within 2^-24 of the value (and 2^-149), with 1e-6
of that for the 64-bit arithmetic.  Gradients are formed in fp32: within
2^-24 (16 + E / 64 + topk) of the magnitudes that the formula adds (an exponential
of 2 units, a division, products and differences; sums of E / 64 chained terms and
6 pairwise steps, of topk slots), and half a step of the logits' type."""
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


def draw(M, E, dtype, seed=0, ties=False):
    rng = np.random.default_rng([seed, M, E])
    l = rng.normal(0, 1.5, (M, E)) + rng.normal(0, 0.5, E)
    if ties:
        l = np.round(l)
    t = torch.from_numpy(l).to(TYPES[dtype])
    return t, t.double().numpy()


def check(l, got, topk, bias=None, **kw):
    w, ids = (t.cpu() for t in got)
    rw, ri = X.route_ref(l, topk, bias, **kw)
    assert np.array_equal(ids.numpy(), ri)
    w = w.double().numpy()
    assert np.array_equal(np.isnan(w), np.isnan(rw))
    err = np.abs(w - rw)[~np.isnan(rw)]
    assert (err <= 2.0 ** -24 * (1 + 1e-6) * np.abs(rw[~np.isnan(rw)]) + 2.0 ** -149).all(), float(err.max())


# (M, E, topk, groups, topk_groups, group_top)
SHAPES = [
    (1, 1, 1, 1, 1, 1), (1, 64, 6, 1, 1, 1), (5, 8, 2, 1, 1, 1), (3, 60, 4, 1, 1, 1), (67, 128, 8, 1, 1, 1), (9, 8, 8, 1, 1, 1),
    (33, 256, 8, 8, 4, 2), (4, 256, 8, 8, 4, 1), (130, 160, 6, 8, 3, 1), (7, 65, 64, 1, 1, 1), (6, 384, 7, 3, 2, 2),
    (5, 1024, 64, 64, 5, 2), (4, 1000, 10, 10, 9, 2), (11, 24, 3, 8, 2, 2), (3, 512, 9, 2, 1, 1), (1921, 60, 4, 1, 1, 1),
]


@pytest.mark.parametrize("M,E,topk,groups,kept,top", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
def test_route(M, E, topk, groups, kept, top, dtype):
    t, l = draw(M, E, dtype)
    bias = np.random.default_rng(E).normal(0, 0.05, E).astype(np.float32)
    tb = torch.from_numpy(bias).cuda()
    for score in ("softmax", "sigmoid"):
        for b in (None, bias):
            kw = dict(score=score, groups=groups, topk_groups=kept, group_top=top, renormalize=b is None, scale=2.5)
            check(l, L.w4a16_route(t.cuda(), topk, None if b is None else tb, **kw), topk, b, **kw)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_go_to_the_lower_index(dtype, score):
    t, l = draw(50, 96, dtype, ties=True)
    zero = np.zeros(96, dtype=np.float32)
    for b in (None, zero):
        for g, kept, top in ((1, 1, 1), (8, 3, 1), (8, 3, 2)):
            kw = dict(score=score, groups=g, topk_groups=kept, group_top=top)
            check(l, L.w4a16_route(t.cuda(), 8, None if b is None else torch.from_numpy(b).cuda(), **kw), 8, b, **kw)
    # all equal
    t = torch.full((3, 96), 0.25, dtype=TYPES[dtype])
    _, ids = L.w4a16_route(t.cuda(), 8, score=score, groups=8, topk_groups=2, group_top=2)
    assert ids.cpu().tolist() == [list(range(8))] * 3


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_keys_next_to_each_other(score):
    # keys that 32 bits cannot tell apart, all in 64 bits: the larger wins, equal ones keep their order
    rng = np.random.default_rng(5)
    l = np.repeat(rng.normal(0, 1, (40, 1)), 64, 1).astype(np.float32)
    b = (rng.integers(0, 4, 64) * 2.0 ** -26).astype(np.float32)
    kw = dict(score=score, renormalize=True)
    check(l.astype(np.float64), L.w4a16_route(torch.from_numpy(l).cuda(), 9, torch.from_numpy(b).cuda(), **kw), 9, b, **kw)
    up = np.repeat(l[:, :1], 64, 1)
    for i in range(64):
        up[:, i] = np.nextafter(up[:, i], np.float32(np.inf if i % 2 else -np.inf))
    b = np.zeros(64, dtype=np.float32)
    check(up.astype(np.float64), L.w4a16_route(torch.from_numpy(up).cuda(), 9, torch.from_numpy(b).cuda(), **kw), 9, b, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups", [1, 4])
def test_masked_infinite_and_nan_logits(score, biased, groups):
    t, l = draw(8, 64, "f32", seed=3)
    l[0, :] = -np.inf                                   # nothing is left
    l[1, 3:] = -np.inf                                  # three are left
    l[2, :16] = -np.inf                                 # a group is empty
    l[3, 5] = np.nan
    l[4, [7, 50]] = np.inf
    l[5, :] = -3.0e38                                   # sigmoid's scores are all zero
    l[6, :] = np.finfo(np.float32).min
    l[6, 9] = 0
    l[7, 20:] = 200.0                                   # sigmoid's scores are all one
    t = torch.from_numpy(l.astype(np.float32)).cuda()
    l = t.cpu().double().numpy()
    b = np.random.default_rng(8).normal(0, 0.05, 64).astype(np.float32) if biased else None
    if biased:
        b[40] = -np.inf
    for renormalize in (False, True):
        kw = dict(score=score, groups=groups, topk_groups=max(1, groups // 2), group_top=2 if groups > 1 else 1,
                  renormalize=renormalize)
        check(l, L.w4a16_route(t, 5, None if b is None else torch.from_numpy(b).cuda(), **kw), 5, b, **kw)


def gradient(dw, l, t, ids, dtype, **kw):
    got = L.w4a16_route_backward(torch.from_numpy(dw).cuda(), t.cuda(), torch.from_numpy(ids).cuda(), **kw)
    assert got.dtype == t.dtype
    ref, bound = X.route_backward_ref(dw, l, ids, **kw)
    got = got.cpu().double().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    fine = ~np.isnan(ref)
    M, E = l.shape
    tiny = 2.0 ** -25 if dtype == "f16" else 2.0 ** -134  # half the smallest step
    allowed = 2.0 ** -24 * (16 + E / 64 + ids.shape[1]) * bound + torch.finfo(TYPES[dtype]).eps / 2 * np.abs(ref) + tiny
    err = np.abs(got - ref)
    assert (err <= allowed)[fine].all(), float((err / allowed)[fine].max())


@pytest.mark.parametrize("M,E,topk,groups,kept,top", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
def test_gradient(M, E, topk, groups, kept, top, dtype):
    t, l = draw(M, E, dtype, seed=1)
    dw = np.random.default_rng([M, E, 7]).normal(size=(M, topk)).astype(np.float32)
    for score in ("softmax", "sigmoid"):
        _, ids = L.w4a16_route(t.cuda(), topk, score=score, groups=groups, topk_groups=kept, group_top=top)
        for renormalize in (False, True):
            gradient(dw, l, t, ids.cpu().numpy(), dtype, score=score, renormalize=renormalize, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_gradient_of_any_choice(score, renormalize):
    t, l = draw(9, 100, "f32", seed=2)
    rng = np.random.default_rng(11)
    ids = rng.integers(0, 100, (9, 6)).astype(np.int32)
    ids[0] = [3, 3, 3, 70, 70, 1]           # the same expert several times
    ids[1] = [-1, 100, 5, -2 ** 31, 2 ** 31 - 1, 6]  # out of range
    ids[2] = -1                             # none
    l[3, :] = -np.inf
    l[4, ids[4, 0]] = -np.inf
    l[5, 17] = np.nan
    l[6, :] = -3.0e38                       # sigmoid's sum is zero
    t = torch.from_numpy(l.astype(np.float32))
    gradient(rng.normal(size=(9, 6)).astype(np.float32), t.double().numpy(), t, ids, "f32", score=score,
             renormalize=renormalize, scale=1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_gradient_against_differences_of_the_kernel(score, renormalize):
    t, l = draw(3, 20, "f32", seed=4)
    t = t.cuda()
    dw = torch.from_numpy(np.random.default_rng(4).normal(size=(3, 4)).astype(np.float32)).cuda()
    kw = dict(score=score, renormalize=renormalize, scale=2.0)
    _, ids = L.w4a16_route(t, 4, **kw)
    got = L.w4a16_route_backward(dw, t, ids, **kw).double()
    h = 2.0 ** -6
    for e in range(20):
        both = []
        for sign in (1, -1):
            u = t.clone()
            u[:, e] += sign * h
            w, moved = L.w4a16_route(u, 4, **kw)
            # (the choice may change its order: weights by expert)
            full = torch.zeros((3, 20), dtype=torch.float64, device="cuda").scatter_(1, moved.long(), w.double())
            if not torch.equal(torch.sort(moved, 1).values, torch.sort(ids, 1).values):
                both = None
                break
            both.append((full.gather(1, ids.long()) * dw).sum(1))
        if both is None:
            continue
        # truncation h^2 / 6 times a third derivative below 4 * 2 * sum |dw|, rounding 2^-24 * 2 / h a term
        allowed = h * h / 6 * 8 * dw.abs().sum(1).double() + 2.0 ** -23 / h * dw.abs().sum(1).double()
        assert ((both[0] - both[1]) / (2 * h) - got[:, e]).abs().le(allowed).all()


def test_out_streams_and_graphs():
    t, l = draw(40, 256, "bf16", seed=6)
    t = t.cuda()
    kw = dict(score="sigmoid", groups=8, topk_groups=4, group_top=2, renormalize=True)
    want = L.w4a16_route(t, 8, **kw)
    dw = torch.ones((40, 8), device="cuda")
    dwant = L.w4a16_route_backward(dw, t, want[1], score="sigmoid", renormalize=True)
    out = (torch.empty((40, 8), device="cuda"), torch.empty((40, 8), dtype=torch.int32, device="cuda"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        L.w4a16_route(t, 8, out=out, **kw)
        dl = L.w4a16_route_backward(dw, t, out[1], score="sigmoid", renormalize=True)
    side.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]) and torch.equal(dl, dwant)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.w4a16_route(t, 8, out=out, **kw)
        L.w4a16_route_backward(dw, t, out[1], score="sigmoid", renormalize=True, out=dl)
    for seed in range(3):
        t.copy_(draw(40, 256, "bf16", seed=20 + seed)[0])
        g.replay()
        torch.cuda.synchronize()
        want = L.w4a16_route(t, 8, **kw)
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
        assert torch.equal(dl, L.w4a16_route_backward(dw, t, want[1], score="sigmoid", renormalize=True))
    with pytest.raises(L.W4A16Error):
        L.w4a16_route(t, 300, **kw)
    assert L.w4a16_route(t[:0], 8, **kw)[0].shape == (0, 8)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,kept,top", [(256, 8, 4, 2), (256, 8, 3, 1), (64, 4, 2, 2), (512, 2, 1, 2), (16, 16, 5, 1), (32, 16, 7, 2)])
def test_groups_next_to_each_other(score, E, groups, kept, top):
    # every group holds the same logits in an order of its own, some of them moved by a unit, and biases
    # far larger than what the groups differ by: sums that 32 bits cannot tell apart
    rng = np.random.default_rng([E, groups, top])
    per = E // groups
    l = np.empty((40, E), dtype=np.float32)
    for m in range(40):
        part = rng.normal(0, 1.5, per).astype(np.float32)
        for g in range(groups):
            l[m, g * per:(g + 1) * per] = rng.permutation(part)
        for e in rng.integers(0, E, 3) if m % 2 else ():
            l[m, e] = np.nextafter(l[m, e], np.float32(np.inf if m % 4 == 1 else -np.inf))
    kw = dict(score=score, groups=groups, topk_groups=kept, group_top=top, renormalize=True)
    topk = min(8, kept * per)
    for bias in (None, np.zeros(E, np.float32), np.tile(np.where(np.arange(per) % 2, 3.0, -3.0).astype(np.float32), groups)):
        tb = None if bias is None else torch.from_numpy(bias).cuda()
        check(l.astype(np.float64), L.w4a16_route(torch.from_numpy(l).cuda(), topk, tb, **kw), topk, bias, **kw)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("E", [32, 100, 256, 512, 513])
@pytest.mark.parametrize("topk", [1, 15, 16, 17])
def test_many_equal_keys(dtype, E, topk):
    # more equal keys than sixteen, at the front, across the last choice, and behind it
    rng = np.random.default_rng([E, topk])
    for equal in (3, 16, 17, 24, E):
        l = rng.normal(0, 1, (9, E))
        for m in range(9):
            l[m, rng.permutation(E)[:equal]] = 2.5 if m % 3 == 0 else (0.5 if m % 3 == 1 else -1.0)
        t = torch.from_numpy(l).to(TYPES[dtype])
        l = t.double().numpy()
        for score in ("softmax", "sigmoid"):
            for bias in (None, np.full(E, 0.25, np.float32)):
                tb = None if bias is None else torch.from_numpy(bias).cuda()
                check(l, L.w4a16_route(t.cuda(), topk, tb, score=score), topk, bias, score=score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_logits_far_out_and_unaligned(score):
    # scores that saturate, biases of every size, and a bias that starts 4 bytes behind a 16-byte piece
    rng = np.random.default_rng(8)
    l = (rng.normal(0, 60, (64, 128)) * rng.choice([1e-3, 1, 10], (64, 1))).astype(np.float32)
    b = (rng.normal(0, 1, 129) * 10.0 ** rng.integers(-8, 9, 129)).astype(np.float32)
    tb = torch.from_numpy(b).cuda()[1:]
    assert tb.data_ptr() % 16 == 4
    for g, kept, top in ((1, 1, 1), (8, 3, 1), (8, 3, 2)):
        kw = dict(score=score, groups=g, topk_groups=kept, group_top=top)
        check(l.astype(np.float64), L.w4a16_route(torch.from_numpy(l).cuda(), 8, tb, **kw), 8, b[1:], **kw)
