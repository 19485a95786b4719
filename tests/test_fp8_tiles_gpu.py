"""The 8-bit products' tiles of every height (32, 64, 96 and 128 tokens), each
with its plan asserted, so that a change of the planner cannot take the cover
away: ragged edges, K ranges, N that is no multiple of 4, values that are not
finite, scales of zero, and experts whose last tile is a part of one; both kinds
of scales, both directions.

Tolerances, fixed before the first run: on a sample of the outputs (the tiles'
edges, the ends and others), as in test_fp8_gpu.py: half a step of their type and
the oracle's slack.  On all outputs, against a product in fp32 of the same
values, the linear layer's (gpu_util.TOL of max|y|)."""
import numpy as np
import pytest

from oracle import experts_ref as X
from fp8_cases import TYPES, Weights, edges, planned, values  # noqa: F401  (planned: a fixture)
from gpu_util import TOL, note
from test_fp8_gpu import check

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import int4_weight_only_linear_amd as L  # noqa: E402


@pytest.fixture(autouse=True)
def _need_gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    note(f"[gpu] {request.node.nodeid}")


def cuda(i):
    return torch.from_numpy(np.asarray(i)).cuda()


def bits(t):
    return t.contiguous().view(torch.int16)


def all_outputs(y, x, layer, dtype, bias=None, weights=None, e=None):
    """Every output against the fp32 product of the quantised values."""
    c, s = L.w4a16_minifloat_quantize(x)
    xd = (c.float() * s.float().repeat_interleave(128, 1)[:, :c.shape[1]])[:, :layer.K].contiguous()
    full = xd @ layer.dense(e).contiguous()
    if bias is not None:
        full = full + bias.float()
    if weights is not None:
        full = full * weights
    assert (y.float() - full).abs().max() <= TOL[0 if dtype == "f16" else 1] * full.abs().max()


# (M, N, K, tile height, K ranges); transposed: N up to a multiple of 16, K less 3
TILES = [
    (31, 257, 144, 32, 1), (129, 131, 400, 32, 1), (67, 131, 4096, 32, 8), (9, 130, 2048, 32, 4), (96, 202, 2304, 32, 3),
    (1000, 3983, 400, 64, 1), (801, 3999, 144, 64, 1), (33, 8195, 5136, 64, 6),
    (1100, 3999, 400, 96, 1), (1345, 4000, 272, 96, 1), (67, 8195, 3600, 96, 4),
    (1700, 3999, 400, 128, 1), (1793, 3970, 144, 128, 1), (100, 8195, 3600, 128, 4),
]


@pytest.mark.parametrize("M,N,K,height,splits", TILES)
@pytest.mark.parametrize("e8m0", [False, True])
@pytest.mark.parametrize("transpose", [False, True])
def test_tiles(M, N, K, height, splits, e8m0, transpose, planned):  # noqa: F811
    rng = np.random.default_rng([M, N, K])
    if transpose:
        N, K = (N + 15) // 16 * 16, K - 3
    dtype = "f16" if (M + e8m0) % 2 else "bf16"
    layer = Weights(rng, N, K, transpose, e8m0, bias=dtype)
    x = values(rng, M, K, dtype)
    buf = torch.full((M * N + 2048,), -7.0, dtype=TYPES[dtype], device="cuda")
    out = buf[1024 + M % 3:1024 + M % 3 + M * N].view(M, N)
    y, plan = planned(lambda: L.w4a16_minifloat_linear(x.cuda(), layer.tw, layer.ts, layer.bias, transpose=transpose, out=out))
    assert plan == (height, splits)
    assert (buf[:1024 + M % 3] == -7).all() and (buf[1024 + M % 3 + M * N:] == -7).all()
    rows, cols = edges(rng, M, height, 8), edges(rng, N, 128, 90)
    codes, scales = X.fp8_quantize_ref(x[rows].double().numpy())
    ref, slack = layer.reference(codes, scales, cols)
    check(y[cuda(rows)][:, cuda(cols)], ref, slack, dtype, layer.bias.cpu().double().numpy()[cols])
    all_outputs(y, x.cuda(), layer, dtype, layer.bias)
    # codes of an earlier quantisation, and the same call again, give the same bits
    c, s = L.w4a16_minifloat_quantize(x.cuda())
    for _ in range(2):
        y2 = L.w4a16_minifloat_linear(c, layer.tw, layer.ts, layer.bias, transpose=transpose, x_scales=s, dtype=TYPES[dtype])
        assert torch.equal(bits(y), bits(y2))


@pytest.mark.parametrize("M,N,K,height,splits", [t for t in TILES if t[0] in (129, 67, 1000, 33, 1100, 1700, 100)])
@pytest.mark.parametrize("e8m0", [False, True])
@pytest.mark.parametrize("transpose", [False, True])
def test_what_is_not_finite_stays_in_its_row_and_feature(M, N, K, height, splits, e8m0, transpose, planned):  # noqa: F811
    rng = np.random.default_rng([M, N, K, 1])
    if transpose:
        N, K = (N + 15) // 16 * 16, K - 3
    layer = Weights(rng, N, K, transpose, e8m0)
    x = values(rng, M, K, "bf16").cuda()
    call = lambda x, w: L.w4a16_minifloat_linear(x, w, layer.ts, transpose=transpose)  # noqa: E731
    want, plan = planned(lambda: call(x, layer.tw))
    assert plan == (height, splits)
    bad_rows, bad_cols = sorted({0, height // 2, M // 2, M - 1}), sorted({3, N // 2, N - 1})
    x[cuda(bad_rows), cuda(rng.integers(0, K, len(bad_rows)))] = float("inf")
    x[bad_rows[-1], K - 1] = float("nan")
    w = layer.w.copy()
    for n in bad_cols:
        k = K - 1 if n % 2 else int(rng.integers(0, K))  # (also the last k, which a part of a block repeats)
        w[(k, n) if transpose else (n, k)] = 127
    y = call(x, torch.from_numpy(w).view(torch.float8_e4m3fn).cuda())
    nan = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    nan[cuda(bad_rows)] = True
    nan[:, cuda(bad_cols)] = True
    assert torch.equal(y.isnan(), nan) and torch.equal(bits(y)[~nan], bits(want)[~nan])


@pytest.mark.parametrize("M,N,K,height,splits", [t for t in TILES if t[0] in (129, 67, 1000, 33, 1100, 1700, 100)])
@pytest.mark.parametrize("transpose", [False, True])
def test_zero_scales(M, N, K, height, splits, transpose, planned):  # noqa: F811
    # blocks of scale zero between others: as if their weights were zeros, but for the NaN codes among them
    rng = np.random.default_rng([M, N, K, 2])
    if transpose:
        N, K = (N + 15) // 16 * 16, K - 3
    layer = Weights(rng, N, K, transpose, False)
    zero = rng.random(layer.ws.shape) < 0.5
    zero[0, 0] = True
    w, ts = layer.w.copy(), layer.ts.clone()
    spread = np.repeat(np.repeat(zero, 128, 0)[:w.shape[0]], 128, 1)[:, :w.shape[1]]
    plain = np.where(spread, 0, w).astype(np.uint8)
    x = values(rng, M, K, "bf16").cuda()
    call = lambda w, ts: L.w4a16_minifloat_linear(x, torch.from_numpy(w).view(torch.float8_e4m3fn).cuda(), ts,  # noqa: E731
                                                  transpose=transpose)
    want = call(plain, layer.ts)
    ts[cuda(zero)] = 0
    y, plan = planned(lambda: call(w, ts))
    assert plan == (height, splits)
    # (the unit that sums are kept in is another one where a block's scale does not enter it)
    assert (y.float() - want.float()).abs().max() <= 2.0 ** -8 * want.float().abs().max()
    rows, cols = edges(rng, M, height, 6), edges(rng, N, 128, 60)
    codes, scales = X.fp8_quantize_ref(x[cuda(rows)].cpu().double().numpy())
    layer.ws = np.where(zero, 0.0, layer.ws)
    ref, slack = layer.reference(codes, scales, cols)
    check(y[cuda(rows)][:, cuda(cols)], ref, slack, "bf16")
    w[(0, 5) if transpose else (5, 0)] = 255
    nan = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    nan[:, 5] = True
    bad = call(w, ts)
    assert torch.equal(bad.isnan(), nan) and torch.equal(bits(bad)[~nan], bits(y)[~nan])


# slots of each of four experts, and of none: last tiles of one place, of a half, a quarter, one less than full, full
COUNTS = {
    32: ([1, 31, 33, 64], 3),
    64: ([129, 160, 255, 383], 5),
    96: ([193, 289, 240, 480], 2),
    128: ([1, 257, 320, 447], 7),
}
EXPERTS = [(32, 272, 400), (64, 3410, 144), (96, 4000, 400), (128, 5000, 400)]


@pytest.mark.parametrize("height,N,K", EXPERTS)
@pytest.mark.parametrize("e8m0", [False, True])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("per_slot", [False, True])
def test_experts(height, N, K, e8m0, transpose, per_slot, planned):  # noqa: F811
    rng = np.random.default_rng([height, N, K])
    if transpose:
        N, K = (N + 15) // 16 * 16, K - 3
    dtype = "bf16" if e8m0 else "f16"
    counts, none = COUNTS[height]
    flat = np.repeat(np.array([0, 1, 2, 3, -1]), [*counts, none])
    topk = 1 if per_slot else 2
    flat = rng.permutation(np.concatenate([flat, np.full(-len(flat) % topk, 4)])).astype(np.int32)
    layer = Weights(rng, N, K, transpose, e8m0, E=4, bias=dtype)
    M = len(flat) // topk
    x = values(rng, len(flat) if per_slot else M, K, dtype)
    weights = rng.normal(0, 1, (M, topk)).astype(np.float32)
    y = torch.full((len(flat), N), float("nan"), dtype=TYPES[dtype], device="cuda")
    call = lambda x, w, y: L.w4a16_minifloat_moe_linear(  # noqa: E731
        x, w, layer.ts, cuda(flat.reshape(M, topk)), cuda(weights), layer.bias, transpose=transpose, x_per_slot=per_slot, out=y)
    _, plan = planned(lambda: call(x.cuda(), layer.tw, y))
    assert plan == (height, 1)
    named = (flat >= 0) & (flat < 4)
    assert torch.count_nonzero(y[cuda(~named)]) == 0 and not y.isnan().any()
    cols = edges(rng, N, 128, 90)
    bias = layer.bias.cpu().double().numpy()
    for e in range(4):
        slots = np.nonzero(flat == e)[0]
        row = slots if per_slot else slots // topk
        all_outputs(y[cuda(slots)], x[row].cuda(), layer, dtype, layer.bias[e], cuda(weights.reshape(-1, 1)[slots]), e)
        some = edges(rng, len(slots), height, 4)
        codes, scales = X.fp8_quantize_ref(x[row[some]].double().numpy())
        ref, slack = layer.reference(codes, scales, cols, e)
        check(y[cuda(slots[some])][:, cuda(cols)], ref, slack, dtype, bias[e][cols], weights.reshape(-1, 1)[slots[some]].astype(np.float64))
    # a token that is not finite, and a NaN weight of one expert, reach its own slots and feature only
    bad = x.clone()
    at = int(np.nonzero(flat == 3)[0][-1])
    bad[at if per_slot else at // topk, K - 1] = float("inf")
    w = layer.tw.clone().view(torch.uint8)
    w[(1, K - 1, 9) if transpose else (1, 9, K - 1)] = 127
    nan = torch.zeros((len(flat), N), dtype=torch.bool, device="cuda")
    mine = np.array([at]) if per_slot else np.arange(at // topk * topk, at // topk * topk + topk)
    nan[cuda(mine[named[mine]])] = True
    nan[cuda(np.nonzero(flat == 1)[0]), 9] = True
    got = call(bad.cuda(), w.view(torch.float8_e4m3fn), torch.empty_like(y))
    assert torch.equal(got.isnan(), nan) and torch.equal(bits(got)[~nan], bits(y)[~nan])
