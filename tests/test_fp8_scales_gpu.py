"""Weight scales that are no ordinary numbers: infinite, NaN, negative, zero and
subnormal fp32 scales, and the smallest and largest e8m0 ones, in the decode
kernel and in tiles of every height, for a layer and for experts.

Tolerances, fixed before the first run: as in test_fp8_gpu.py where the formula
gives a number (half a step of the output's type and the oracle's slack);
otherwise the same infinity, or NaN."""
import numpy as np
import pytest

from oracle import experts_ref as X
from fp8_cases import TYPES, Weights, edges, planned  # noqa: F401  (a fixture)
from gpu_util import note

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import int4_weight_only_linear_amd as L  # noqa: E402

INF, NAN = np.inf, np.nan


@pytest.fixture(autouse=True)
def _need_gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    note(f"[gpu] {request.node.nodeid}")


# scales of the five blocks of k of one block of features
PATTERNS = [
    [2e-4, -3e-4, 1.5e-4, -1e-4, 2.5e-4],
    [1e-4, INF, 2e-4, 1e-4, 3e-4],
    [1e-4, INF, 2e-4, INF, 3e-4],
    [INF, INF, -INF, 1e-4, 1e-4],
    [-INF, 2e-4, 1e-4, -INF, -INF],
    [1e-4, 2e-4, NAN, 1e-4, 3e-4],
    [1e26, 1e-45, 2e25, -3e-45, 1e-45],
    [1e-45, 1e26, 0.0, 5e-41, -1e26],
    [1e-40, -7e-41, 3e-42, 1.1e-38, -1e-40],
    [0.0, -0.0, 1e-4, 0.0, 0.0],
    [-1.9999999, 1.0, -1.0, 2.0, -0.0],
]


def scales_of(N, E):
    blocks = (N + 127) // 128
    return np.array([[PATTERNS[(b + e) % len(PATTERNS)] for b in range(blocks)] for e in range(E)], dtype=np.float32)


def compare(got, codes, scales, layer, cols, e, dtype):
    """Block by block, so that a scale that is not finite meets the sign of its block's sum."""
    got = got.cpu().double().numpy()
    w, ws = layer.of(cols, e)
    ws = ws.T if layer.tr else ws              # [features, blocks of k]
    for f in np.unique(cols // 128):
        at = np.nonzero(cols // 128 == f)[0]
        s = ws[at[0]]
        finite = np.isfinite(s)
        total, slack, bad = 0, 0, np.zeros(got[:, at].shape, dtype=bool)
        for b in range(len(s)):
            k = slice(128 * b, min(layer.K, 128 * (b + 1)))
            part = w[k][:, at] if layer.tr else w[at][:, k]
            y, off = X.fp8_linear_ref(codes[:, 128 * b:128 * (b + 1)], scales[:, b:b + 1], part, np.ones((1, 1)), k.stop - k.start, layer.tr)
            if not finite[b]:
                bad |= np.abs(y) <= off        # (a sum whose sign is not certain)
            with np.errstate(invalid="ignore"):
                total = total + y * s[b]
            # (the accumulators are rounded at most twice for each block that follows)
            slack = slack + (off * np.abs(s[b]) + 2.0 ** -23 * len(s) * np.abs(y * s[b]) if finite[b] else 0)
        have = got[:, at]
        assert np.array_equal(np.isnan(have) | bad, np.isnan(total) | bad), (f, s)
        with np.errstate(invalid="ignore"):
            same = (have == total) | np.isnan(total) | bad
            allowed = torch.finfo(TYPES[dtype]).eps / 2 * (np.abs(total) + slack) + slack + 2.0 ** -134
            assert (same | (np.abs(have - total) <= allowed)).all(), (f, s, have[~same][:4], total[~same][:4])


def draw_x(rng, M, K):
    x = rng.normal(size=(M, K)) * 2.0 ** 20
    return torch.from_numpy(x).to(torch.bfloat16)


# (M, N, tile height; None: decode)
ROWS = [(1, 1408, None), (2, 1403, None), (8, 1408, None), (20, 1400, 32), (1000, 4000, 64), (1100, 3999, 96), (1700, 3999, 128)]


@pytest.mark.parametrize("M,N,height", ROWS)
@pytest.mark.parametrize("transpose", [False, True])
def test_scales_of_every_kind(M, N, height, transpose, planned):  # noqa: F811
    rng = np.random.default_rng([M, N])
    K = 640
    if transpose:
        N, K = (N + 15) // 16 * 16, 637
        height = height or 32
    s = scales_of(N, 1)[0]
    layer = Weights(rng, N, K, transpose, False, scales=np.ascontiguousarray(s.T) if transpose else s)
    x = draw_x(rng, M, K)
    y, plan = planned(lambda: L.w4a16_minifloat_linear(x.cuda(), layer.tw, layer.ts, transpose=transpose))
    assert plan == (None if height is None else (height, 1))
    rows = edges(rng, M, height or 16, 6)
    cols = np.arange(N) if N < 2000 else edges(rng, N, 128, 160)
    codes, scales = X.fp8_quantize_ref(x[rows].double().numpy())
    compare(y[torch.from_numpy(rows).cuda()][:, torch.from_numpy(cols).cuda()], codes, scales, layer, cols, None, "bf16")


@pytest.mark.parametrize("transpose", [False, True])
def test_scales_of_every_kind_in_ranges(transpose, planned):  # noqa: F811
    # the blocks of k in ranges of four: scales meet across the ranges' sums
    rng = np.random.default_rng(4)
    M, N, K = 33, 8208 if transpose else 8195, 5136
    of = np.array(PATTERNS, dtype=np.float32)
    s = np.stack([np.resize(np.roll(of[b % len(of)], b), (K + 127) // 128) for b in range((N + 127) // 128)])
    layer = Weights(rng, N, K, transpose, False, scales=np.ascontiguousarray(s.T) if transpose else s)
    x = draw_x(rng, M, K)
    y, plan = planned(lambda: L.w4a16_minifloat_linear(x.cuda(), layer.tw, layer.ts, transpose=transpose))
    assert plan == (64, 6)
    rows, cols = edges(rng, M, 64, 3), edges(rng, N, 128, 120)
    codes, scales = X.fp8_quantize_ref(x[rows].double().numpy())
    compare(y[torch.from_numpy(rows).cuda()][:, torch.from_numpy(cols).cuda()], codes, scales, layer, cols, None, "bf16")


# (M, E, N, tile height)
@pytest.mark.parametrize("M,E,N,height", [(3, 6, 1408, None), (40, 6, 1403, 32), (1000, 4, 4000, 96), (1200, 4, 4800, 128)])
@pytest.mark.parametrize("transpose", [False, True])
def test_scales_of_every_kind_of_experts(M, E, N, height, transpose, planned):  # noqa: F811
    rng = np.random.default_rng([M, E])
    K = 640
    if transpose:
        N, K = (N + 15) // 16 * 16, 637
        height = height or 32
    s = scales_of(N, E)
    layer = Weights(rng, N, K, transpose, False, E=E, scales=np.ascontiguousarray(s.transpose(0, 2, 1)) if transpose else s)
    x = draw_x(rng, M, K)
    ids = rng.integers(0, E, M).astype(np.int32)
    y, plan = planned(lambda: L.w4a16_minifloat_moe_linear(x.cuda(), layer.tw, layer.ts, torch.from_numpy(ids.reshape(-1, 1)).cuda(),
                                                           transpose=transpose))
    assert plan == (None if height is None else (height, 1))
    cols = edges(rng, N, 128, 160)
    for e in range(E):
        rows = np.nonzero(ids == e)[0]
        if len(rows):
            rows = rows[edges(rng, len(rows), height or 16, 2)]
            codes, scales = X.fp8_quantize_ref(x[rows].double().numpy())
            compare(y[torch.from_numpy(rows).cuda()][:, torch.from_numpy(cols).cuda()], codes, scales, layer, cols, e, "bf16")


@pytest.mark.parametrize("M,N,height", ROWS)
@pytest.mark.parametrize("transpose", [False, True])
def test_powers_of_two_at_their_ends(M, N, height, transpose, planned):  # noqa: F811
    # weights' scales of 2^-127, 2^127 and NaN, and of the tokens'
    rng = np.random.default_rng([M, N, 1])
    K = 640
    if transpose:
        N, K = (N + 15) // 16 * 16, 637
        height = height or 32
    of = np.array([[0, 0, 1, 0, 2], [254, 253, 0, 254, 120], [127, 128, 126, 127, 100], [127, 255, 0, 127, 127], [1, 2, 127, 5, 60]],
                  dtype=np.uint8)
    s = np.stack([of[b % len(of)] for b in range((N + 127) // 128)])
    layer = Weights(rng, N, K, transpose, True, scales=np.ascontiguousarray(s.T) if transpose else s)
    codes, scales = X.fp8_quantize_ref(rng.normal(size=(M, K)))
    # tokens whose power meets the weights': the product's stays among the numbers of the output
    scales[:, :5] = np.array([[127, 127, 127, 127, 127], [0, 0, 0, 0, 0], [250, 247, 252, 250, 245], [127, 255, 127, 127, 127],
                              [1, 0, 3, 5, 2]], dtype=np.uint8)[np.arange(M) % 5]
    tx = torch.from_numpy(codes).view(torch.float8_e4m3fn).cuda()
    ts = torch.from_numpy(scales).view(torch.float8_e8m0fnu).cuda()
    y, plan = planned(lambda: L.w4a16_minifloat_linear(tx, layer.tw, layer.ts, transpose=transpose, x_scales=ts, dtype=torch.bfloat16))
    assert plan == (None if height is None else (height, 1))
    rows = edges(rng, M, height or 16, 12)
    cols = np.arange(N) if N < 2000 else edges(rng, N, 128, 160)
    xs = np.where(scales[rows] == 255, NAN, 2.0 ** (scales[rows].astype(np.float64) - 127))
    got = y[torch.from_numpy(rows).cuda()][:, torch.from_numpy(cols).cuda()].cpu().double().numpy()
    w, ws = layer.of(cols)
    ws = ws.T if transpose else ws
    for f in np.unique(cols // 128):
        at = np.nonzero(cols // 128 == f)[0]
        total, slack = np.zeros((len(rows), len(at))), np.zeros((len(rows), len(at)))
        for b in range(5):
            k = slice(128 * b, min(K, 128 * (b + 1)))
            part = w[k][:, at] if transpose else w[at][:, k]
            v, off = X.fp8_linear_ref(codes[rows][:, 128 * b:128 * (b + 1)], np.full((len(rows), 1), 127, np.uint8), part, np.ones((1, 1)),
                                      k.stop - k.start, transpose)
            with np.errstate(invalid="ignore"):
                total += v * (xs[:, b:b + 1] * ws[at[0], b])
                slack += off * (xs[:, b:b + 1] * ws[at[0], b])
        have = got[:, at]
        # what passes fp32's range is not compared, nor what lies within a step of it
        out = ~(np.abs(total) + slack < 2.0 ** 127) & ~np.isnan(total)
        assert np.array_equal(np.isnan(have)[~out], np.isnan(total)[~out])
        fine = ~out & ~np.isnan(total)
        # (below the normal numbers the matrix unit may give zero, for each of the 80 sums of eight products)
        allowed = 2.0 ** -8 * (np.abs(total) + slack) + slack + 81 * 2.0 ** -126
        assert (np.abs(have - total) <= allowed)[fine].all()


@pytest.mark.parametrize("M,N,height", ROWS)
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("size,scale", [(2.0 ** 121, 2e-4), (2.0 ** -110, 2e30), (2.0 ** -129, 2e37), (1e6, 1e-36)])
def test_tokens_and_scales_far_from_one(M, N, height, transpose, size, scale, planned):  # noqa: F811
    # the sum of a block's codes with one of the scales alone may pass fp32's range, the product does not
    rng = np.random.default_rng([M, N, 2])
    K = 640
    if transpose:
        N, K = (N + 15) // 16 * 16, 637
        height = height or 32
    blocks = ((K + 127) // 128, (N + 127) // 128) if transpose else ((N + 127) // 128, (K + 127) // 128)
    layer = Weights(rng, N, K, transpose, False, scales=(rng.uniform(0.5, 1.5, blocks) * scale).astype(np.float32))
    x = torch.from_numpy(rng.uniform(0.5, 8, (M, K)) * rng.choice([-1, 1], (M, K)) * size).to(torch.bfloat16)
    y, plan = planned(lambda: L.w4a16_minifloat_linear(x.cuda(), layer.tw, layer.ts, transpose=transpose))
    assert plan == (None if height is None else (height, 1))
    rows = edges(rng, M, height or 16, 6)
    cols = np.arange(N) if N < 2000 else edges(rng, N, 128, 160)
    codes, scales = X.fp8_quantize_ref(x[rows].double().numpy())
    compare(y[torch.from_numpy(rows).cuda()][:, torch.from_numpy(cols).cuda()], codes, scales, layer, cols, None, "bf16")
