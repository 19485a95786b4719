"""8-bit quantisation and products of 8-bit weights, through the C ABI, against
the float64 oracle.

Tolerances, fixed before the first run.  Codes and scales are equal, bit for
bit.  Outputs: half a step of their type, and the oracle's slack (what the
matrix unit's sums may drop; see fp8_linear_ref) times the slot's weight; two
more roundings in fp32 for bias and weight (2^-23 of the value and the bias).  At
sizes where forming the slack takes too long, the linear layer's tolerance
(gpu_util.TOL of max|y|)."""
import numpy as np
import pytest

from oracle import experts_ref as X
from gpu_util import TOL, note

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import int4_weight_only_linear_amd as L  # noqa: E402

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def _need_gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    note(f"[gpu] {request.node.nodeid}")


def values(rng, M, K, dtype):
    x = rng.normal(size=(M, K)) * np.exp(rng.normal(0, 0.7, K))
    return torch.from_numpy(x).to(TYPES[dtype])


def bytes_of(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


# ---------------------------------------------------------- quantisation ---

@pytest.mark.parametrize("M,K", [(1, 1), (1, 128), (3, 16), (2, 127), (5, 129), (4, 512), (7, 513), (67, 2560), (2, 14336), (9, 3587),
                                 (33, 2056), (130, 640)])
@pytest.mark.parametrize("dtype", TYPES)
def test_quantize(M, K, dtype):
    x = values(np.random.default_rng([M, K]), M, K, dtype)
    codes, scales = L.w4a16_minifloat_quantize(x.cuda())
    rc, rs = X.fp8_quantize_ref(x.double().numpy())
    assert np.array_equal(bytes_of(codes), rc) and np.array_equal(bytes_of(scales), rs)


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_every_value(dtype):
    # each value beside the block's largest, from far above it to far below
    bits = np.arange(65536, dtype=np.uint16)
    every = torch.from_numpy(bits.view(np.int16)).view(TYPES[dtype])
    for top in (448.0, 1.0, 300.0):
        x = torch.full((65536, 128), 0.0, dtype=TYPES[dtype])
        x[:, 0], x[:, 77] = every, top
        codes, scales = L.w4a16_minifloat_quantize(x.cuda())
        rc, rs = X.fp8_quantize_ref(x[:, [0, 77]].double().numpy())
        got = bytes_of(codes)
        nan = np.isin(rc[:, 0], (127, 255))
        assert np.array_equal(nan, np.isin(got[:, 0], (127, 255)))
        assert np.array_equal(got[~nan, 0], rc[~nan, 0]) and np.array_equal(got[:, 77], rc[:, 1])
        assert np.array_equal(bytes_of(scales)[:, 0], rs[:, 0])
        assert not got[:, 1:77].any() and not got[:, 78:].any()


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_blocks_do_not_mix(dtype):
    x = torch.zeros((4, 600), dtype=TYPES[dtype])
    x[0, 5], x[0, 130], x[0, 599] = float("inf"), 3.0, -2.0
    x[1, :] = float("nan")
    x[2, 0] = 2.0 ** -24
    x[3, 127], x[3, 128] = 60000.0, 2.0 ** -14
    codes, scales = L.w4a16_minifloat_quantize(x.cuda())
    rc, rs = X.fp8_quantize_ref(x.double().numpy())
    got = bytes_of(codes)
    nan = np.isin(rc, (127, 255))
    assert np.array_equal(nan, np.isin(got, (127, 255))) and np.array_equal(got[~nan], rc[~nan])
    assert np.array_equal(bytes_of(scales), rs)


def test_quantize_unaligned_rows():
    # a base that is two bytes off, and rows of odd length
    flat = values(np.random.default_rng(1), 1, 8 * 1024 + 1, "bf16").cuda().view(-1)
    for K in (1024, 1023):
        x = flat[1:1 + 8 * K].view(8, K)
        assert x.is_contiguous() and x.data_ptr() % 16
        codes, scales = L.w4a16_minifloat_quantize(x)
        rc, rs = X.fp8_quantize_ref(x.cpu().double().numpy())
        assert np.array_equal(bytes_of(codes), rc) and np.array_equal(bytes_of(scales), rs)


# -------------------------------------------------------------- products ---

class Layer:
    """Weights of one layer (E None) or of E experts, on the host and the device."""

    def __init__(self, rng, N, K, transpose, e8m0, E=None, bias=None):
        self.N, self.K, self.tr, self.E = N, K, transpose, E
        lead = () if E is None else (E,)
        shape = lead + ((K, N) if transpose else (N, K))
        blocks = lead + tuple((n + 127) // 128 for n in shape[-2:])
        self.w = X.to_e4m3(np.clip(rng.normal(0, 107, shape), -448, 448))
        if e8m0:
            s = rng.integers(110, 118, blocks).astype(np.uint8)
            self.ws, t = 2.0 ** (s.astype(np.float64) - 127), torch.from_numpy(s).view(torch.float8_e8m0fnu)
        else:
            s = (rng.uniform(0.5, 1.5, blocks) * 2e-4).astype(np.float32)
            self.ws, t = s.astype(np.float64), torch.from_numpy(s)
        self.tw = torch.from_numpy(self.w).view(torch.float8_e4m3fn).cuda()
        self.ts = t.cuda()
        self.bias = None if bias is None else torch.from_numpy(rng.normal(0, 0.5, lead + (N,))).to(TYPES[bias]).cuda()


def check(y, ref, slack, dtype, bias=None, weight=None):
    """y against ref = weight * (product + bias), slack of the product."""
    ref, slack = ref.copy(), slack.copy()
    extra = np.zeros_like(ref)
    if bias is not None:
        ref += bias
        extra += 2.0 ** -23 * (np.abs(ref) + np.abs(bias))
    if weight is not None:
        ref, slack, extra = ref * weight, slack * np.abs(weight), extra * np.abs(weight) + 2.0 ** -23 * np.abs(ref * weight)
    got = y.cpu().double().numpy()
    assert got.shape == ref.shape
    allowed = torch.finfo(TYPES[dtype]).eps / 2 * (np.abs(ref) + slack) + slack + extra + (2.0 ** -25 if dtype == "f16" else 0)
    err = np.abs(got - ref)
    assert (err <= allowed).all(), float(np.nanmax(err / allowed))


# (M, N, K): one token to several tiles, ragged tokens, features and blocks
SIZES = [(1, 64, 128), (1, 272, 2048), (2, 33, 256), (5, 130, 1040), (16, 128, 512), (17, 96, 640), (31, 257, 144), (33, 144, 400),
         (64, 384, 256), (67, 200, 1152), (129, 129, 272), (200, 640, 128), (257, 300, 256), (300, 520, 16)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("e8m0", [False, True])
def test_linear(M, N, K, dtype, transpose, e8m0):
    if transpose:
        N, K = (N + 15) // 16 * 16, K - 3  # any K
    rng = np.random.default_rng([M, N, K])
    layer = Layer(rng, N, K, transpose, e8m0, bias=dtype if M % 2 else None)
    x = values(rng, M, K, dtype)
    codes, scales = X.fp8_quantize_ref(x.double().numpy())
    ref, slack = X.fp8_linear_ref(codes, scales, layer.w, layer.ws, K, transpose)
    bias = None if layer.bias is None else layer.bias.cpu().double().numpy()
    y = L.w4a16_minifloat_linear(x.cuda(), layer.tw, layer.ts, layer.bias, transpose=transpose)
    assert y.dtype == TYPES[dtype]
    check(y, ref, slack, dtype, bias)
    # codes of an earlier quantisation give the same bits
    c, s = L.w4a16_minifloat_quantize(x.cuda())
    y2 = L.w4a16_minifloat_linear(c, layer.tw, layer.ts, layer.bias, transpose=transpose, x_scales=s, dtype=TYPES[dtype])
    assert torch.equal(y.view(torch.int16), y2.view(torch.int16))


LARGE = [(1, 4096, 4096, False), (3, 28672, 4096, False), (8, 4096, 14336, False), (12, 6144, 4096, False), (16, 2560, 9728, False),
         (67, 4096, 14336, False), (128, 4096, 4096, False), (300, 6144, 4096, False), (1000, 2560, 2560, False),
         (1921, 4096, 6144, True), (513, 4096, 1536, False), (40, 1024, 20480, False), (700, 8192, 1024, True)]


@pytest.mark.parametrize("M,N,K,transpose", LARGE)
@pytest.mark.parametrize("dtype", TYPES)
def test_linear_large(M, N, K, transpose, dtype):
    rng = np.random.default_rng([M, N, K])
    layer = Layer(rng, N, K, transpose, dtype == "f16")
    x = values(rng, M, K, dtype)
    y = L.w4a16_minifloat_linear(x.cuda(), layer.tw, layer.ts, transpose=transpose).cpu().double().numpy()
    rows = sorted({0, M // 3, M - 1})
    codes, scales = X.fp8_quantize_ref(x[rows].double().numpy())
    t = X.e4m3_values()
    W = t[layer.w] * X.spread(layer.ws, *layer.w.shape)
    ref = (t[codes[:, :K]] * np.repeat(2.0 ** (scales - 127.0), 128, 1)[:, :K]) @ (W if transpose else W.T)
    assert np.abs(y[rows] - ref).max() <= TOL[0 if dtype == "f16" else 1] * np.abs(ref).max()
    # every row, against torch's product of the same values in fp32 (of K terms: far below the tolerance)
    c, s = L.w4a16_minifloat_quantize(x.cuda())
    xd = c.float() * s.float().repeat_interleave(128, 1)[:, :c.shape[1]]
    full = (xd[:, :K].contiguous() @ torch.from_numpy((W if transpose else W.T).astype(np.float32)).cuda()).cpu().double().numpy()
    assert np.abs(y - full).max() <= TOL[0 if dtype == "f16" else 1] * np.abs(full).max()


@pytest.mark.parametrize("M", [1, 4, 40, 150])
@pytest.mark.parametrize("transpose", [False, True])
def test_values_that_are_not_finite_stay_in_their_row(M, transpose):
    rng = np.random.default_rng(M)
    N, K = 160, 288
    layer = Layer(rng, N, K, transpose, False)
    x = values(rng, M, K, "bf16").cuda()
    want = L.w4a16_minifloat_linear(x, layer.tw, layer.ts, transpose=transpose)
    bad = x.clone()
    bad[M // 2, 7] = float("inf")
    y = L.w4a16_minifloat_linear(bad, layer.tw, layer.ts, transpose=transpose)
    assert y[M // 2].isnan().all()
    keep = [m for m in range(M) if m != M // 2]
    assert torch.equal(y[keep].view(torch.int16), want[keep].view(torch.int16))
    # a NaN weight reaches its feature only, also from the last k
    w = layer.tw.clone().view(torch.uint8)
    if transpose:
        w[K - 1, 3] = 127
    else:
        w[3, K - 1] = 127
    y = L.w4a16_minifloat_linear(x, w.view(torch.float8_e4m3fn), layer.ts, transpose=transpose)
    assert y[:, 3].isnan().all()
    keep = [n for n in range(N) if n != 3]
    assert torch.equal(y[:, keep].view(torch.int16), want[:, keep].view(torch.int16))


def test_zero_tokens_and_zero_scales():
    rng = np.random.default_rng(0)
    layer = Layer(rng, 144, 256, False, False, bias="bf16")
    x = torch.zeros((5, 256), dtype=torch.bfloat16, device="cuda")
    y = L.w4a16_minifloat_linear(x, layer.tw, layer.ts, layer.bias)
    assert torch.equal(y, layer.bias.expand(5, 144))
    assert L.w4a16_minifloat_linear(x[:0], layer.tw, layer.ts).shape == (0, 144)
    layer.ts.zero_()
    y = L.w4a16_minifloat_linear(values(rng, 5, 256, "bf16").cuda(), layer.tw, layer.ts)
    assert torch.count_nonzero(y) == 0


# --------------------------------------------------------------- experts ---

def draw_ids(rng, M, topk, E, how):
    if how == "one":
        return np.full((M, topk), E - 1, dtype=np.int32)
    if how == "none":
        return np.full((M, topk), -1, dtype=np.int32)
    ids = np.stack([rng.permutation(E)[:topk] if topk <= E else rng.integers(0, E, topk) for _ in range(M)]).astype(np.int32)
    if how == "some":
        ids[rng.random((M, topk)) < 0.3] = -1
        ids.flat[0] = E
        ids.flat[-1] = 2 ** 31 - 1
    if how == "skewed":
        ids = np.minimum(ids, rng.geometric(0.4, (M, topk)) - 1).astype(np.int32)
    return ids


def moe_ref(x, layer, ids, per_slot):
    M, topk = ids.shape
    codes, scales = X.fp8_quantize_ref(x.double().numpy())
    y, slack = np.zeros((M * topk, layer.N)), np.zeros((M * topk, layer.N))
    flat = ids.reshape(-1)
    for e in np.unique(flat):
        if 0 <= e < layer.E:
            slots = np.nonzero(flat == e)[0]
            rows = slots if per_slot else slots // topk
            y[slots], slack[slots] = X.fp8_linear_ref(codes[rows], scales[rows], layer.w[e], layer.ws[e], layer.K, layer.tr)
    return y, slack


# (M, topk, E, N, K, ids, per_slot)
MOE = [
    (1, 1, 1, 64, 128, "all", False), (1, 8, 16, 96, 256, "all", False), (2, 8, 128, 130, 272, "all", True), (8, 4, 6, 48, 400, "some", False),
    (5, 2, 3, 144, 128, "one", False), (16, 4, 64, 64, 512, "skewed", True), (40, 2, 8, 200, 256, "some", False),
    (33, 6, 60, 32, 144, "all", True), (150, 1, 2, 130, 272, "skewed", False), (70, 8, 9, 64, 128, "skewed", False),
    (9, 3, 5, 80, 256, "none", True), (300, 2, 3, 144, 160, "some", True), (64, 8, 4, 32, 128, "all", False), (3, 5, 2, 48, 128, "all", True),
    (130, 3, 1000, 16, 64, "all", False), (100, 8, 256, 32, 128, "skewed", False), (120, 8, 240, 40, 272, "some", True),
]


@pytest.mark.parametrize("M,topk,E,N,K,how,per_slot", MOE)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("transpose", [False, True])
def test_moe(M, topk, E, N, K, how, per_slot, dtype, transpose):
    if transpose:
        N, K = (N + 15) // 16 * 16, K - 3
    rng = np.random.default_rng([M, topk, E, N])
    layer = Layer(rng, N, K, transpose, M % 2 == 0, E=E, bias=dtype if topk % 2 else None)
    x = values(rng, M * topk if per_slot else M, K, dtype)
    ids = draw_ids(rng, M, topk, E, how)
    ref, slack = moe_ref(x, layer, ids, per_slot)
    flat = ids.reshape(-1)
    named = (flat >= 0) & (flat < E)
    bias = None
    if layer.bias is not None:
        bias = layer.bias.cpu().double().numpy()[np.where(named, flat, 0)] * named[:, None]
    weights = None if M % 3 == 0 else rng.normal(0, 1, (M, topk)).astype(np.float32)
    y = torch.full((M * topk, N), float("nan"), dtype=TYPES[dtype], device="cuda")
    got = L.w4a16_minifloat_moe_linear(x.cuda(), layer.tw, layer.ts, torch.from_numpy(ids).cuda(),
                                 None if weights is None else torch.from_numpy(weights).cuda(), layer.bias, transpose=transpose,
                                 x_per_slot=per_slot, out=y)
    assert got is y
    check(y, ref, slack, dtype, bias, None if weights is None else weights.reshape(-1, 1).astype(np.float64))
    assert torch.count_nonzero(y[torch.from_numpy(~named).cuda()]) == 0
    c, s = L.w4a16_minifloat_quantize(x.cuda())
    again = L.w4a16_minifloat_moe_linear(c, layer.tw, layer.ts, torch.from_numpy(ids).cuda(),
                                   None if weights is None else torch.from_numpy(weights).cuda(), layer.bias, transpose=transpose,
                                   x_per_slot=per_slot, x_scales=s, dtype=TYPES[dtype])
    assert torch.equal(y.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("M", [3, 60, 700])
def test_moe_of_one_expert_is_the_linear_layer(M):
    rng = np.random.default_rng(M)
    layer = Layer(rng, 272, 640, False, False, bias="f16")
    x = values(rng, M, 640, "f16").cuda()
    ids = torch.zeros((M, 1), dtype=torch.int32, device="cuda")
    y = L.w4a16_minifloat_moe_linear(x, layer.tw[None], layer.ts[None], ids, bias=layer.bias[None])
    want = L.w4a16_minifloat_linear(x, layer.tw, layer.ts, layer.bias)
    # (tiles of other sizes may add the blocks in another order: a step of the type)
    assert ((y.float() - want.float()).abs() <= 2.0 ** -10 * want.float().abs() + 2.0 ** -20 * want.float().abs().max()).all()


@pytest.mark.parametrize("M,topk,E", [(64, 8, 32), (2048, 4, 16), (512, 8, 128)])
def test_moe_large(M, topk, E):
    rng = np.random.default_rng([M, E])
    N, K = 768, 1024
    layer = Layer(rng, N, K, False, False, E=E)
    x = values(rng, M, K, "bf16")
    ids = draw_ids(rng, M, topk, E, "skewed")
    y = L.w4a16_minifloat_moe_linear(x.cuda(), layer.tw, layer.ts, torch.from_numpy(ids).cuda()).float()
    c, s = L.w4a16_minifloat_quantize(x.cuda())
    xd = c.float() * s.float().repeat_interleave(128, 1)[:, :K]
    flat = ids.reshape(-1)
    top = float(y.abs().max())
    for e in np.unique(flat):
        slots = torch.from_numpy(np.nonzero(flat == e)[0]).cuda()
        W = torch.from_numpy((X.e4m3_values()[layer.w[e]] * X.spread(layer.ws[e], N, K)).astype(np.float32)).cuda()
        assert (y[slots] - xd[slots // topk] @ W.T).abs().max() <= TOL[1] * top


def test_equal_inputs_give_equal_bits():
    rng = np.random.default_rng(12)
    layer = Layer(rng, 520, 1040, False, False, E=12)
    for M in (2, 50, 400):
        x = values(rng, M, 1040, "bf16").cuda()
        ids = torch.from_numpy(draw_ids(rng, M, 4, 12, "skewed")).cuda()
        runs = [L.w4a16_minifloat_moe_linear(x, layer.tw, layer.ts, ids) for _ in range(5)]
        assert all(torch.equal(r.view(torch.int16), runs[0].view(torch.int16)) for r in runs)
        runs = [L.w4a16_minifloat_linear(x, layer.tw[3].contiguous(), layer.ts[3].contiguous()) for _ in range(5)]
        assert all(torch.equal(r.view(torch.int16), runs[0].view(torch.int16)) for r in runs)


@pytest.mark.parametrize("M", [2, 30, 200])
def test_streams_graphs_and_workspaces(M):
    rng = np.random.default_rng(M)
    layer = Layer(rng, 272, 1152, False, False, E=6)
    one_w, one_s = layer.tw[0].contiguous(), layer.ts[0].contiguous()
    x = values(rng, M, 1152, "bf16").cuda()
    ids = torch.from_numpy(draw_ids(rng, M, 3, 6, "all")).cuda()
    want = L.w4a16_minifloat_linear(x, one_w, one_s), L.w4a16_minifloat_moe_linear(x, layer.tw, layer.ts, ids)
    same = lambda a, b: torch.equal(a.view(torch.int16), b.view(torch.int16))  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = L.w4a16_minifloat_linear(x, one_w, one_s), L.w4a16_minifloat_moe_linear(x, layer.tw, layer.ts, ids)
    side.synchronize()
    assert same(y[0], want[0]) and same(y[1], want[1])
    need = (L.w4a16_minifloat_linear_workspace_size(M, 272, 1152, L.W4A16_BF16),
            L.w4a16_minifloat_moe_workspace_size(M, 3, 6, 272, 1152, L.W4A16_BF16))
    ws = torch.zeros(max(*need, 2 * M * 1152), dtype=torch.uint8, device="cuda")
    out = [torch.empty_like(w) for w in want]

    def both():
        # two calls that share one workspace, one after the other
        L.w4a16_minifloat_linear(x, one_w, one_s, out=out[0], workspace=ws)
        L.w4a16_minifloat_moe_linear(x, layer.tw, layer.ts, ids, out=out[1], workspace=ws)

    both()
    assert torch.count_nonzero(ws[:65536]) == 0
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    for seed in range(4):
        x.copy_(values(np.random.default_rng(100 + seed), M, 1152, "bf16"))
        ids.copy_(torch.from_numpy(draw_ids(np.random.default_rng(seed), M, 3, 6, "some")))
        g.replay()
        torch.cuda.synchronize()
        assert same(out[0], L.w4a16_minifloat_linear(x, one_w, one_s))
        assert same(out[1], L.w4a16_minifloat_moe_linear(x, layer.tw, layer.ts, ids))
    with pytest.raises(L.W4A16Error) as e:
        L.w4a16_minifloat_moe_linear(x, layer.tw, layer.ts, ids, workspace=ws[:4096])
    assert e.value.status == 6
    with pytest.raises(L.W4A16Error):  # the workspace is x's own memory
        L.w4a16_minifloat_linear(ws[:2 * M * 1152].view(torch.bfloat16).view(M, 1152), one_w, one_s, workspace=ws)


def test_guards_around_outputs():
    # nothing outside y is written, whatever the tile's edges
    rng = np.random.default_rng(3)
    for M, N in ((3, 100), (70, 131), (140, 36)):
        layer = Layer(rng, N, 256, False, False)
        x = values(rng, M, 256, "f16").cuda()
        buf = torch.full((M * N + 2048,), -7.0, dtype=torch.float16, device="cuda")
        out = buf[1024:1024 + M * N].view(M, N)
        L.w4a16_minifloat_linear(x, layer.tw, layer.ts, out=out)
        assert (buf[:1024] == -7).all() and (buf[1024 + M * N:] == -7).all()
        assert torch.equal(out, L.w4a16_minifloat_linear(x, layer.tw, layer.ts))


# -------------------------------------------------- as they are used ---

@pytest.mark.parametrize("M", [1, 6, 90])
def test_a_layer_of_experts(M):
    """Router, gate and up, down, sum over the slots, and back to the input: against the same chain
    in float64 on the values that each step hands on."""
    rng = np.random.default_rng(M)
    E, topk, H, F = 16, 4, 256, 384
    x = values(rng, M, H, "bf16").cuda()
    router = torch.from_numpy(rng.normal(0, H ** -0.5, (E, H)).astype(np.float32)).cuda()
    bias = torch.from_numpy(rng.normal(0, 0.05, E).astype(np.float32)).cuda()
    up, down = Layer(rng, 2 * F, H, False, False, E=E), Layer(rng, H, F, False, True, E=E)
    logits = x.float() @ router.T
    kw = dict(score="sigmoid", renormalize=True, scale=2.0)
    weights, ids = L.w4a16_route(logits, topk, bias, groups=4, topk_groups=2, group_top=2, **kw)
    rw, ri = X.route_ref(logits.cpu().double().numpy(), topk, bias.cpu().numpy(), groups=4, topk_groups=2, group_top=2, **kw)
    assert np.array_equal(ids.cpu().numpy(), ri)
    h = L.w4a16_minifloat_moe_linear(x, up.tw, up.ts, ids)
    ref, slack = moe_ref(x.cpu(), up, ri, False)
    check(h, ref, slack, "bf16")
    act = (torch.nn.functional.silu(h[:, :F].float()) * h[:, F:].float()).to(torch.bfloat16)
    y = L.w4a16_minifloat_moe_linear(act, down.tw, down.ts, ids, weights, x_per_slot=True)
    ref, slack = moe_ref(act.cpu(), down, ri, True)
    check(y, ref, slack, "bf16", weight=weights.cpu().double().numpy().reshape(-1, 1))
    out = y.view(M, topk, H).float().sum(1)
    # the gradient of sum(out * g): through the experts' second product and through the router's weights
    g = values(rng, M, H, "bf16").cuda()
    dy = g.repeat_interleave(topk, 0)
    dact = L.w4a16_minifloat_moe_linear(dy, down.tw, down.ts, ids, weights, transpose=True, x_per_slot=True)
    back = Layer.__new__(Layer)
    back.w, back.ws, back.N, back.K, back.tr, back.E = down.w, down.ws, F, H, True, E
    ref, slack = moe_ref(dy.cpu(), back, ri, True)
    check(dact, ref, slack, "bf16", weight=weights.cpu().double().numpy().reshape(-1, 1))
    plain = L.w4a16_minifloat_moe_linear(act, down.tw, down.ts, ids, x_per_slot=True)
    dw = (plain.float() * dy.float()).sum(1).view(M, topk)
    dl = L.w4a16_route_backward(dw, logits, ids, **kw)
    ref, bound = X.route_backward_ref(dw.cpu().numpy(), logits.cpu().double().numpy(), ri, **kw)
    assert (np.abs(dl.cpu().double().numpy() - ref) <= 2.0 ** -24 * (17 + topk) * bound + 2.0 ** -24 * np.abs(ref)).all()
    assert out.isfinite().all()


def test_the_routers_choice_feeds_the_4_bit_experts():
    from synth import make_case
    import oracle as O
    E, topk, M, N, K = 6, 2, 5, 64, 256
    cases = [make_case(M, N, K, 128, O.BF16, True, False, seed=("route", e)) for e in range(E)]
    stack = lambda get: torch.from_numpy(np.stack([get(c) for c in cases])).cuda()  # noqa: E731
    wq = stack(lambda c: L.w4a16_pack_weights(c.q))
    s = stack(lambda c: c.s_bits.view(np.int16)).view(torch.bfloat16)
    x = torch.from_numpy(cases[0].x_bits.view(np.int16)).cuda().view(torch.bfloat16)
    logits = torch.from_numpy(np.random.default_rng(0).normal(size=(M, E)).astype(np.float32)).cuda()
    logits[2, 1:] = float("-inf")  # one expert is left: the second slot has none
    weights, ids = L.w4a16_route(logits, topk, renormalize=True)
    assert ids[2, 1] == -1
    y = L.w4a16_moe_linear(x, wq, s, ids, topk_weights=weights, group_size=128)
    ref = O.moe_linear_ref(cases[0].x_bits, np.stack([O.pack_weights(c.q) for c in cases]), np.stack([c.s_bits for c in cases]),
                           None, None, ids.cpu().numpy(), weights.cpu().numpy(), M, topk, E, N, K, 128, O.BF16)
    got = y.cpu().double().numpy()
    assert np.abs(got - ref.reshape(got.shape)).max() <= TOL[1] * np.abs(ref).max()
    assert not got[2 * topk + 1].any()


@pytest.mark.parametrize("M,N,K", [(8, 192, 9216), (8, 96, 9856), (8, 96, 10240), (2, 64, 38400), (2, 64, 40960)])
@pytest.mark.parametrize("dtype", TYPES)
def test_few_tokens_of_many_features(M, N, K, dtype):
    # the tokens' codes fill more than half of a CU's memory, or are made by a launch of their own
    rng = np.random.default_rng([M, N, K])
    layer = Layer(rng, N, K, False, dtype == "f16", bias=dtype)
    x = values(rng, M, K, dtype)
    codes, scales = X.fp8_quantize_ref(x.double().numpy())
    t = X.e4m3_values()
    ref = (t[codes[:, :K]] * np.repeat(2.0 ** (scales - 127.0), 128, 1)[:, :K]) @ (t[layer.w] * X.spread(layer.ws, N, K)).T
    ref += layer.bias.cpu().double().numpy()
    y = L.w4a16_minifloat_linear(x.cuda(), layer.tw, layer.ts, layer.bias)
    assert np.abs(y.cpu().double().numpy() - ref).max() <= TOL[0 if dtype == "f16" else 1] * np.abs(ref).max()
    c, s = L.w4a16_minifloat_quantize(x.cuda())
    y2 = L.w4a16_minifloat_linear(c, layer.tw, layer.ts, layer.bias, x_scales=s, dtype=TYPES[dtype])
    assert torch.equal(y.view(torch.int16), y2.view(torch.int16))


@pytest.mark.parametrize("transpose", [False, True])
def test_experts_with_a_few_slots_more_than_a_tile(transpose):
    # tiles whose last half, quarter or all but one place is empty, beside full ones
    rng = np.random.default_rng(12)
    N, K = 144, 272
    ids = np.repeat(np.arange(8), [129, 160, 192, 193, 224, 255, 256, 1])
    layer = Layer(rng, N, K, transpose, False, E=8)
    x = values(rng, len(ids), K, "bf16")
    order = rng.permutation(len(ids))
    ids = ids[order].astype(np.int32).reshape(-1, 1)
    y = L.w4a16_minifloat_moe_linear(x.cuda(), layer.tw, layer.ts, torch.from_numpy(ids).cuda(), transpose=transpose)
    codes, scales = X.fp8_quantize_ref(x.double().numpy())
    for e in range(8):
        rows = np.nonzero(ids[:, 0] == e)[0]
        ref, slack = X.fp8_linear_ref(codes[rows], scales[rows], layer.w[e], layer.ws[e], K, transpose)
        check(y.reshape(len(ids), -1)[torch.from_numpy(rows).cuda()], ref, slack, "bf16")


@pytest.mark.parametrize("M", [1, 5, 40, 100, 150])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("experts", [False, True])
def test_a_zero_scale_keeps_what_is_not_a_number(M, transpose, experts):
    # blocks of scale zero between others: their weights count as zeros, and a NaN of x or w in one stays one
    rng = np.random.default_rng(M)
    N, K = 272, 528
    layer = Layer(rng, N, K, transpose, False, E=2 if experts else None)
    zero = rng.random(layer.ws.shape) < 0.5
    zero[..., 0, 0] = True
    zero[..., -1, -1] = False
    layer.ts[torch.from_numpy(zero).cuda()] = 0
    w = layer.w.copy()
    k, n = 5, 7                           # in the first block, whose scale is zero
    w[..., k if transpose else n, n if transpose else k] = 255
    x = values(rng, M, K, "bf16")
    x[M // 2, 9] = float("nan")
    ws = np.where(zero, 0.0, layer.ws)
    tw = torch.from_numpy(w).view(torch.float8_e4m3fn).cuda()
    codes, scales = X.fp8_quantize_ref(x.double().numpy())
    if experts:
        ids = torch.from_numpy(rng.integers(0, 2, (M, 1)).astype(np.int32))
        y = L.w4a16_minifloat_moe_linear(x.cuda(), tw, layer.ts, ids.cuda(), transpose=transpose).cpu()
    else:
        ids = torch.zeros((M, 1), dtype=torch.int32)
        y = L.w4a16_minifloat_linear(x.cuda(), tw, layer.ts, transpose=transpose).cpu()
    for e in range(2):
        rows = np.nonzero(ids[:, 0].numpy() == e)[0]
        if not len(rows):
            continue
        we, se = (w[e], ws[e]) if experts else (w, ws)
        got = y[rows].double().numpy()
        nan = np.zeros((len(rows), N), dtype=bool)
        nan[:, n] = True
        nan[rows == M // 2] = True
        assert np.array_equal(np.isnan(got), nan)
        ok, c = np.where(we == 255, 0, we).astype(np.uint8), np.where(np.isin(codes[rows], (127, 255)), 0, codes[rows]).astype(np.uint8)
        ref, slack = X.fp8_linear_ref(c, scales[rows], ok, se, K, transpose)
        allowed = torch.finfo(torch.bfloat16).eps / 2 * (np.abs(ref) + slack) + slack
        assert (np.abs(got - ref) <= allowed)[~nan].all()
