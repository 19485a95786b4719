"""Routing, quantisation and 8-bit products where offsets pass 2^31 elements, and
blocks of subnormal values.

The large inputs repeat a part of themselves, so that every repetition must have
the same bits as the first (tolerance: none); the first is what the other tests
compare with the oracle at smaller sizes."""
import numpy as np
import pytest

from oracle import experts_ref as X
from fp8_cases import TYPES, Weights, values
from gpu_util import TOL, note
from test_route_gpu import check as check_route

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import int4_weight_only_linear_amd as L  # noqa: E402


@pytest.fixture(autouse=True)
def _need_gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    note(f"[gpu] {request.node.nodeid}")
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def repeats(t, rows):
    """Whether t repeats its first `rows` rows, compared a part at a time."""
    if t.element_size() < 4:
        t = t.view(torch.int16 if t.element_size() == 2 else torch.uint8)
    first = t[:rows]
    return all(torch.equal(t[i:i + rows], first[:min(rows, len(t) - i)]) for i in range(rows, len(t), rows))


def test_routing_of_many_tokens():
    # the most tokens that a call takes, 2.4 G logits
    M, E, topk, part = 1 << 25, 72, 2, 1 << 16
    l = torch.randn((part, E), generator=torch.Generator("cuda").manual_seed(1), device="cuda").to(torch.bfloat16)
    logits = l.repeat(M // part, 1)
    w, ids = L.w4a16_route(logits, topk, score="sigmoid", renormalize=True, groups=4, topk_groups=2)
    check_route(l[:64].cpu().double().numpy(), (w[:64], ids[:64]), topk, None, score="sigmoid", renormalize=True, groups=4, topk_groups=2)
    assert repeats(w, part) and repeats(ids, part)
    dw = torch.randn((part, topk), device="cuda").repeat(M // part, 1)
    out = torch.full_like(logits, float("nan"))
    L.w4a16_route_backward(dw, logits, ids, score="sigmoid", renormalize=True, out=out)
    assert repeats(out, part) and torch.count_nonzero(out[:part]) > part


@pytest.mark.parametrize("transpose", [False, True])
def test_many_tokens(transpose):
    # 3.1 G codes of x
    M, N, K, part = 220000, 80, 14336, 2048
    layer = Weights(np.random.default_rng(2), N, K, transpose, True)
    few = values(np.random.default_rng(3), part, K, "bf16").cuda()
    x = few.repeat(-(-M // part), 1)[:M]
    codes, scales = L.w4a16_minifloat_quantize(x)
    assert repeats(codes, part) and repeats(scales, part)
    y = L.w4a16_minifloat_linear(x, layer.tw, layer.ts, transpose=transpose)
    assert repeats(y, part) and torch.count_nonzero(y[:part]) > part
    del x, scales
    c, s = L.w4a16_minifloat_quantize(few)
    assert torch.equal(codes[:part].view(torch.uint8), c.view(torch.uint8))
    full = c.float() * s.float().repeat_interleave(128, 1) @ layer.dense().contiguous()
    assert (y[:part].float() - full).abs().max() <= TOL[1] * full.abs().max()


@pytest.mark.parametrize("M", [2, 40])
@pytest.mark.parametrize("experts", [False, True])
def test_many_features(M, experts):
    # 3.1 G codes of a layer's weights, in the decode kernel and in tiles
    N, K, part = 220032, 14336, 4096
    layer = Weights(np.random.default_rng(4), part, K, False, False)
    w = layer.tw.view(torch.uint8).repeat(-(-N // part), 1)[:N].view(torch.float8_e4m3fn)
    s = layer.ts.repeat(-(-N // part), 1)[:(N + 127) // 128].contiguous()
    x = values(np.random.default_rng(5), M, K, "bf16").cuda()
    if experts:
        ids = torch.zeros((M, 1), dtype=torch.int32, device="cuda")
        y = L.w4a16_minifloat_moe_linear(x, w[None], s[None], ids)
    else:
        y = L.w4a16_minifloat_linear(x, w, s)
    assert repeats(y.T.contiguous(), part)
    c, t = L.w4a16_minifloat_quantize(x)
    full = c.float() * t.float().repeat_interleave(128, 1) @ layer.dense().contiguous()
    assert (y[:, :part].float() - full).abs().max() <= TOL[1] * full.abs().max()


@pytest.mark.parametrize("M", [2, 150])
def test_a_long_sum_over_features(M):
    # transposed weights of 3.1 G codes: tokens that are zero but for the last features
    N, K, part = 14336, 220032, 4096
    layer = Weights(np.random.default_rng(6), N, part, True, False)
    w = torch.zeros((K, N), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    w[-part:] = layer.tw
    s = torch.ones(((K + 127) // 128, (N + 127) // 128), device="cuda")
    s[-part // 128:] = layer.ts
    few = values(np.random.default_rng(7), M, part, "bf16").cuda()
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    x[:, -part:] = few
    y = L.w4a16_minifloat_linear(x, w, s, transpose=True).float()
    c, t = L.w4a16_minifloat_quantize(few)
    full = c.float() * t.float().repeat_interleave(128, 1) @ layer.dense().contiguous()
    assert (y - full).abs().max() <= TOL[1] * full.abs().max()


@pytest.mark.parametrize("M", [5, 300])
def test_many_experts_weights(M):
    # experts whose weights lie past 2^32 bytes
    E, N, K = 40, 8192, 14336
    layer = Weights(np.random.default_rng(8), N, K, False, True)
    w = torch.empty((E, N, K), dtype=torch.float8_e4m3fn, device="cuda")
    w[:] = layer.tw
    w[E - 1].view(torch.uint8)[:] = layer.tw.view(torch.uint8).flip(0)
    s = layer.ts.view(torch.uint8).expand(E, -1, -1).contiguous()
    s[E - 1] = s[E - 1].flip(0)
    x = values(np.random.default_rng(9), M, K, "bf16").cuda()
    ids = (torch.arange(M, device="cuda") % 2 * (E - 1)).to(torch.int32).view(M, 1)
    y = L.w4a16_minifloat_moe_linear(x, w, s.view(torch.float8_e8m0fnu), ids)
    want = L.w4a16_minifloat_moe_linear(x, w[:1], s[:1].view(torch.float8_e8m0fnu), torch.zeros_like(ids))
    want[1::2] = want[1::2].flip(1)
    # (another plan may add the blocks in another order)
    assert (y.float() - want.float()).abs().max() <= TOL[1] * want.float().abs().max()


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_blocks_of_subnormal_values(dtype):
    rng = np.random.default_rng(10)
    low = -24 if dtype == "f16" else -133
    x = torch.from_numpy(rng.normal(size=(200, 640)) * 2.0 ** rng.integers(low - 1, low + 14, (200, 1))).to(TYPES[dtype])
    codes, scales = L.w4a16_minifloat_quantize(x.cuda())
    rc, rs = X.fp8_quantize_ref(x.double().numpy())
    assert np.array_equal(codes.view(torch.uint8).cpu().numpy(), rc) and np.array_equal(scales.view(torch.uint8).cpu().numpy(), rs)
    # every subnormal value and the smallest normal ones, alone in their blocks
    bits = np.arange(2048 if dtype == "f16" else 512, dtype=np.uint16)
    bits = np.concatenate([bits, bits | 0x8000])
    x = torch.zeros((len(bits), 128), dtype=TYPES[dtype])
    x[:, 5] = torch.from_numpy(bits.view(np.int16)).view(TYPES[dtype])
    codes, scales = L.w4a16_minifloat_quantize(x.cuda())
    rc, rs = X.fp8_quantize_ref(x.double().numpy())
    assert np.array_equal(codes.view(torch.uint8).cpu().numpy(), rc) and np.array_equal(scales.view(torch.uint8).cpu().numpy(), rs)
