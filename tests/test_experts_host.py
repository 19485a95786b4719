"""Routing, 8-bit quantisation and 8-bit products on the host: argument checks
before any device is touched, and workspace sizes.  Fake pointers, never
dereferenced."""
import pytest

import int4_weight_only_linear_amd as L
from int4_weight_only_linear_amd import _binding as B

P = 1 << 34  # apart by more than any extent below


def route(**kw):
    a = dict(logits=P, bias=None, weights=2 * P, ids=3 * P, M=4, E=64, topk=6, groups=1, kept=1, top=1, dt=1, score=0, renorm=1,
             scale=1.0)
    assert set(kw) <= set(a)
    a.update(kw)
    return B.lib.w4a16_route(*a.values(), None)


def route_backward(**kw):
    a = dict(dw=P, logits=2 * P, ids=3 * P, out=4 * P, M=4, E=64, topk=6, dt=1, score=0, renorm=1, scale=1.0)
    assert set(kw) <= set(a)
    a.update(kw)
    return B.lib.w4a16_route_backward(*a.values(), None)


def quantize(**kw):
    a = dict(x=P, codes=2 * P, scales=3 * P, M=4, K=256, dt=1)
    assert set(kw) <= set(a)
    a.update(kw)
    return B.lib.w4a16_minifloat_quantize(*a.values(), None)


def linear(**kw):
    a = dict(x=P, xs=None, w=2 * P, ws=3 * P, bias=None, y=4 * P, M=4, N=64, K=256, xdt=1, sdt=2, dt=1, tr=0, work=5 * P, n=1 << 24)
    assert set(kw) <= set(a)
    a.update(kw)
    return B.lib.w4a16_minifloat_linear(*a.values(), None)


def moe(**kw):
    a = dict(x=P, xs=None, w=2 * P, ws=3 * P, bias=None, ids=6 * P, tw=None, y=4 * P, M=4, topk=2, E=8, N=64, K=256, xdt=1, sdt=2,
             dt=1, tr=0, slot=0, work=5 * P, n=1 << 24)
    assert set(kw) <= set(a)
    a.update(kw)
    return B.lib.w4a16_minifloat_moe_linear(*a.values(), None)


ROUTER = [
    (dict(dt=3), 1, "logits must be"),
    (dict(score=2), 1, "unknown score"),
    (dict(M=-1), 1, "topk <= E"),
    (dict(topk=0), 1, "topk <= E"),
    (dict(topk=65), 1, "topk <= E"),
    (dict(E=1025), 2, "at most 1024"),
    (dict(E=128, topk=65), 2, "topk 64"),
    (dict(M=(1 << 25) + 1), 2, "tokens"),
    (dict(scale=float("nan")), 1, "finite"),
    (dict(logits=None), 1, "NULL"),
    (dict(ids=None), 1, "NULL"),
    (dict(logits=P + 1), 3, "aligned"),
    (dict(dt=2, logits=P + 2), 3, "aligned"),
    (dict(ids=3 * P + 2), 3, "aligned"),
]


@pytest.mark.parametrize("kw,status,msg", ROUTER + [
    (dict(groups=0), 1, "topk_groups <= groups"),
    (dict(groups=3), 1, "multiple of groups"),
    (dict(E=650, groups=65), 1, "<= 64"),
    (dict(groups=4, kept=5), 1, "topk_groups <= groups"),
    (dict(groups=4, kept=0), 1, "topk_groups <= groups"),
    (dict(groups=4, kept=2, top=3), 1, "two largest"),
    (dict(groups=64, kept=6, top=2), 1, "two largest"),
    (dict(groups=16, kept=1, top=1), 1, "out of 1 groups"),
    (dict(weights=None), 1, "NULL"),
    (dict(bias=P + 2), 3, "aligned"),
    (dict(weights=P + 4), 1, "overlap"),
    (dict(ids=2 * P), 1, "overlap"),
    (dict(bias=7 * P, ids=7 * P), 1, "overlap"),
])
def test_route_refuses(kw, status, msg):
    assert route(**kw) == status, L.w4a16_last_error()
    assert msg in L.w4a16_last_error()


@pytest.mark.parametrize("kw,status,msg", ROUTER + [
    (dict(dw=None), 1, "NULL"),
    (dict(out=None), 1, "NULL"),
    (dict(out=4 * P + 1), 3, "aligned"),
    (dict(out=2 * P), 1, "overlap"),
    (dict(out=P + 32), 1, "overlap"),
])
def test_route_backward_refuses(kw, status, msg):
    assert route_backward(**kw) == status, L.w4a16_last_error()
    assert msg in L.w4a16_last_error()


@pytest.mark.parametrize("kw,status,msg", [
    (dict(dt=2), 1, "fp16 (0) or bf16"),
    (dict(M=-1), 1, "M >= 0"),
    (dict(K=0), 1, "K >= 1"),
    (dict(K=(1 << 24) + 1), 2, "too large"),
    (dict(M=1 << 30, K=4096), 2, "too large"),
    (dict(x=None), 1, "NULL"),
    (dict(x=P + 1), 3, "2-byte"),
    (dict(codes=2 * P + 8), 3, "16-byte"),
    (dict(scales=3 * P + 2), 3, "4-byte"),
    (dict(codes=P), 1, "overlap"),
    (dict(scales=2 * P + 4), 1, "overlap"),
])
def test_quantize_refuses(kw, status, msg):
    assert quantize(**kw) == status, L.w4a16_last_error()
    assert msg in L.w4a16_last_error()


PRODUCT = [
    (dict(dt=2), 1, "outputs must be"),
    (dict(xdt=0), 1, "output's type or e4m3"),
    (dict(sdt=1), 1, "fp32 or e8m0"),
    (dict(M=-1), 1, "M >= 0"),
    (dict(N=0), 1, "N >= 1"),
    (dict(K=0), 1, "K >= 1"),
    (dict(K=250), 2, "multiple of 16"),
    (dict(tr=1, N=60), 2, "multiple of 16"),
    (dict(N=1 << 25), 2, "too large"),
    (dict(K=1 << 25), 2, "too large"),
    (dict(x=None), 1, "NULL"),
    (dict(w=None), 1, "NULL"),
    (dict(ws=None), 1, "NULL"),
    (dict(y=None), 1, "NULL"),
    (dict(xdt=3), 1, "NULL"),                 # codes without their scales
    (dict(xs=8 * P), 1, "go with e4m3"),
    (dict(w=2 * P + 8), 3, "16-byte"),
    (dict(xdt=3, xs=8 * P, x=P + 8), 3, "16-byte"),
    (dict(x=P + 1), 3, "2-byte"),
    (dict(ws=3 * P + 2), 3, "4-byte"),
    (dict(xdt=3, xs=8 * P + 2), 3, "4-byte"),
    (dict(bias=9 * P + 1), 3, "2-byte"),
    (dict(y=P + 64), 1, "overlap"),
    (dict(y=2 * P + 64), 1, "overlap"),
    (dict(bias=9 * P, y=9 * P), 1, "overlap"),
]


@pytest.mark.parametrize("kw,status,msg", PRODUCT)
def test_linear_refuses(kw, status, msg):
    assert linear(**kw) == status, L.w4a16_last_error()
    assert msg in L.w4a16_last_error()


@pytest.mark.parametrize("kw,status,msg", PRODUCT + [
    (dict(E=0), 1, "E >= 1"),
    (dict(E=1025), 2, "1024 experts"),
    (dict(topk=0), 1, "topk >= 1"),
    (dict(M=1 << 20, topk=1 << 20), 2, "slots"),
    (dict(ids=None), 1, "NULL"),
    (dict(ids=6 * P + 2), 3, "4-byte"),
    (dict(tw=7 * P + 2), 3, "4-byte"),
    (dict(y=6 * P), 1, "overlap"),
])
def test_moe_refuses(kw, status, msg):
    if "M" in kw and kw["M"] == -1:
        msg = "M >= 0"
    assert moe(**kw) == status, L.w4a16_last_error()
    assert msg in L.w4a16_last_error()


def test_empty_batches_are_no_ops():
    assert route(M=0, logits=None, weights=None, ids=None) == 0
    assert route_backward(M=0, dw=None, logits=None, ids=None, out=None) == 0
    assert quantize(M=0, x=None, codes=None, scales=None) == 0
    assert linear(M=0, x=None, y=None, work=None, n=0) == 0
    assert moe(M=0, x=None, y=None, ids=None, work=None, n=0) == 0


def test_workspace_sizes():
    # counters, then codes and scales of x
    assert L.w4a16_minifloat_linear_workspace_size(4, 64, 256, L.W4A16_BF16) >= 65536 + 4 * 256 + 16
    assert L.w4a16_minifloat_linear_workspace_size(0, 64, 256, L.W4A16_BF16) == 0
    small = L.w4a16_minifloat_moe_workspace_size(4, 2, 8, 64, 256, L.W4A16_BF16)
    per_slot = L.w4a16_minifloat_moe_workspace_size(4, 2, 8, 64, 256, L.W4A16_BF16, x_per_slot=True)
    assert 65536 < small < per_slot
    assert L.w4a16_minifloat_moe_workspace_size(4, 2, 0, 64, 256, L.W4A16_BF16) == 0
    assert L.w4a16_minifloat_moe_workspace_size(1 << 30, 1 << 30, 8, 64, 256, L.W4A16_BF16) == 0


def test_binding_checks_types():
    torch = pytest.importorskip("torch")
    w, s = torch.zeros((64, 256)).to(torch.float8_e4m3fn), torch.ones((1, 2))
    x = torch.zeros((3, 256), dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="float8_e4m3fn"):
        L.w4a16_minifloat_linear(x, w.float(), s)
    with pytest.raises(TypeError, match="float32 or float8_e8m0fnu"):
        L.w4a16_minifloat_linear(x, w, s.half())
    with pytest.raises(ValueError, match="scales are"):
        L.w4a16_minifloat_linear(x, w, s[:, :1])
    with pytest.raises(ValueError, match="columns"):
        L.w4a16_minifloat_linear(x[:, :128].contiguous(), w, s)
    with pytest.raises(ValueError, match="codes need x_scales"):
        L.w4a16_minifloat_linear(x.to(torch.float8_e4m3fn), w, s)
    with pytest.raises(ValueError, match="go with float8_e4m3fn"):
        L.w4a16_minifloat_linear(x, w, s, dtype=torch.float16)
    with pytest.raises(ValueError, match="must be on|must be"):
        L.w4a16_minifloat_linear(x, w, s)  # host tensors
    with pytest.raises(TypeError, match="int32"):
        L.w4a16_minifloat_moe_linear(x, w[None], s[None], torch.zeros((3, 2), dtype=torch.int64))
    with pytest.raises(ValueError, match="x must be 2-D"):
        L.w4a16_minifloat_moe_linear(x, w[None], s[None], torch.zeros((2, 2), dtype=torch.int32))
    with pytest.raises(ValueError, match="score must be"):
        L._binding._score_code("relu")
    with pytest.raises(TypeError, match="bias must be float32"):
        L.w4a16_route(torch.zeros((2, 8)), 2, torch.zeros(8, dtype=torch.float16))
    with pytest.raises(TypeError, match="dweights"):
        L.w4a16_route_backward(torch.zeros((2, 3)), torch.zeros((2, 8)), torch.zeros((2, 2), dtype=torch.int32))
