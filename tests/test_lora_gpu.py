"""Low-rank adapters beside the projection, through the C ABI, against the
float64 oracle: every kernel the dispatcher picks, token orders, ranks, ragged
sizes, tokens without an adapter, and the call's refusals.

Tolerances, fixed before the first run: y as the linear layer's (gpu_util.TOL
of max|y|).  u is a sum of K products accumulated in fp32: within
2^-24 (K / 32 + 32) of sum |x||A| (an fp32 sum in MFMA chunks of 32 k, the
chunks' sums chained, then at most 32 waves and ranges added)."""
import numpy as np
import pytest

import oracle as O
from oracle import adapters_ref as A
from synth import make_case
from synth.gen import stream_seed, to_act_bits
from gpu_util import DeviceCase, assert_close, bits_to_device, device_to_bits, note

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import int4_weight_only_linear_amd as L  # noqa: E402


@pytest.fixture(autouse=True)
def _need_gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    note(f"[gpu] {request.node.nodeid}")


def draw_ids(rng, M, S, order):
    if order == "one":
        return np.full(M, S - 1, dtype=np.int32)
    ids = rng.integers(-1, S + 1, M).astype(np.int32)  # -1 and S: no adapter
    return np.sort(ids) if order == "runs" else ids


class LoraCase:
    def __init__(self, M, N, K, group, dt, sym, bias, S, R, order, seed=0, alpha=True):
        self.c = make_case(M, N, K, group, dt, sym, bias, seed=("lora", seed, M, N, K, group))
        rng = np.random.default_rng(stream_seed("adapters", seed, M, N, K, S, R))
        self.S, self.R = S, R
        self.la = to_act_bits(rng.normal(0, K ** -0.5, (S, R, K)).astype(np.float32), dt)
        self.lb = to_act_bits(rng.normal(0, 2 * R ** -0.5, (S, N, R)).astype(np.float32), dt)
        self.ids = draw_ids(rng, M, S, order)
        self.alpha = rng.uniform(0.5, 3, S).astype(np.float32) if alpha else None
        self.d = DeviceCase(self.c)
        dev = self.d.x.device
        self.t_la, self.t_lb = bits_to_device(self.la, dt, dev), bits_to_device(self.lb, dt, dev)
        self.t_ids = torch.from_numpy(self.ids).to(dev)
        self.t_alpha = None if self.alpha is None else torch.from_numpy(self.alpha).to(dev)

    def run(self, **kw):
        d = self.d
        return L.w4a16_lora_linear(d.x, d.wq, d.s, self.t_la, self.t_lb, self.t_ids, d.zp, d.bias, self.t_alpha,
                                   group_size=self.c.group, **kw)

    def ref(self):
        c = self.c
        zpk = None if c.zp is None else O.pack_zeros(c.zp)
        return A.lora_linear_ref(c.x_bits, O.pack_weights(c.q), c.s_bits, zpk, c.bias_bits, self.la, self.lb, self.ids,
                                 self.alpha, c.M, c.N, c.K, c.group, self.S, self.R, c.dtype)


def check(case, y, u=None):
    ry, ru = case.ref()
    c = case.c
    assert_close(device_to_bits(y), ry, c.dtype, "y")
    if u is not None:
        x = np.abs(O.act_bits_to_f64(c.x_bits.reshape(c.M, c.K), c.dtype))
        la = np.abs(O.act_bits_to_f64(case.la, c.dtype))
        bound = np.zeros_like(ru)
        for m, a in enumerate(case.ids.tolist()):
            if 0 <= a < case.S:
                bound[m] = la[a] @ x[m]
        err = np.abs(u.double().cpu().numpy() - ru)
        assert np.all(err <= 2.0 ** -24 * (c.K / 32 + 32) * bound), float(err.max())


# (M, N, K, group, dtype, sym, bias, S, R, order)
CASES = [
    (1, 64, 256, 32, O.BF16, True, False, 1, 8, "one"),          # the few-token decode instance
    (1, 272, 4096, 128, O.BF16, False, True, 5, 16, "mixed"),
    (4, 256, 1024, 64, O.F16, False, True, 3, 24, "mixed"),
    (8, 96, 2560, 128, O.BF16, True, False, 8, 64, "mixed"),
    (5, 40, 16384, 64, O.F16, True, True, 2, 128, "runs"),       # decode with a long K, several ranges of u
    (3, 48, 28672, 32, O.BF16, False, False, 4, 16, "mixed"),    # decode split K
    (16, 80, 1056, 32, O.F16, False, True, 20, 16, "mixed"),     # the general decode kernel, ragged K
    (13, 51, 2592, 32, O.BF16, True, True, 6, 40, "mixed"),      # ragged N and K
    (24, 200, 512, 128, O.F16, False, False, 7, 8, "mixed"),     # 32-token GEMM tiles
    (33, 333, 1184, 32, O.BF16, True, True, 33, 16, "mixed"),
    (67, 264, 2560, 64, O.F16, True, False, 16, 32, "mixed"),    # 128-token tiles
    (129, 520, 1024, 128, O.BF16, False, True, 3, 72, "runs"),
    (300, 256, 4096, 128, O.BF16, False, False, 1, 16, "one"),
    (515, 1032, 640, 128, O.F16, True, True, 9, 128, "mixed"),
    (700, 8264, 256, 64, O.BF16, False, False, 4, 48, "runs"),   # tall tiles with a tail launch
]


@pytest.mark.parametrize("M,N,K,group,dt,sym,bias,S,R,order", CASES)
def test_forward(M, N, K, group, dt, sym, bias, S, R, order):
    case = LoraCase(M, N, K, group, dt, sym, bias, S, R, order)
    check(case, case.run())
    y, u = case.run(save_u=True)
    check(case, y, u)


@pytest.mark.parametrize("M", [1, 7, 16, 40, 200])
def test_no_adapter_is_the_linear_layer(M):
    # every id outside the stack: bit for bit w4a16_linear's output, u zero
    case = LoraCase(M, 144, 512, 64, O.BF16, False, True, 3, 16, "mixed", alpha=False)
    case.t_ids.copy_(torch.tensor([-1, 3, -(1 << 31), (1 << 31) - 1] * M, dtype=torch.int32)[:M])
    y, u = case.run(save_u=True)
    d = case.d
    base = L.w4a16_linear(d.x, d.wq, d.s, d.zp, d.bias, group_size=64)
    assert torch.equal(y.view(torch.int16), base.view(torch.int16))
    assert torch.count_nonzero(u) == 0


@pytest.mark.parametrize("M", [3, 50, 400])
def test_unnamed_adapters_are_never_used(M):
    # NaN and infinity in the stacks of adapters that no token names, and in
    # the activations of tokens without an adapter, stay where they are
    case = LoraCase(M, 136, 768, 128, O.F16, False, False, 4, 16, "mixed", seed=1)
    ids = case.t_ids
    ids[ids == 2] = 1
    clean = case.run()
    case.t_la[2], case.t_lb[2] = float("nan"), float("inf")
    assert torch.equal(case.run().view(torch.int16), clean.view(torch.int16))
    ids[0] = -1
    clean = case.run()
    case.d.x[0] = float("nan")
    y, u = case.run(save_u=True)
    assert torch.isnan(y[0]).all() and torch.count_nonzero(u[0]) == 0
    assert torch.equal(y[1:].view(torch.int16), clean[1:].view(torch.int16))


def test_repeated_calls_and_shared_workspace():
    # same inputs, same bits; one workspace serves other shapes in between
    # (its counters come back zero) and other streams have their own
    a = LoraCase(16, 96, 28672, 128, O.BF16, False, False, 6, 32, "mixed")
    b = LoraCase(90, 200, 1024, 64, O.F16, True, True, 5, 16, "mixed")
    ya, yb = a.run(), b.run()
    for _ in range(3):
        assert torch.equal(a.run().view(torch.int16), ya.view(torch.int16))
        assert torch.equal(b.run().view(torch.int16), yb.view(torch.int16))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y2 = a.run()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert torch.equal(y2.view(torch.int16), ya.view(torch.int16))


@pytest.mark.parametrize("M", [2, 64, 300])
def test_graph_replays(M):
    case = LoraCase(M, 256, 2048, 128, O.BF16, False, False, 5, 16, "mixed")
    dt = O.BF16
    c = case.c
    ws = torch.zeros(L.w4a16_lora_workspace_size(M, c.N, c.K, c.group, L.W4A16_BF16, True, 16), dtype=torch.uint8,
                     device="cuda")
    out = torch.empty((M, c.N), dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        case.run(out=out, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        case.run(out=out, workspace=ws)
    for i in range(4):
        case.d.x.copy_(torch.randn_like(case.d.x))
        case.t_ids.copy_(case.t_ids.roll(1))
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        eager = case.run()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), eager.view(torch.int16)), (dt, i)


def test_refusals():
    case = LoraCase(4, 64, 256, 32, O.BF16, True, False, 2, 8, "mixed")
    d = case.d
    ok = lambda **kw: L.w4a16_lora_linear(**{**dict(x=d.x, wq=d.wq, scales=d.s, la=case.t_la, lb=case.t_lb,  # noqa: E731
                                                    ids=case.t_ids, group_size=32), **kw})
    ok()
    with pytest.raises(TypeError):
        ok(ids=case.t_ids.long())
    with pytest.raises(TypeError):
        ok(la=case.t_la.half(), lb=case.t_lb.half())
    with pytest.raises(ValueError):
        ok(lb=case.t_lb[:, :32].contiguous())
    with pytest.raises(ValueError):
        ok(la=case.t_la.transpose(0, 1).contiguous().transpose(0, 1))
    with pytest.raises(L.W4A16Error, match="multiple of 8"):
        ok(la=torch.zeros(2, 12, 256, dtype=torch.bfloat16, device="cuda"),
           lb=torch.zeros(2, 64, 12, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(L.W4A16Error, match="128"):
        ok(la=torch.zeros(2, 136, 256, dtype=torch.bfloat16, device="cuda"),
           lb=torch.zeros(2, 64, 136, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(L.W4A16Error, match="WORKSPACE"):
        ok(workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        ok(alpha=torch.ones(2, dtype=torch.float64, device="cuda"))
    # no tokens: nothing to do
    y = ok(x=d.x[:0], ids=case.t_ids[:0])
    assert y.shape == (0, 64)


@pytest.mark.parametrize("dt", [O.F16, O.BF16])
@pytest.mark.parametrize("M", [9, 50, 150, 700])
def test_a_broken_adapter_stays_with_its_tokens(M, dt):
    # infinities and NaN in adapters that some tokens name: everyone else's
    # outputs keep their bits, on every kernel and tile
    case = LoraCase(M, 192, 512, 64, dt, False, True, 4, 24, "mixed", seed=9)
    y = case.run()
    for value, up in ((float("inf"), True), (float("nan"), True), (float("nan"), False)):
        la, lb = case.t_la.clone(), case.t_lb.clone()
        (lb if up else la)[2, 7, 5] = value
        (lb if up else la)[1] = value
        d = case.d
        got = L.w4a16_lora_linear(d.x, d.wq, d.s, la, lb, case.t_ids, d.zp, d.bias, case.t_alpha, group_size=64)
        clean = torch.from_numpy((case.ids != 1) & (case.ids != 2)).cuda()
        assert torch.equal(got[clean], y[clean]), (value, up)
        assert not torch.isfinite(got[case.t_ids == 1]).any()
        assert not torch.isfinite(got[case.t_ids == 2]).all(dim=1).any()
