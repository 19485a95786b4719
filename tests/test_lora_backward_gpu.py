"""Gradients of the projection with low-rank adapters, through the C ABI,
against the float64 formulas and against differences of the forward oracle.

Tolerances, fixed before the first run: dx like the linear layer's outputs
(gpu_util.TOL of its largest value: the same product with weights rounded to
the activation dtype).  dla and dlb are sums over tokens of products whose
factors carry at least 16 bits (the activation is exact, g and u are value +
remainder) in fp32: one final rounding (2^-8 bf16, 2^-11 fp16 of the value)
plus 2^-15 of the sum of the products' magnitudes."""
import numpy as np
import pytest

import oracle as O
from oracle import adapters_ref as A
from synth.gen import stream_seed, to_act_bits
from gpu_util import assert_close, bits_to_device, device_to_bits, note
from test_lora_gpu import LoraCase

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import int4_weight_only_linear_amd as L  # noqa: E402


@pytest.fixture(autouse=True)
def _need_gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    note(f"[gpu] {request.node.nodeid}")


class Grad(LoraCase):
    def __init__(self, M, N, K, group, dt, sym, S, R, order, seed=0, alpha=True):
        super().__init__(M, N, K, group, dt, sym, False, S, R, order, seed, alpha)
        rng = np.random.default_rng(stream_seed("dy", seed, M, N))
        self.dy = to_act_bits(rng.normal(0, 0.1, (M, N)).astype(np.float32), dt)
        self.t_dy = bits_to_device(self.dy, dt, self.d.x.device)
        self.u = A.lora_linear_ref(*self._args(), self.M_, self.N_, self.K_, group, S, R, dt)[1].astype(np.float32)
        self.t_u = torch.from_numpy(self.u).to(self.d.x.device)

    M_ = property(lambda self: self.c.M)
    N_ = property(lambda self: self.c.N)
    K_ = property(lambda self: self.c.K)

    def _args(self):
        c = self.c
        zpk = None if c.zp is None else O.pack_zeros(c.zp)
        return c.x_bits, O.pack_weights(c.q), c.s_bits, zpk, None, self.la, self.lb, self.ids, self.alpha

    def backward(self, **kw):
        d = self.d
        return L.w4a16_lora_backward(self.t_dy, d.x, self.t_u, d.wq, d.s, self.t_la, self.t_lb, self.t_ids, d.zp,
                                     self.t_alpha, group_size=self.c.group, **kw)

    def ref(self):
        c = self.c
        x, wq, s, zpk, _, la, lb, ids, alpha = self._args()
        return A.lora_backward_ref(self.dy, x, self.u, wq, s, zpk, la, lb, ids, alpha, c.M, c.N, c.K, c.group, self.S,
                                   self.R, c.dtype)

    def magnitudes(self):
        """Sums of the magnitudes of dla's and dlb's products."""
        c = self.c
        f = lambda b, shape: np.abs(O.act_bits_to_f64(b.reshape(shape), c.dtype))  # noqa: E731
        dy, x = f(self.dy, (c.M, c.N)), f(c.x_bits, (c.M, c.K))
        lb = f(self.lb, (self.S, c.N, self.R))
        pa, pb = np.zeros((self.S, self.R, c.K)), np.zeros((self.S, c.N, self.R))
        for s in range(self.S):
            rows = np.nonzero(self.ids == s)[0]
            k = 1.0 if self.alpha is None else float(self.alpha[s])
            pa[s] = (k * dy[rows] @ lb[s]).T @ x[rows]
            pb[s] = dy[rows].T @ (k * np.abs(self.u[rows]))
        return pa, pb


def check_sum(t, ref, mag, dt):
    got = O.act_bits_to_f64(device_to_bits(t), dt)
    unit = 2.0 ** -8 if dt == O.BF16 else 2.0 ** -11
    tiny = 2.0 ** -25 if dt == O.F16 else 0.0
    assert np.all(np.abs(got - ref) <= unit * np.abs(ref) + 2.0 ** -15 * mag + tiny), float(np.abs(got - ref).max())


# (M, N, K, group, dtype, sym, S, R, order)
CASES = [
    (1, 16, 32, 32, O.BF16, True, 1, 8, "one"),
    (5, 64, 256, 64, O.F16, False, 2, 16, "mixed"),
    (33, 51, 288, 32, O.BF16, True, 3, 24, "mixed"),        # N no multiple of 8, ragged last run
    (64, 200, 1056, 32, O.F16, False, 4, 32, "mixed"),
    (100, 130, 512, 128, O.F16, True, 20, 8, "mixed"),
    (128, 512, 640, 128, O.BF16, False, 1, 64, "one"),
    (257, 328, 2592, 32, O.BF16, False, 2, 128, "runs"),
    (700, 264, 544, 32, O.F16, True, 5, 40, "runs"),
    (1025, 1000, 256, 64, O.BF16, True, 1, 16, "one"),      # one adapter's tokens over several workgroups
    (1500, 96, 384, 128, O.BF16, False, 3, 48, "mixed"),
]


@pytest.mark.parametrize("M,N,K,group,dt,sym,S,R,order", CASES)
def test_gradients(M, N, K, group, dt, sym, S, R, order):
    case = Grad(M, N, K, group, dt, sym, S, R, order)
    dx, dla, dlb = case.backward()
    rx, ra, rb = case.ref()
    assert_close(device_to_bits(dx), rx, dt, "dx")
    pa, pb = case.magnitudes()
    check_sum(dla, ra, pa, dt)
    check_sum(dlb, rb, pb, dt)
    again = case.backward()
    assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip((dx, dla, dlb), again))
    none, dla2, dlb2 = case.backward(need_dx=False)
    assert none is None and torch.equal(dla2.view(torch.int16), dla.view(torch.int16))
    assert torch.equal(dlb2.view(torch.int16), dlb.view(torch.int16))


def test_per_channel_scales():
    case = Grad(70, 48, 384, 384, O.BF16, False, 2, 16, "mixed")
    dx, _, _ = case.backward()
    assert_close(device_to_bits(dx), case.ref()[0], O.BF16, "dx")


@pytest.mark.parametrize("dt", [O.F16, O.BF16])
def test_differences(dt):
    """The gradient of sum(dy * y) along random directions of x, A and B equals the central
    difference of the float64 forward formula: y is bilinear in each factor's direction, so the
    difference is exact up to float64, and what remains is the gradients' own error."""
    M, N, K, S, R = 40, 72, 256, 3, 16
    case = Grad(M, N, K, 64, dt, False, S, R, "mixed")
    got = [O.act_bits_to_f64(device_to_bits(t), dt) for t in case.backward()]
    dy = O.act_bits_to_f64(case.dy.reshape(M, N), dt)
    W = O.dequant_f32(O.pack_weights(case.c.q), case.c.s_bits, O.pack_zeros(case.c.zp), N, K, 64, dt).astype(np.float64)
    x = O.act_bits_to_f64(case.c.x_bits.reshape(M, K), dt)
    la, lb = O.act_bits_to_f64(case.la, dt), O.act_bits_to_f64(case.lb, dt)

    def loss(x, la, lb):
        y = x @ W.T
        for m, a in enumerate(case.ids.tolist()):
            if 0 <= a < S:
                y[m] += float(case.alpha[a]) * (lb[a] @ (la[a] @ x[m]))
        return float((dy * y).sum())

    rng = np.random.default_rng(1)
    for i, at in enumerate((x, la, lb)):
        for _ in range(3):
            v = rng.normal(0, 1, at.shape)
            args = [x, la, lb]
            hi, lo = list(args), list(args)
            hi[i], lo[i] = at + 0.5 * v, at - 0.5 * v
            want = loss(*hi) - loss(*lo)
            # independent roundings of the gradient's values: 6 standard deviations
            # of a sum of them, each at most the dtype's half spacing
            # (and as much again for the weights' rounding in dx)
            unit = 2.0 ** -8 if dt == O.BF16 else 2.0 ** -11
            sigma = unit * np.sqrt(np.square(got[i] * v).sum()) * 2
            assert abs(float((got[i] * v).sum()) - want) <= 6 * sigma


def test_tokens_without_adapter_and_unused_adapters():
    case = Grad(90, 64, 256, 64, O.BF16, True, 4, 16, "mixed")
    case.t_ids[case.t_ids == 1] = -1
    dx, dla, dlb = case.backward()
    assert torch.count_nonzero(dla[1]) == 0 and torch.count_nonzero(dlb[1]) == 0
    # infinities and NaN where nothing may look: adapters without tokens, u of
    # tokens without an adapter
    case.t_la[1], case.t_lb[1] = float("nan"), float("inf")
    case.t_u[case.t_ids < 0] = float("nan")
    again = case.backward()
    assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip((dx, dla, dlb), again))
    # x and dy of a token without an adapter stay out of dla and dlb
    m = int((case.t_ids < 0).nonzero()[0])
    case.d.x[m], case.t_dy[m] = float("inf"), float("nan")
    dx2, dla2, dlb2 = case.backward()
    assert torch.isnan(dx2[m]).all()
    keep = torch.arange(90, device="cuda") != m
    assert torch.equal(dx2[keep].view(torch.int16), dx[keep].view(torch.int16))
    assert torch.equal(dla2.view(torch.int16), dla.view(torch.int16)) and torch.equal(dlb2.view(torch.int16), dlb.view(torch.int16))
    # nobody has an adapter
    case.t_ids.fill_(99)
    _, dla, dlb = case.backward()
    assert torch.count_nonzero(dla) == 0 and torch.count_nonzero(dlb) == 0
    # no tokens
    e = case.d.x[:0]
    dx, dla, dlb = L.w4a16_lora_backward(case.t_dy[:0], e, case.t_u[:0], case.d.wq, case.d.s, case.t_la, case.t_lb,
                                         case.t_ids[:0], case.d.zp, case.t_alpha, group_size=64)
    assert dx.shape == (0, 256) and torch.count_nonzero(dla) == 0 and torch.count_nonzero(dlb) == 0


def test_infinite_dy_beside_ragged_rows():
    # rows of W past N weigh nothing, whatever dy's next row begins with
    case = Grad(66, 72, 128, 32, O.BF16, True, 1, 8, "one")
    case.t_dy[1::2] = float("inf")
    dx, _, _ = case.backward()
    rx = case.ref()[0]
    assert_close(device_to_bits(dx)[0::2], rx[0::2], O.BF16, "dx")
    assert not torch.isfinite(dx[1::2].float()).any()


@pytest.mark.parametrize("M", [70, 600])
def test_graph_replays(M):
    case = Grad(M, 264, 512, 64, O.BF16, False, 3, 16, "mixed")
    ws = torch.zeros(L.w4a16_lora_backward_workspace_size(M, 264, 512, 64, 3, 16, L.W4A16_BF16), dtype=torch.uint8, device="cuda")
    out = tuple(torch.empty_like(t) for t in (case.d.x, case.t_la, case.t_lb))
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    case.backward()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        case.backward(out=out, workspace=ws)
    for _ in range(4):
        case.t_dy.copy_(torch.randn_like(case.t_dy))
        case.t_ids.copy_(case.t_ids.roll(3))
        for t in out:
            t.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        eager = case.backward()
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(out, eager))


def test_outputs_right_before_inputs():
    # dx is as wide as x, not as dy: an input right behind it is no overlap
    M, N, K = 24, 512, 64
    case = Grad(M, N, K, 32, O.F16, True, 1, 8, "one")
    both = torch.empty(2, M, K, dtype=torch.float16, device="cuda")
    both[1] = case.d.x
    case.d.x = both[1]
    dx, _, _ = case.backward(out=(both[0], torch.empty_like(case.t_la), torch.empty_like(case.t_lb)))
    assert_close(device_to_bits(dx), case.ref()[0], O.F16, "dx")


def test_refusals():
    case = Grad(4, 64, 256, 32, O.BF16, True, 2, 8, "mixed")
    d = case.d
    ok = lambda **kw: L.w4a16_lora_backward(**{**dict(dy=case.t_dy, x=d.x, u=case.t_u, wq=d.wq, scales=d.s,  # noqa: E731
                                                      la=case.t_la, lb=case.t_lb, ids=case.t_ids, group_size=32), **kw})
    ok()
    with pytest.raises(ValueError):
        ok(dy=case.t_dy[:, :32].contiguous())
    with pytest.raises(TypeError):
        ok(dy=case.t_dy.half())
    with pytest.raises(TypeError):
        ok(u=case.t_u.double())
    with pytest.raises(ValueError):
        ok(out=(None, torch.empty_like(case.t_lb), torch.empty_like(case.t_lb)))
    with pytest.raises(L.W4A16Error, match="overlap"):
        ok(out=(d.x, torch.empty_like(case.t_la), torch.empty_like(case.t_lb)))
    with pytest.raises(L.W4A16Error, match="overlap"):
        ok(out=(None, case.t_la, torch.empty_like(case.t_lb)))
    with pytest.raises(L.W4A16Error, match="WORKSPACE"):
        ok(workspace=torch.zeros(4096, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("dt", [O.F16, O.BF16])
@pytest.mark.parametrize("M", [40, 150, 700])
def test_a_broken_adapter_stays_with_its_tokens(M, dt):
    # infinities and NaN in an adapter's factors: the other tokens' dx and the
    # other adapters' gradients keep their bits
    case = Grad(M, 192, 512, 64, dt, True, 4, 24, "mixed")
    d = case.d
    run = lambda la, lb: L.w4a16_lora_backward(case.t_dy, d.x, case.t_u, d.wq, d.s, la, lb, case.t_ids, d.zp,  # noqa: E731
                                               case.t_alpha, group_size=64)
    dx, dla, dlb = run(case.t_la, case.t_lb)
    for value, down in ((float("inf"), True), (float("nan"), True), (float("nan"), False)):
        la, lb = case.t_la.clone(), case.t_lb.clone()
        (la if down else lb)[2, 7, 5] = value
        gx, ga, gb = run(la, lb)
        clean = case.t_ids != 2
        assert torch.equal(gx[clean], dx[clean])
        others = [0, 1, 3]
        assert torch.equal(ga[others], dla[others]) and torch.equal(gb[others], dlb[others])
        assert not torch.isfinite(gx[~clean]).all(dim=1).any()
