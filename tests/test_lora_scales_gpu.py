"""fp16 adapters whose products are far from 1 (factors B that training has
just begun to move from zero, scaled losses, large alpha): the second product
and the gradients keep their precision whatever the size of u and g.

The projection's scales are zero, so the adapters' terms are the whole outputs.
Tolerances, fixed before the first run.  The factors of a sum are exact inputs
and w = alpha u or g, carried to 2^-23 of the largest of its row (a token's
ranks in y and dx, a rank's 32 tokens in dla and dlb), after an fp32 sum that is
itself within 2^-24 (n / 32 + 40) of its products' magnitudes (32 of a chunk,
the chunks chained, at most 40 waves and ranges).  The products are again summed
in fp32.  The result is rounded once: 2^-11 of itself, or 2^-25."""
import numpy as np
import pytest

import oracle as O
from synth.gen import to_act_bits
from gpu_util import device_to_bits, note
from test_lora_gpu import L, torch
from test_lora_backward_gpu import Grad

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


@pytest.fixture(autouse=True)
def _need_gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    note(f"[gpu] {request.node.nodeid}")


def sums(n):
    return E * (n / 32 + 40)


class Scaled(Grad):
    """Adapter s at 2^up[s] (B, and alpha), token m's x and dy at 2^x_by[m], 2^dy_by[m]."""

    def __init__(self, M, N, K, S, R, order, b_by, alpha_by, x_by, dy_by):
        super().__init__(M, N, K, 32, O.F16, True, S, R, order, seed=3)
        c = self.c
        val = lambda b: O.act_bits_to_f64(b, O.F16)  # noqa: E731
        pick = lambda v, n: np.array([v[i % len(v)] for i in range(n)])  # noqa: E731
        self.d.s.zero_()
        c.s_bits = np.zeros_like(c.s_bits)
        self.lb = to_act_bits((val(self.lb) * 2.0 ** pick(b_by, S)[:, None, None]).astype(np.float32), O.F16)
        self.alpha = (self.alpha * 2.0 ** pick(alpha_by, S)).astype(np.float32)
        c.x_bits = to_act_bits((val(c.x_bits).reshape(M, K) * 2.0 ** pick(x_by, M)[:, None]).astype(np.float32), O.F16)
        self.dy = to_act_bits((val(self.dy).reshape(M, N) * 2.0 ** pick(dy_by, M)[:, None]).astype(np.float32), O.F16)
        up = lambda t, b: t.copy_(torch.from_numpy(val(b).reshape(tuple(t.shape))).to(torch.float16))  # noqa: E731
        up(self.t_lb, self.lb), up(self.d.x, c.x_bits), up(self.t_dy, self.dy)
        self.t_alpha.copy_(torch.from_numpy(self.alpha))
        self.x64, self.la64, self.lb64, self.dy64 = (val(b).reshape(s) for b, s in (
            (c.x_bits, (M, K)), (self.la, (S, R, K)), (self.lb, (S, N, R)), (self.dy, (M, N))))
        self.u = np.zeros((M, R), dtype=np.float32)
        for m, a in enumerate(self.ids.tolist()):
            if 0 <= a < S:
                self.u[m] = self.la64[a] @ self.x64[m]
        self.t_u.copy_(torch.from_numpy(self.u))

    def named(self):
        return [(m, a, float(self.alpha[a])) for m, a in enumerate(self.ids.tolist()) if 0 <= a < self.S]


def close(t, want, slack, what):
    got = O.act_bits_to_f64(device_to_bits(t), O.F16)
    over = np.abs(want) > 65504 * (1 - 2.0 ** -11)  # fp16 has no such value: infinite, or its largest one
    bound = 2.0 ** -11 * np.abs(want) + 2.0 ** -25 + slack
    bad = ~(np.abs(got - want) <= bound) & ~(over & (np.abs(got) >= 65504 * (1 - 2.0 ** -10)) & (np.sign(got) == np.sign(want)))
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], want[bad][:4], bound[bad][:4])


def run(case):
    c, S, R = case.c, case.S, case.R
    # forward
    want, slack = np.zeros((c.M, c.N)), np.zeros((c.M, c.N))
    for m, a, k in case.named():
        u = k * (case.la64[a] @ case.x64[m])
        du = abs(k) * sums(c.K) * (np.abs(case.la64[a]) @ np.abs(case.x64[m])) + 2.0 ** -23 * np.abs(u).max()
        b = np.abs(case.lb64[a])
        want[m] = case.lb64[a] @ u
        slack[m] = b @ du + sums(R) * (b @ np.abs(u))
    y, u = case.run(save_u=True)
    close(y, want, slack, "y")
    assert torch.equal(case.run().view(torch.int16), y.view(torch.int16))
    # gradients
    dx, dxs = np.zeros((c.M, c.K)), np.zeros((c.M, c.K))
    ga, gas = np.zeros((S, R, c.K)), np.zeros((S, R, c.K))
    gb, gbs = np.zeros((S, c.N, R)), np.zeros((S, c.N, R))
    for s in range(S):
        rows, k = np.nonzero(case.ids == s)[0], float(case.alpha[s])
        g = k * case.dy64[rows] @ case.lb64[s]
        dg = abs(k) * sums(c.N) * (np.abs(case.dy64[rows]) @ np.abs(case.lb64[s]))
        w = k * case.u[rows].astype(np.float64)
        a = np.abs(case.la64[s])
        top = 2.0 ** -23 * np.abs(g).max(1, keepdims=True) if len(rows) else 0
        dx[rows] = g @ case.la64[s]
        dxs[rows] = (dg + top) @ a + sums(R) * (np.abs(g) @ a)
        step = np.arange(len(rows)) // 32  # the adapter's tokens, 32 at a time
        peak = lambda v: np.array([np.abs(v[step == t]).max(0) for t in step]).reshape(v.shape)  # noqa: E731
        ax, ady = np.abs(case.x64[rows]), np.abs(case.dy64[rows])
        ga[s], gb[s] = g.T @ case.x64[rows], case.dy64[rows].T @ w
        gas[s] = (dg + 2.0 ** -23 * peak(g)).T @ ax + sums(len(rows)) * (np.abs(g).T @ ax)
        gbs[s] = ady.T @ (2 * E * np.abs(w) + 2.0 ** -23 * peak(w)) + sums(len(rows)) * (ady.T @ np.abs(w))
    got = case.backward()
    for t, w, sl, what in zip(got, (dx, ga, gb), (dxs, gas, gbs), ("dx", "dla", "dlb")):
        close(t, w, sl, what)
    again = case.backward(need_dx=False)[1:]
    assert all(torch.equal(p.view(torch.int16), q.view(torch.int16)) for p, q in zip(got[1:], again))


SHAPES = [(40, 72, 256, 3, 24, "mixed"),     # 32-token tiles, one K range of u
          (150, 200, 1184, 2, 40, "mixed"),  # 128-token tiles, several ranges
          (33, 96, 64, 1, 8, "one"),
          (700, 130, 544, 3, 72, "runs"),
          (1300, 48, 96, 1, 128, "one")]     # one adapter's tokens over several workgroups


@pytest.mark.parametrize("M,N,K,S,R,order", SHAPES)
@pytest.mark.parametrize("b_by,alpha_by,x_by,dy_by", [
    ((-13,), (0,), (0,), (0,)),                    # B just begun: g about 1e-5
    ((-10,), (-3,), (4,), (-6,)),                  # and small gradients: 1e-6
    ((0,), (0,), (-9,), (0,)),                     # small activations: u about 1e-3
    ((4,), (-16,), (0,), (0,)),                    # small alpha, large B
    ((-10,), (19,), (0,), (0,)),                   # alpha u past fp16's range
    ((-8, 0, 3), (0, 5, -4), (-8, 0, 0, 5), (0, -12, 3, -4, 0)),   # adapters and tokens of all sizes, mixed
])
def test_products_of_any_size(M, N, K, S, R, order, b_by, alpha_by, x_by, dy_by):
    run(Scaled(M, N, K, S, R, order, b_by, alpha_by, x_by, dy_by))


def test_tokens_of_ordinary_size_keep_their_bits():
    # beside tokens whose operands are shifted, and in a rank of zeros
    case = Scaled(200, 72, 256, 2, 16, "mixed", (0,), (0,), (0,), (0,))
    case.t_la[:, 3] = 0
    y, dx = case.run(), case.backward()[0]
    odd = torch.arange(0, 200, 7, device="cuda")
    case.d.x[odd] *= 2.0 ** -10
    case.t_dy[odd] *= 2.0 ** -10
    keep = torch.ones(200, dtype=torch.bool, device="cuda")
    keep[odd] = False
    assert torch.equal(case.run()[keep].view(torch.int16), y[keep].view(torch.int16))
    assert torch.equal(case.backward()[0][keep].view(torch.int16), dx[keep].view(torch.int16))


def test_zero_factors_give_zeros():
    case = Scaled(90, 64, 128, 2, 16, "mixed", (0,), (0,), (0,), (0,))
    case.t_lb.zero_()
    assert torch.count_nonzero(case.run()) == 0
    dx, dla, dlb = case.backward()
    assert torch.count_nonzero(dx) == 0 and torch.count_nonzero(dla) == 0 and torch.count_nonzero(dlb) > 0
