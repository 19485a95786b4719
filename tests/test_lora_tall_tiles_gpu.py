"""Adapters on the tiles that large calls take: 192 and 256 tokens, the launch of
half-height tiles after the last full round, and the input gradient's 128- and
256-token tiles, whole and in ranges of n.  Every test asserts the plan that it
is there for, so that a change of the planners cannot take the cover away.
Mixed tokens, ranks that end inside a step of 16, ragged rows, one token past a
tile; checked on the tokens at the tiles' edges and a sample of the others.

Tolerances as in test_lora_gpu.py and test_lora_backward_gpu.py."""
import re

import numpy as np
import pytest

import oracle as O
from synth import make_case
from synth.gen import stream_seed, to_act_bits
from gpu_util import TOL, DeviceCase, bits_to_device, device_to_bits, note
from test_lora_gpu import L, draw_ids, torch
from test_lora_backward_gpu import check_sum

pytestmark = pytest.mark.gpu

PATH_GEMM = L.PATH_GEMM


@pytest.fixture(autouse=True)
def _need_gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    note(f"[gpu] {request.node.nodeid}")


@pytest.fixture
def tuned(monkeypatch):
    def set_(name, value):
        monkeypatch.setenv(name, value)
        L.w4a16_reload_tuning()
    yield set_
    monkeypatch.undo()
    L.w4a16_reload_tuning()


class Large:
    """A case whose references are formed for chosen tokens only."""

    def __init__(self, M, N, K, group, dt, sym, bias, S, R, seed=0):
        self.M, self.N, self.K, self.group, self.dt, self.S, self.R = M, N, K, group, dt, S, R
        self.c = make_case(M, N, K, group, dt, sym, bias, seed=("tall", seed, M, N, K))
        rng = self.rng = np.random.default_rng(stream_seed("tall adapters", seed, M, N, K, R))
        self.la = to_act_bits(rng.normal(0, K ** -0.5, (S, R, K)).astype(np.float32), dt)
        self.lb = to_act_bits(rng.normal(0, 2 * R ** -0.5, (S, N, R)).astype(np.float32), dt)
        self.ids = draw_ids(rng, M, S, "mixed")
        self.alpha = rng.uniform(0.5, 3, S).astype(np.float32)
        self.d = DeviceCase(self.c)
        dev = self.d.x.device
        self.t_la, self.t_lb = bits_to_device(self.la, dt, dev), bits_to_device(self.lb, dt, dev)
        self.t_ids, self.t_alpha = torch.from_numpy(self.ids).to(dev), torch.from_numpy(self.alpha).to(dev)
        val = lambda b, shape: O.act_bits_to_f64(b.reshape(shape), dt)  # noqa: E731
        self.x, self.A, self.B = val(self.c.x_bits, (M, K)), val(self.la, (S, R, K)), val(self.lb, (S, N, R))
        zpk = None if sym else O.pack_zeros(self.c.zp)
        self.W = O.dequant_f32(O.pack_weights(self.c.q), self.c.s_bits, zpk, N, K, group, dt)
        self.bias = None if not bias else val(self.c.bias_bits, (N,))

    def run(self, la=None, lb=None):
        d = self.d
        return L.w4a16_lora_linear(d.x, d.wq, d.s, self.t_la if la is None else la, self.t_lb if lb is None else lb,
                                   self.t_ids, d.zp, d.bias, self.t_alpha, group_size=self.group)

    def tokens(self, *edges):
        """The tokens around multiples of the tile heights, the last ones, and a sample."""
        at = {m + o for e in edges for m in range(0, self.M + e, e) for o in (-1, 0, 1)}
        at |= set(range(self.M - 3, self.M)) | set(self.rng.integers(0, self.M, 40).tolist())
        return np.array(sorted(m for m in at if 0 <= m < self.M))

    def y_ref(self, rows):
        y = self.x[rows] @ self.W.T.astype(np.float64)
        if self.bias is not None:
            y += self.bias
        for i, m in enumerate(rows.tolist()):
            a = int(self.ids[m])
            if 0 <= a < self.S:
                y[i] += float(self.alpha[a]) * (self.B[a] @ (self.A[a] @ self.x[m]))
        return y


def close(t, rows, want, dt, what):
    got = O.act_bits_to_f64(device_to_bits(t[torch.from_numpy(rows).to(t.device)]), dt)
    assert np.isfinite(t.float().sum(dim=1).cpu().numpy()).all(), what
    err, scale = np.abs(got - want).max(), np.abs(want).max()
    assert err <= TOL[dt] * scale, (what, float(err), float(scale))


# (M, N, K, group, dtype, R), tile tokens and features, tail tile tokens
NATURAL = [
    ((391, 16424, 64, 32, O.BF16, 24), (192, 256, 0)),
    ((129, 16816, 64, 32, O.F16, 40), (256, 128, 0)),
    ((588, 16768, 64, 32, O.BF16, 128), (256, 256, 0)),
    ((388, 21912, 128, 128, O.F16, 8), (256, 256, 0)),
    ((263, 21832, 128, 128, O.F16, 40), (192, 256, 0)),
    ((854, 18736, 1024, 32, O.F16, 24), (256, 128, 128)),
    ((1413, 24744, 1024, 32, O.BF16, 40), (256, 256, 128)),
    ((1413, 24744, 1024, 128, O.F16, 72), (256, 256, 128)),
]


@pytest.mark.parametrize("shape,plan", NATURAL)
def test_forward(shape, plan):
    M, N, K, group, dt, R = shape
    p = L.w4a16_plan(M, N, K, group, dt, True)
    assert (p["path"], p["tile_tokens"], p["tile_features"], p["tail_tile_tokens"]) == (PATH_GEMM, *plan)
    case = Large(M, N, K, group, dt, False, True, 5, R)
    y = case.run()
    rows = case.tokens(plan[0], plan[2] or plan[0])
    close(y, rows, case.y_ref(rows), dt, "y")
    assert torch.equal(case.run().view(torch.int16), y.view(torch.int16))


# every tile height and width, in one and in several K ranges (one pass, two)
FORCED = [(1, 1, 0, 1), (1, 3, 0, 2), (1, 3, 1, 1), (4, 1, 0, 1), (4, 2, 0, 2), (4, 3, 1, 2), (6, 1, 0, 2), (6, 3, 0, 2),
          (8, 1, 0, 1), (8, 2, 0, 1), (8, 1, 0, 2), (8, 3, 0, 2)]


@pytest.mark.parametrize("R", [24, 40, 128])
@pytest.mark.parametrize("dt", [O.F16, O.BF16])
@pytest.mark.parametrize("mb,splits,two_pass,cb", FORCED)
def test_forward_on_every_tile(tuned, mb, splits, two_pass, cb, dt, R):
    M, N, K, group = 64 * mb + 1, 333, 1184, 32
    tuned("W4A16_GEMM_TILE", f"{mb},{splits},{two_pass},{cb}")
    p = L.w4a16_plan(M, N, K, group, dt, False)
    assert (p["path"], p["tile_tokens"], p["tile_features"], p["splits"], p["two_pass"]) == (PATH_GEMM, 32 * mb, 128 * cb, splits, two_pass)
    case = Large(M, N, K, group, dt, True, True, 7, R)
    y = case.run()
    rows = np.arange(M)
    close(y, rows, case.y_ref(rows), dt, "y")
    # infinities and NaN of two adapters stay with their tokens
    clean = torch.from_numpy((case.ids != 1) & (case.ids != 2)).cuda()
    for value, up in ((float("inf"), True), (float("nan"), False)):
        la, lb = case.t_la.clone(), case.t_lb.clone()
        (lb if up else la)[2, 7, 5] = value
        (lb if up else la)[1] = value
        got = case.run(la, lb)
        assert torch.equal(got[clean].view(torch.int16), y[clean].view(torch.int16)), (value, up)
        assert not torch.isfinite(got[case.t_ids == 1]).any()
        assert not torch.isfinite(got[case.t_ids == 2]).all(dim=1).any()


# (M, N, K, R), dx tile tokens, whether n is in ranges
BACKWARD = [((1803, 264, 2080, 24), 128, False), ((779, 8768, 64, 40), 128, True),
            ((1707, 67, 4640, 128), 256, False), ((258, 4907, 4416, 24), 256, True)]


@pytest.mark.parametrize("dt", [O.F16, O.BF16])
@pytest.mark.parametrize("shape,bm,split", BACKWARD)
def test_gradients(tuned, capfd, shape, bm, split, dt):
    M, N, K, R = shape
    S = 5
    case = Large(M, N, K, 32, dt, N % 8 != 0, False, S, R)
    rng = np.random.default_rng(1)
    dy_bits = to_act_bits(rng.normal(0, 0.1, (M, N)).astype(np.float32), dt)
    t_dy, dy = bits_to_device(dy_bits, dt, "cuda"), O.act_bits_to_f64(dy_bits.reshape(M, N), dt)
    u = np.zeros((M, R), dtype=np.float32)
    for s in range(S):
        u[case.ids == s] = case.x[case.ids == s] @ case.A[s].T
    d = case.d
    run = lambda la, lb: L.w4a16_lora_backward(t_dy, d.x, torch.from_numpy(u).cuda(), d.wq, d.s, la, lb, case.t_ids,  # noqa: E731
                                               d.zp, case.t_alpha, group_size=32)
    tuned("W4A16_LOG", "1")
    capfd.readouterr()
    dx, dla, dlb = run(case.t_la, case.t_lb)
    line = re.search(r"lora_backward .* dx bm=(\d+) splits=(\d+)", capfd.readouterr().err)
    assert line and int(line.group(1)) == bm and (int(line.group(2)) > 1) == split, line
    tuned("W4A16_LOG", "0")
    rows = case.tokens(bm)
    want = dy[rows] @ case.W.astype(np.float64)
    for i, m in enumerate(rows.tolist()):
        a = int(case.ids[m])
        if 0 <= a < S:
            want[i] += float(case.alpha[a]) * (dy[m] @ case.B[a]) @ case.A[a]
    close(dx, rows, want, dt, "dx")
    for s in range(S):
        at, k = case.ids == s, float(case.alpha[s])
        g = k * dy[at] @ case.B[s]
        check_sum(dla[s], g.T @ case.x[at], (k * np.abs(dy[at]) @ np.abs(case.B[s])).T @ np.abs(case.x[at]), dt)
        check_sum(dlb[s], k * dy[at].T @ u[at], k * np.abs(dy[at]).T @ np.abs(u[at]), dt)
    again = run(case.t_la, case.t_lb)
    assert all(torch.equal(p.view(torch.int16), q.view(torch.int16)) for p, q in zip((dx, dla, dlb), again))
    # infinities and NaN of one adapter stay with its tokens
    clean = case.t_ids != 2
    for value, down in ((float("inf"), True), (float("nan"), True), (float("nan"), False)):
        la, lb = case.t_la.clone(), case.t_lb.clone()
        (la if down else lb)[2, 7, 5] = value
        gx, ga, gb = run(la, lb)
        assert torch.equal(gx[clean].view(torch.int16), dx[clean].view(torch.int16)), (value, down)
        others = [0, 1, 3, 4]
        assert torch.equal(ga[others], dla[others]) and torch.equal(gb[others], dlb[others])
        assert not torch.isfinite(gx[~clean]).all(dim=1).any()
