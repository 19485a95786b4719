"""AdamW's parameters, bit for bit: the step written as single fp32 operations
(numpy rounds each once) gives the same p, in either state, whatever the other
elements of a block hold and from p = 0 too, where p is the update itself."""
import numpy as np
import pytest

from gpu_util import note
from test_adamw_gpu import HYPER, L, step, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    note(f"[gpu] {request.node.nodeid}")


def plain(p, g, m, v, h):
    f = np.float32
    gs = g * f(h["grad_scale"])
    m = m * f(h["beta1"]) + gs * f(1.0 - h["beta1"])
    v = v * f(h["beta2"]) + (gs * gs) * f(1.0 - h["beta2"])
    decay = f(1.0 - h["lr"] * h["weight_decay"])
    rate = f(h["lr"] / (1.0 - h["beta1"] ** h["step"]))
    root = f(1.0 / np.sqrt(1.0 - h["beta2"] ** h["step"]))
    return p * decay - (m / (np.sqrt(v) * root + f(h["eps"]))) * rate, m, v


@pytest.mark.parametrize("kw", [{}, dict(step=1, weight_decay=0.0), dict(eps=0.0, beta2=0.999), dict(eps=1e-3, step=10000)])
@pytest.mark.parametrize("scale", [1.0, 1e-3, 1e-9, 1e-18, 1e12])
@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("n", [256 * 200, 256 * 30 + 77])
def test_plain_sequence(bits, scale, kw, n):
    h = {**HYPER, **kw}
    rng = np.random.default_rng(17)
    f = np.float32
    p = np.where(rng.integers(0, 2, n), 0, rng.normal(0, 0.3, n)).astype(f)
    g = (rng.normal(0, 1, n) * np.exp(rng.normal(0, 2, n)) * scale).astype(f)
    g[:256 * 10:7] = 0
    blocks = (n + 255) // 256
    dev = lambda a: torch.from_numpy(a.copy()).cuda()  # noqa: E731
    if bits == 8:
        cm, cv = rng.integers(-127, 128, n).astype(np.int8), rng.integers(0, 256, n).astype(np.uint8)
        cm[:256 * 5], cv[:256 * 5] = 0, 0
        ms, rs = (rng.uniform(0.1, 1, blocks).astype(f) * f(scale) for _ in range(2))
        spread = lambda a: np.repeat(a, 256)[:n]  # noqa: E731
        c = cm.astype(f) * f(1 / 127)
        m = (c * np.abs(c)) * spread(ms)
        c = cv.astype(f) * f(1 / 255)
        r = (c * c) * spread(rs)
        v = r * r
        state = [dev(a) for a in (cm, cv, ms, rs)]
        more = dict(m_scales=[state[2]], v_scales=[state[3]])
    else:
        m, v = (rng.normal(0, 1, n) * scale).astype(f), np.square(rng.normal(0, 1, n) * scale).astype(f)
        state, more = [dev(m), dev(v)], {}
    t, copy = dev(p), torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    step(L.w4a16_adamw_plan([t], [dev(g)], [state[0]], [state[1]], copies=[copy], **more), seed=3, **kw)
    with np.errstate(all="ignore"):
        want, _, _ = plain(p, g, m, v, h)
    got = t.cpu().numpy()
    same = (got.view(np.uint32) == want.view(np.uint32)) | (np.isnan(got) & np.isnan(want))
    assert same.all(), (int((~same).sum()), got[~same][:4], want[~same][:4])
    assert torch.equal(copy.float().nan_to_num(7.0), t.to(torch.bfloat16).float().nan_to_num(7.0))


def test_neighbours_do_not_change_an_element():
    # the same element beside ordinary ones, beside a v of zero, and in a
    # tensor's last, incomplete block
    out = []
    for kind in range(3):
        n = 256 if kind < 2 else 200
        g = np.random.default_rng(5).normal(0, 1, 256).astype(np.float32)[:n]
        if kind == 1:
            g[1] = 0
        z = lambda k, dt: torch.zeros(k, dtype=dt, device="cuda")  # noqa: E731
        p = z(n, torch.float32)
        plan = L.w4a16_adamw_plan([p], [torch.from_numpy(g).cuda()], [z(n, torch.int8)], [z(n, torch.uint8)],
                                  m_scales=[z(1, torch.float32)], v_scales=[z(1, torch.float32)])
        step(plan, seed=1)
        out.append(p.cpu().numpy()[2:200])
    assert np.array_equal(out[0].view(np.uint32), out[1].view(np.uint32))
    assert np.array_equal(out[0].view(np.uint32), out[2].view(np.uint32))
