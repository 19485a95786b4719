"""The AdamW step over many tensors, through the C ABI, against float64.

Tolerances, fixed before the first run, from the step's operations, each
rounded once to 24 bits (E = 2^-24): m is three operations on two products,
within 4 E of |b1 m| + |(1-b1) g|; v, of positive terms, within 6 E of itself;
the update's factors (a square root, a product, a sum, a quotient, a product
and constants rounded to fp32) add 12 E of the update to what m's error gives,
and p's own three operations 4 E of |p|.  Codes: the exact code's fp32 value
is within 255 * 16 E of it, so a code is floor(exact + dither) unless that
falls within 1e-3 of a whole number, and then it is one of the two there."""
import ctypes

import numpy as np
import pytest

from oracle import adapters_ref as A
from gpu_util import note

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import int4_weight_only_linear_amd as L  # noqa: E402
from int4_weight_only_linear_amd import _binding as B  # noqa: E402

E = 2.0 ** -24
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.05, step=7, grad_scale=0.25)
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(autouse=True)
def _need_gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    note(f"[gpu] {request.node.nodeid}")


def step(plan, seed=0, **kw):
    h = {**HYPER, **kw}
    L.w4a16_adamw_step(plan, lr=h["lr"], betas=(h["beta1"], h["beta2"]), eps=h["eps"], weight_decay=h["weight_decay"],
                       step=h["step"], grad_scale=h["grad_scale"], seed=seed)
    torch.cuda.synchronize()


def draw(sizes, param, grad, seed, scale=1e-2):
    rng = np.random.default_rng(seed)
    t = lambda a, dt: torch.from_numpy(a.astype(np.float32)).cuda().to(dt)  # noqa: E731
    P = [t(rng.normal(0, 0.5, n), DTYPES[param]) for n in sizes]
    G = [t(rng.normal(0, scale, n) * np.exp(rng.normal(0, 1, n)), DTYPES[grad]) for n in sizes]
    return rng, P, G


def f64(t):
    return t.double().cpu().numpy()


def check_p(p_new, p0, m_ref, m_err, v_ref, param, h):
    upd = h["lr"] / (1 - h["beta1"] ** h["step"]) / (np.sqrt(v_ref / (1 - h["beta2"] ** h["step"])) + h["eps"])
    want = p0 * (1 - h["lr"] * h["weight_decay"]) - upd * m_ref
    bound = upd * m_err + 12 * E * np.abs(upd * m_ref) + 4 * E * np.abs(p0)
    # one rounding of an fp32 value within the bound: between the roundings of its ends
    ends = [torch.from_numpy(w).float().to(DTYPES[param]).double().numpy() for w in (want - bound, want + bound)]
    assert np.all(p_new >= ends[0]) and np.all(p_new <= ends[1])


SIZES = [1, 255, 256, 257, 4096, 4097, 16 * 640, 70001, 3, 0, 8191]


@pytest.mark.parametrize("param,grad,copy", [("f32", "f32", None), ("f32", "bf16", "bf16"), ("f32", "f16", "f16"),
                                             ("bf16", "bf16", None), ("f16", "f16", None), ("f32", "bf16", "f16"),
                                             ("bf16", "f32", None), ("f16", "bf16", None)])
def test_moments_in_32_bits(param, grad, copy):
    rng, P, G = draw(SIZES, param, grad, (param, grad) == ("f32", "f32"))
    Ms = [torch.from_numpy(rng.normal(0, 3e-3, n).astype(np.float32)).cuda() for n in SIZES]
    Vs = [torch.from_numpy(np.square(rng.normal(0, 3e-3, n)).astype(np.float32)).cuda() for n in SIZES]
    C = None if copy is None else [torch.full((n,), 9.0, dtype=DTYPES[copy], device="cuda") for n in SIZES]
    before = [[f64(t) for t in ts] for ts in (P, G, Ms, Vs)]
    step(L.w4a16_adamw_plan(P, G, Ms, Vs, copies=C))
    h = HYPER
    for i, n in enumerate(SIZES):
        p0, g0, m0, v0 = (b[i] for b in before)
        _, m, v = A.adamw_ref(p0, g0, m0, v0, **h)
        m_err = 4 * E * (np.abs(h["beta1"] * m0) + np.abs((1 - h["beta1"]) * g0 * h["grad_scale"]))
        assert np.all(np.abs(f64(Ms[i]) - m) <= m_err)
        assert np.all(np.abs(f64(Vs[i]) - v) <= 6 * E * v)
        check_p(f64(P[i]), p0, m, m_err, v, param, h)
        assert np.array_equal(f64(G[i]), g0)
        if C:
            assert torch.equal(C[i], P[i].to(DTYPES[copy]))


@pytest.mark.parametrize("param,grad,shift", [("f32", "bf16", 0), ("bf16", "bf16", 0), ("f16", "f32", 0), ("f32", "f32", 1)])
def test_moments_in_8_bits(param, grad, shift):
    # shift: every tensor one element off its alignment (element-wise accesses)
    rng, P, G = draw(SIZES, param, grad, 5)
    off = lambda t: torch.cat([t.new_zeros(1), t])[1:] if shift else t  # noqa: E731
    P, G = [off(t) for t in P], [off(t) for t in G]
    blocks = [(n + 255) // 256 for n in SIZES]
    CM = [off(torch.from_numpy(rng.integers(-127, 128, n).astype(np.int8)).cuda()) for n in SIZES]
    CV = [off(torch.from_numpy(rng.integers(1, 256, n).astype(np.uint8)).cuda()) for n in SIZES]
    MS = [torch.from_numpy(rng.uniform(1e-4, 1e-2, b).astype(np.float32)).cuda() for b in blocks]
    RS = [torch.from_numpy(rng.uniform(1e-4, 1e-2, b).astype(np.float32)).cuda() for b in blocks]
    before = [[f64(t) for t in ts] for ts in (P, G, CM, CV, MS, RS)]
    plan = L.w4a16_adamw_plan(P, G, CM, CV, m_scales=MS, v_scales=RS)
    assert plan.blocks == sum(blocks)
    step(plan, seed=12345)
    mo, vo = L.w4a16_adamw_moments(plan)
    torch.cuda.synchronize()
    h, first = HYPER, 0
    for i, n in enumerate(SIZES):
        p0, g0, cm0, cv0, ms0, rs0 = (b[i] for b in before)
        m0, v0 = A.adamw_decode(cm0, cv0, ms0, rs0)
        _, m, v = A.adamw_ref(p0, g0, m0, v0, **h)
        # the decoding's three operations on top of the step's
        m_err = 8 * E * (np.abs(h["beta1"] * m0) + np.abs((1 - h["beta1"]) * g0 * h["grad_scale"]))
        check_p(f64(P[i]), p0, m, m_err, v, param, h)
        ms, rs, r = f64(MS[i]), f64(RS[i]), np.sqrt(v)
        dm, dv = A.adamw_dither(first * 256 + np.arange(n), 12345)
        for b in range(blocks[i]):
            s = slice(256 * b, min(n, 256 * b + 256))
            assert abs(ms[b] - np.abs(m[s]).max()) <= m_err[s].max()
            assert abs(rs[b] - r[s].max()) <= 8 * E * rs[b]
            for code, t, d, lo in ((np.abs(f64(CM[i])[s]), 127 * np.sqrt(np.abs(m[s]) / ms[b]), dm[s], 0),
                                   (f64(CV[i])[s], 255 * np.sqrt(r[s] / rs[b]), dv[s], 1)):
                # (an m that nearly cancels has its error of b1 m + (1 - b1) g in its share)
                slack = 1e-3 + (127 * np.sqrt(m_err[s] / ms[b]) if lo == 0 else 0)
                top = 255 if lo else 127
                assert np.all(code <= np.clip(np.floor(t + d + slack), lo, top))
                assert np.all(code >= np.clip(np.floor(t + d - slack), lo, top))
            sign_clear = np.abs(m[s]) > m_err[s]
            got = f64(CM[i])[s]
            assert np.all((got == 0) | (np.sign(got) == np.sign(m[s])) | ~sign_clear)
        # the decoding's sequence of fp32 operations, bit for bit
        a = first * 256
        spread = lambda t: np.repeat(t.cpu().numpy(), 256)[:n]  # noqa: E731
        c = CM[i].cpu().numpy().astype(np.float32) * np.float32(1 / 127)
        assert np.array_equal(mo[a:a + n].cpu().numpy(), c * np.abs(c) * spread(MS[i]))
        c = CV[i].cpu().numpy().astype(np.float32) * np.float32(1 / 255)
        rd = c * c * spread(RS[i])
        assert np.array_equal(vo[a:a + n].cpu().numpy(), rd * rd)
        assert torch.count_nonzero(mo[a + n:(first + blocks[i]) * 256]) == 0
        assert torch.count_nonzero(vo[a + n:(first + blocks[i]) * 256]) == 0
        first += blocks[i]


@pytest.mark.parametrize("scale", [1.0, 1e-3, 1e-18, 0.0])
def test_codes_are_the_plain_sequence_of_fp32_operations(scale):
    # every code and scale, bit for bit, of the step written as single fp32
    # operations (numpy rounds each once); 1e-18: moments near the end of fp32
    n = 256 * 200
    rng = np.random.default_rng(11)
    g = (rng.normal(0, 1, n) * np.exp(rng.normal(0, 2, n)) * scale).astype(np.float32)
    g[:256 * 20:3] = 0
    cm, cv = rng.integers(-127, 128, n).astype(np.int8), rng.integers(0, 256, n).astype(np.uint8)
    ms, rs = (rng.uniform(0.1, 1, n // 256).astype(np.float32) * np.float32(scale) for _ in range(2))
    cm[:256 * 10], cv[:256 * 10] = 0, 0
    dev = lambda a: torch.from_numpy(a.copy()).cuda()  # noqa: E731
    t = [dev(a) for a in (cm, cv, ms, rs)]
    step(L.w4a16_adamw_plan([torch.zeros(n, device="cuda")], [dev(g)], [t[0]], [t[1]], m_scales=[t[2]], v_scales=[t[3]]),
         seed=77)
    f, h = np.float32, HYPER
    spread = lambda a: np.repeat(a, 256)  # noqa: E731
    with np.errstate(all="ignore"):
        c = cm.astype(f) * f(1 / 127)
        m = (c * np.abs(c)) * spread(ms)
        c = cv.astype(f) * f(1 / 255)
        r = (c * c) * spread(rs)
        v = r * r
        gs = g * f(h["grad_scale"])
        m = m * f(h["beta1"]) + gs * f(1 - h["beta1"])
        v = v * f(h["beta2"]) + (gs * gs) * f(1 - h["beta2"])
        r = np.sqrt(v)
        m2, r2 = np.abs(m).reshape(-1, 256).max(1), r.reshape(-1, 256).max(1)
        inv = lambda a: spread(np.where(a > f(2.0 ** -100), f(1) / a, f(0)).astype(f))  # noqa: E731
        dm, dv = A.adamw_dither(np.arange(n), 77)
        qm = np.minimum(np.floor(np.sqrt(np.abs(m) * inv(m2)) * f(127) + dm.astype(f)), f(127))
        qv = np.floor(np.sqrt(r * inv(r2)) * f(255) + dv.astype(f))
        qv = np.minimum(np.where(r > 0, np.maximum(qv, f(1)), qv), f(255))
    assert np.array_equal(t[2].cpu().numpy(), m2) and np.array_equal(t[3].cpu().numpy(), r2)
    assert np.array_equal(t[0].cpu().numpy(), np.where(m < 0, -qm, qm).astype(np.int8))
    assert np.array_equal(t[1].cpu().numpy(), qv.astype(np.uint8))


def zeros8(n):
    b = (n + 255) // 256
    z = lambda k, dt: torch.zeros(k, dtype=dt, device="cuda")  # noqa: E731
    return z(n, torch.int8), z(n, torch.uint8), z(b, torch.float32), z(b, torch.float32)


def test_from_nothing_and_zero_gradients():
    # the first step from all-zero codes and scales; a zero gradient leaves them zero
    n = 1000
    p = torch.ones(n, device="cuda")
    g = torch.zeros(n, device="cuda")
    g[300:] = torch.linspace(-1, 1, 700, device="cuda")
    m, v, ms, rs = zeros8(n)
    plan = L.w4a16_adamw_plan([p], [g], [m], [v], m_scales=[ms], v_scales=[rs])
    step(plan, step=1, weight_decay=0.0, grad_scale=1.0)
    assert torch.count_nonzero(m[:300]) == 0 and torch.count_nonzero(v[:300]) == 0
    assert ms[0] == 0 and rs[0] == 0 and (p[:300] == 1).all()
    # with bias correction the first update is lr * sign(g)
    moved = g.abs() > 1e-3
    assert torch.allclose((1 - p)[moved], 3e-3 * torch.sign(g[moved]), rtol=1e-4)
    assert (v[300:][g[300:] != 0] >= 1).all()


def test_codes_are_unbiased_and_follow_slow_moments():
    # constant gradients: over many steps the mean of the decoded moments
    # follows the 32-bit ones, although one step moves v by a tenth of a code
    n = 4096
    rng = np.random.default_rng(3)
    g = torch.from_numpy((rng.normal(0, 1, n) * np.exp(rng.normal(0, 0.5, n))).astype(np.float32)).cuda()
    m8, v8, ms, rs = zeros8(n)
    a = L.w4a16_adamw_plan([torch.zeros(n, device="cuda")], [g], [m8], [v8], m_scales=[ms], v_scales=[rs])
    m32, v32 = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    b = L.w4a16_adamw_plan([torch.zeros(n, device="cuda")], [g], [m32], [v32])
    for t in range(1, 301):
        if t == 200:
            g.mul_(0.1)
        for plan in (a, b):
            L.w4a16_adamw_step(plan, lr=1e-3, betas=(0.9, 0.99), step=t, seed=t)
    mo, vo = L.w4a16_adamw_moments(a)
    assert abs(float((torch.sqrt(vo) / torch.sqrt(v32)).mean()) - 1) < 0.02
    assert abs(float((mo / m32).mean()) - 1) < 0.02


def test_same_seed_same_codes_and_another_seed_others():
    n = 10000
    g = torch.randn(n, generator=torch.Generator().manual_seed(1)).cuda()
    out = []
    for seed in (1, 1, 2):
        m, v, ms, rs = zeros8(n)
        plan = L.w4a16_adamw_plan([torch.zeros(n, device="cuda")], [g], [m], [v], m_scales=[ms], v_scales=[rs])
        step(plan, seed=seed)
        out.append((m, v))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    assert not torch.equal(out[0][0], out[2][0]) and not torch.equal(out[0][1], out[2][1])


def test_nan_gradient_stays_in_its_block():
    n = 1024
    g = torch.ones(n, device="cuda")
    g[300] = float("nan")
    p = torch.zeros(n, device="cuda")
    m, v, ms, rs = zeros8(n)
    plan = L.w4a16_adamw_plan([p], [g], [m], [v], m_scales=[ms], v_scales=[rs])
    step(plan)
    assert torch.isnan(p).nonzero().flatten().tolist() == [300]
    assert torch.isnan(ms).nonzero().flatten().tolist() == [1] and torch.isnan(rs).nonzero().flatten().tolist() == [1]


def test_guard_bands_and_graph_replays():
    # neighbours of every buffer keep their values; replays equal eager steps
    sizes = [300, 5, 4096]
    full = [torch.full((n + 64,), 7.0, device="cuda") for n in sizes]
    P = [f[32:32 + n] for f, n in zip(full, sizes)]
    for p in P:
        p.zero_()
    G = [torch.randn(n, generator=torch.Generator().manual_seed(n)).cuda() for n in sizes]
    S = [zeros8(n) for n in sizes]
    plan = L.w4a16_adamw_plan(P, G, [s[0] for s in S], [s[1] for s in S], m_scales=[s[2] for s in S], v_scales=[s[3] for s in S])
    ref_p = [p.clone() for p in P]
    ref_s = [[t.clone() for t in s] for s in S]
    ref = L.w4a16_adamw_plan(ref_p, G, [s[0] for s in ref_s], [s[1] for s in ref_s], m_scales=[s[2] for s in ref_s],
                             v_scales=[s[3] for s in ref_s])
    st = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=st):
        L.w4a16_adamw_step(plan, lr=1e-3, step=3, seed=9)
    for _ in range(4):
        graph.replay()
        L.w4a16_adamw_step(ref, lr=1e-3, step=3, seed=9)
        torch.cuda.synchronize()
        for a, b in zip(P, ref_p):
            assert torch.equal(a, b)
        for a, b in zip(S, ref_s):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    for f, n in zip(full, sizes):
        assert (f[:32] == 7).all() and (f[32 + n:] == 7).all()


def test_refusals():
    z = lambda n, dt=torch.float32: torch.zeros(n, dtype=dt, device="cuda")  # noqa: E731
    ok = lambda **kw: L.w4a16_adamw_plan(**{**dict(params=[z(8)], grads=[z(8)], exp_avgs=[z(8)], exp_avg_sqs=[z(8)]), **kw})  # noqa: E731
    plan = ok()
    for bad in (dict(grads=[z(9)]), dict(grads=[]), dict(params=[], grads=[], exp_avgs=[], exp_avg_sqs=[]),
                dict(m_scales=[z(1)])):
        with pytest.raises(ValueError):
            ok(**bad)
    for bad in (dict(exp_avgs=[z(8, torch.int8)]), dict(params=[z(8, torch.float64)]), dict(copies=[z(8)]),
                dict(params=[z(8), z(8, torch.float16)], grads=[z(8), z(8)], exp_avgs=[z(8), z(8)], exp_avg_sqs=[z(8), z(8)])):
        with pytest.raises(TypeError):
            ok(**bad)
    shared = z(8)
    with pytest.raises(L.W4A16Error, match="overlap"):
        ok(exp_avgs=[shared], exp_avg_sqs=[shared])
    for bad in (dict(step=0), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=-1.0), dict(lr=float("nan"))):
        with pytest.raises(L.W4A16Error, match="INVALID_ARG"):
            step(plan, **bad)
    with pytest.raises(L.W4A16Error, match="UNSUPPORTED"):
        L.w4a16_adamw_moments(plan, z(256), z(256))
    rows = (B.AdamwTensor * 1)(B.AdamwTensor(None, None, None, None, None, None, None, 5))
    host, info = np.zeros(64, dtype=np.int64), B.AdamwPlanInfo()
    for args, status in (((32, 2, 2, 1, host.ctypes.data, 512), 1), ((16, 2, 2, 1, host.ctypes.data, 512), 1),
                         ((32, 7, 2, 1, host.ctypes.data, 512), 1), ((32, 2, 2, 1, host.ctypes.data, 8), 6),
                         ((32, 2, 2, 1, host.ctypes.data + 4, 256), 3)):
        assert B.lib.w4a16_adamw_table(rows, 1, *args, ctypes.byref(info)) == status
        assert not host.any()
