"""The oracle of routing and 8-bit products, checked on its own: against
torch's conversions, brute force and differences."""
import numpy as np
import pytest

from oracle import experts_ref as X

torch = pytest.importorskip("torch")


def test_codes_are_those_of_the_type():
    table = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(X.e4m3_values(), table, equal_nan=True)
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.normal(0, 1, 20000) * 2.0 ** rng.integers(-12, 8, 20000), table[np.isfinite(table)],
                        (table[:125] + table[1:126]) / 2, [0.0, -0.0, 448.0, -448.0]])
    v = np.clip(v, -448, 448).astype(np.float32)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(X.to_e4m3(v.astype(np.float64)), want)


def test_scale_is_the_smallest_power_of_two():
    x = np.zeros((6, 256))
    x[0, 3], x[1, 3], x[2, 3], x[3, 3], x[4, 3], x[5, 200] = 448, 448.5, 224, 224.1, 2.0 ** -140, np.inf
    _, scales = X.fp8_quantize_ref(x)
    assert scales[:, 0].tolist() == [127, 128, 126, 127, 1, 127] and scales.shape == (6, 4)
    assert (scales[:, 1:] == 127).all()


@pytest.mark.parametrize("groups,kept,top", [(1, 1, 1), (4, 2, 1), (4, 3, 2)])
def test_route_against_brute_force(groups, kept, top):
    rng = np.random.default_rng(1)
    l, b = rng.normal(size=(20, 16)), rng.normal(size=16) * 0.1
    w, ids = X.route_ref(l, 3, b, score="sigmoid", groups=groups, topk_groups=kept, group_top=top, renormalize=True, scale=2.0)
    s = 1 / (1 + np.exp(-l))
    for m in range(20):
        key = s[m] + b
        gk = np.sort(key.reshape(groups, -1), 1)[:, -top:].sum(1)
        alive = np.repeat(gk >= np.sort(gk)[-kept], 16 // groups)
        want = [e for e in np.argsort(-key) if alive[e]][:3]
        assert ids[m].tolist() == want
        assert np.allclose(w[m], 2 * s[m][want] / s[m][want].sum())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_gradient_against_differences(score, renormalize):
    rng = np.random.default_rng(2)
    l, dw = rng.normal(size=(4, 10)), rng.normal(size=(4, 3))
    ids = np.array([[1, 2, 3], [9, 0, 4], [5, -1, 2], [7, 7, 1]])  # one missing, one twice
    kw = dict(score=score, renormalize=renormalize, scale=1.5)
    got, bound = X.route_backward_ref(dw, l, ids, **kw)
    h = 1e-6
    for e in range(10):
        up, down = l.copy(), l.copy()
        up[:, e] += h
        down[:, e] -= h
        diff = ((X.route_weights_ref(up, ids, **kw) - X.route_weights_ref(down, ids, **kw)) * dw).sum(1) / (2 * h)
        assert np.allclose(got[:, e], diff, atol=1e-8)
    assert (np.abs(got) <= bound * (1 + 1e-12)).all()


def test_product_is_the_sum_over_blocks():
    rng = np.random.default_rng(3)
    x = rng.normal(size=(3, 300))
    codes, scales = X.fp8_quantize_ref(x)
    w = X.to_e4m3(np.clip(rng.normal(0, 100, (130, 300)), -448, 448))
    ws = rng.uniform(0.5, 2, (2, 3))
    y, slack = X.fp8_linear_ref(codes, scales, w, ws, 300, False)
    t = X.e4m3_values()
    want = np.zeros((3, 130))
    for b in range(3):
        k = slice(128 * b, min(300, 128 * (b + 1)))
        part = t[codes[:, k]] @ t[w[:, k]].T * 2.0 ** (scales[:, b, None] - 127.0)
        want += part * np.repeat(ws[:, b], 128)[:130]
    assert np.allclose(y, want, rtol=1e-12) and (slack > 0).all()
    y2, slack2 = X.fp8_linear_ref(codes, scales, np.ascontiguousarray(w.T), ws.T, 300, True)
    # (the library adds the 300 products in another order: 300 * 2^-53 of their magnitudes, here below 1e9)
    assert np.abs(y - y2).max() < 300 * 2.0 ** -53 * 1e9 and np.allclose(slack, slack2, rtol=1e-12)
