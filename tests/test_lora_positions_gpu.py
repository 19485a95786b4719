"""Decode with adapters, bit for bit: on inputs whose every partial sum is exact
in fp32 (small integers and powers of two), the order of the sums does not
matter and y is the formula's value rounded once, wherever a token stands in
the call and whichever wave adds its adapter's term.  A term that lands in
another token's sums, is lost, or is added before a sum is there, shows."""
import numpy as np
import pytest

import oracle as O
from synth.gen import to_act_bits
from test_lora_gpu import LoraCase, torch
from gpu_util import device_to_bits, note, torch_dtype

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    note(f"[gpu] {request.node.nodeid}")


# few tokens in every instance (1, 2, 4 and 8 rows), whole and split K, one
# wave and many; then the general kernel up to 16 tokens
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 6, 7, 8, 9, 13, 16])
@pytest.mark.parametrize("N,K,group,dt,sym", [
    (80, 4096, 128, O.BF16, False),
    (48, 28672, 128, O.F16, False),
    (51, 512, 32, O.BF16, True),
    (96, 1056, 32, O.F16, True),
    (64, 2560, 64, O.BF16, True),
])
def test_every_position(M, N, K, group, dt, sym):
    S, R = 5, 40
    case = LoraCase(M, N, K, group, dt, sym, False, S, R, "mixed")
    rng = np.random.default_rng(M * 1000 + K)
    # |x| <= 2, |q - z| <= 15: sums of x . W below 2 * 15 * 28672 < 2^20 (times
    # the scale); the kernels' own sums of x (1024 + q) over a group below 2^19.
    # |A| <= 1 on one k in 16: |u| <= 2 * 28672 / 16 + slack < 2^13, |B| <= 2:
    # the term below 2^13 * 2 * 40 * 2 < 2^21.  All are multiples of the scale 2^-6.
    x = rng.integers(-2, 3, (M, K)).astype(np.float64)
    la = np.where(rng.integers(0, 16, (S, R, K)) == 0, rng.integers(-1, 2, (S, R, K)), 0).astype(np.float64)
    lb = rng.integers(-2, 3, (S, N, R)).astype(np.float64) * 2.0 ** -6
    alpha = np.array([1, 2, 0.5, 1, 2])
    ids = ((np.arange(M) * 2 + M) % (S + 1) - 1).astype(np.int32)
    up = lambda v, t: t.copy_(torch.from_numpy(v).to(torch_dtype(dt)))  # noqa: E731
    up(x, case.d.x), up(la, case.t_la), up(lb, case.t_lb)
    case.d.s.fill_(2.0 ** -6)
    case.t_ids.copy_(torch.from_numpy(ids))
    case.t_alpha.copy_(torch.from_numpy(alpha))
    q = case.c.q.astype(np.float64)
    z = 8.0 if sym else np.repeat(case.c.zp.astype(np.float64), group, axis=1)
    want = x @ ((q - z) * 2.0 ** -6).T
    for m, a in enumerate(ids.tolist()):
        if a >= 0:
            want[m] += alpha[a] * (lb[a] @ (la[a] @ x[m]))
    assert np.abs(want).max() < 2 ** 15 and np.all(want * 128 == np.round(want * 128))
    want = to_act_bits(want.astype(np.float32), dt).reshape(M, N)
    for keep in (False, True):
        y = case.run(save_u=keep)
        got = device_to_bits(y[0] if keep else y)
        value = lambda b: O.act_bits_to_f64(b, dt)  # noqa: E731
        assert np.array_equal(value(got), value(want)), (keep, np.argwhere(value(got) != value(want))[:8].tolist())
