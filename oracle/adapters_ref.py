"""Low-rank adapters beside the W4A16 projection, their gradients and the
AdamW step, in float64 from the exact inputs (the formulas of include/w4a16.h)."""
from __future__ import annotations

import numpy as np

from .w4a16_ref import act_bits_to_f64, dequant_f32, linear_ref


def _stack(bits, shape, dtype):
    return act_bits_to_f64(np.asarray(bits).reshape(shape), dtype)


def lora_linear_ref(x_bits, wq, scale_bits, zpk, bias_bits, la_bits, lb_bits, ids, alpha, M: int, N: int, K: int,
                    group: int, S: int, R: int, dtype: int):
    """(y [M, N], u [M, R]): one token at a time."""
    y = linear_ref(x_bits, wq, scale_bits, zpk, bias_bits, M, N, K, group, dtype)
    x = act_bits_to_f64(np.asarray(x_bits).reshape(M, K), dtype)
    la, lb = _stack(la_bits, (S, R, K), dtype), _stack(lb_bits, (S, N, R), dtype)
    u = np.zeros((M, R))
    for m, a in enumerate(np.asarray(ids).tolist()):
        if 0 <= a < S:
            u[m] = la[a] @ x[m]
            y[m] += (1.0 if alpha is None else float(alpha[a])) * (lb[a] @ u[m])
    return y, u


def lora_backward_ref(dy_bits, x_bits, u, wq, scale_bits, zpk, la_bits, lb_bits, ids, alpha, M: int, N: int, K: int,
                      group: int, S: int, R: int, dtype: int):
    """(dx [M, K], dla [S, R, K], dlb [S, N, R])."""
    dy = act_bits_to_f64(np.asarray(dy_bits).reshape(M, N), dtype)
    x = act_bits_to_f64(np.asarray(x_bits).reshape(M, K), dtype)
    la, lb = _stack(la_bits, (S, R, K), dtype), _stack(lb_bits, (S, N, R), dtype)
    dx = dy @ dequant_f32(wq, scale_bits, zpk, N, K, group, dtype).astype(np.float64)
    dla, dlb = np.zeros((S, R, K)), np.zeros((S, N, R))
    for m, a in enumerate(np.asarray(ids).tolist()):
        if 0 <= a < S:
            k = 1.0 if alpha is None else float(alpha[a])
            g = k * (dy[m] @ lb[a])
            dx[m] += g @ la[a]
            dla[a] += np.outer(g, x[m])
            dlb[a] += np.outer(dy[m], k * np.asarray(u[m], dtype=np.float64))
    return dx, dla, dlb


def adamw_ref(p, g, m, v, *, lr, beta1, beta2, eps, weight_decay, step, grad_scale):
    """(p, m, v) after one step on float64 arrays."""
    g = g * grad_scale
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    mh, vh = m / (1 - beta1 ** step), v / (1 - beta2 ** step)
    return p - lr * weight_decay * p - lr * mh / (np.sqrt(vh) + eps), m, v


def adamw_dither(count, seed: int):
    """The (m, v) dithers of the elements at places `count` (block * 256 + place in the block)."""
    x = (np.asarray(count, dtype=np.uint64) + np.uint64(seed * 0x9E3779B9 % (1 << 32))) % np.uint64(1 << 32)
    x ^= x >> np.uint64(16)
    x = x * np.uint64(0x7FEB352D) % np.uint64(1 << 32)
    x ^= x >> np.uint64(15)
    x = x * np.uint64(0x846CA68B) % np.uint64(1 << 32)
    x ^= x >> np.uint64(16)
    return (x & np.uint64(0xFFFF)).astype(np.float64) / 65536, (x >> np.uint64(16)).astype(np.float64) / 65536


def adamw_decode(cm, cv, ms, rs):
    """The float64 moments that codes [n] and block scales stand for."""
    n = len(cm)
    ms, rs = (np.repeat(np.asarray(t, dtype=np.float64), 256)[:n] for t in (ms, rs))
    c = np.asarray(cm, dtype=np.float64) / 127
    return np.sign(c) * c * c * ms, ((np.asarray(cv, dtype=np.float64) / 255) ** 2 * rs) ** 2
