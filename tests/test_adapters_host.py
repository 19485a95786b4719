"""The adapters' and AdamW entry points on the host: argument checks before any
device is touched, workspace sizes, and the layout of the AdamW table.  Fake
pointers, never dereferenced."""
import ctypes

import numpy as np
import pytest

import int4_weight_only_linear_amd as L
from int4_weight_only_linear_amd import _binding as B

P = 1 << 28  # apart by more than any extent below


def forward(**kw):
    a = dict(x=P, wq=2 * P, s=3 * P, zp=None, bias=None, la=4 * P, lb=5 * P, ids=6 * P, alpha=None, y=7 * P, u=None,
             M=4, N=64, K=256, g=128, S=3, R=16, dt=1, ws=8 * P, n=1 << 24)
    assert set(kw) <= set(a)
    a.update(kw)
    return B.lib.w4a16_lora_linear(*a.values(), None)


def backward(**kw):
    a = dict(dy=P, x=2 * P, u=3 * P, wq=4 * P, s=5 * P, zp=None, la=6 * P, lb=7 * P, ids=8 * P, alpha=None, dx=9 * P,
             dla=10 * P, dlb=11 * P, M=4, N=64, K=256, g=128, S=3, R=16, dt=1, ws=12 * P, n=1 << 24)
    assert set(kw) <= set(a)
    a.update(kw)
    return B.lib.w4a16_lora_backward(*a.values(), None)


SHARED = [
    (dict(S=0), 1, "at least one adapter"),
    (dict(S=1 << 31), 1, "at least one adapter"),
    (dict(R=0), 1, "multiple of 8"),
    (dict(R=12), 1, "multiple of 8"),
    (dict(R=-8), 1, "multiple of 8"),
    (dict(R=136), 2, "128"),
    (dict(S=(1 << 31) - 1, R=128, K=1 << 24), 1, "too large"),
    (dict(la=None), 1, "NULL"),
    (dict(lb=None), 1, "NULL"),
    (dict(ids=None), 1, "NULL"),
    (dict(la=20 * P + 8), 3, "16-byte"),
    (dict(lb=20 * P + 2), 3, "16-byte"),
    (dict(ids=20 * P + 2), 3, "4-byte"),
    (dict(alpha=20 * P + 1), 3, "4-byte"),
    (dict(g=48), 2, "group size"),
    (dict(dt=2), 1, "dtype"),
    (dict(M=-1), 1, "M must be"),
    (dict(N=0), 1, "N must be"),
    (dict(x=None), 1, "NULL"),
    (dict(wq=None), 1, "NULL"),
    (dict(x=20 * P + 8), 3, "x must be 16-byte"),
]


@pytest.mark.parametrize("kw,status,msg", SHARED + [
    (dict(y=None), 1, "NULL"),
    (dict(u=20 * P + 4), 3, "u must be 16-byte"),
    (dict(y=4 * P + 256), 1, "overlap"),   # in la
    (dict(y=6 * P), 1, "overlap"),         # on ids
    (dict(u=5 * P), 1, "overlap"),         # on lb
    (dict(u=7 * P + 64), 1, "overlap"),    # in y
    (dict(u=P), 1, "overlap"),             # on x
    (dict(alpha=20 * P, y=20 * P), 1, "overlap"),
])
def test_forward_refuses(kw, status, msg):
    assert forward(**kw) == status, L.w4a16_last_error()
    assert msg in L.w4a16_last_error()


@pytest.mark.parametrize("kw,status,msg", SHARED + [
    (dict(dy=None), 1, "NULL"),
    (dict(u=None), 1, "u must not"),
    (dict(dla=None), 1, "dla and dlb"),
    (dict(dlb=None), 1, "dla and dlb"),
    (dict(dx=20 * P + 8), 3, "16-byte"),
    (dict(dla=20 * P + 8), 3, "16-byte"),
    (dict(dy=20 * P + 2), 3, "16-byte"),
    (dict(S=65536), 2, "65535"),
    (dict(M=1 << 30), 2, "too many tokens"),
    (dict(N=1 << 21, K=1 << 14), 2, "4 GiB"),
    (dict(dx=2 * P), 1, "overlap"),             # on x
    (dict(dx=P + 16), 1, "overlap"),            # in dy
    (dict(dla=6 * P), 1, "overlap"),            # on la
    (dict(dlb=10 * P + 64), 1, "overlap"),      # in dla
    (dict(dla=3 * P), 1, "overlap"),            # on u
])
def test_backward_refuses(kw, status, msg):
    assert backward(**kw) == status, L.w4a16_last_error()
    assert msg in L.w4a16_last_error()


def test_no_tokens_need_no_pointers():
    assert forward(M=0, x=None, wq=None, s=None, la=None, lb=None, ids=None, y=None, ws=None, n=0) == 0


@pytest.mark.parametrize("M,N,K,g,zp", [(1, 64, 256, 128, False), (16, 40, 96, 32, True), (67, 4864, 896, 64, True),
                                        (1921, 264, 1216, 32, False)])
def test_workspace_sizes(M, N, K, g, zp):
    for dt in (0, 1):
        sizes = [L.w4a16_lora_workspace_size(M, N, K, g, dt, zp, R, save_u) for R in (8, 64, 128) for save_u in (True, False)]
        assert all(n > 0 and n % 256 == 0 for n in sizes)
        # u in the workspace where the caller does not keep it
        assert all(kept <= own for kept, own in zip(sizes[::2], sizes[1::2]))
        # the projection's own region first
        assert min(sizes) > L.w4a16_workspace_size(M, N, K, g, dt, zp)
        back = [L.w4a16_lora_backward_workspace_size(M, N, K, g, S, 16, dt) for S in (1, 5, 17)]
        assert all(n % 256 == 0 for n in back) and back == sorted(back)
        # room for the transposed factors at least
        assert back[2] > 2 * 17 * 16 * (K + N)


@pytest.mark.parametrize("kw", [dict(M=0), dict(N=0), dict(K=0), dict(group_size=48), dict(R=4), dict(R=136), dict(dtype=2)])
def test_workspace_sizes_of_what_is_refused(kw):
    a = dict(M=4, N=64, K=256, group_size=128, dtype=1, R=16)
    a.update(kw)
    assert L.w4a16_lora_workspace_size(has_zp=False, **a) == 0
    assert L.w4a16_lora_backward_workspace_size(S=2, **a) == 0


def test_backward_workspace_size_of_too_many_adapters():
    assert L.w4a16_lora_backward_workspace_size(4, 64, 256, 128, 65536, 16, 1) == 0
    assert L.w4a16_lora_backward_workspace_size(4, 64, 256, 128, 0, 16, 1) == 0


# ---- the AdamW table ---------------------------------------------------------

class Table:
    """Rows of fake tensors of the given sizes and the table laid out of them."""

    def __init__(self, sizes, bits=32, param=2, grad=2, copy=1, **change):
        self.rows = (B.AdamwTensor * len(sizes))()
        for i, n in enumerate(sizes):
            at = [(1 + 8 * i + j) * P for j in range(7)]
            if bits == 32:
                at[4] = at[5] = None
            self.rows[i] = B.AdamwTensor(*at, n)
        for (i, field), value in change.pop("set", {}).items():
            setattr(self.rows[i], field, value)
        self.size = int(B.lib.w4a16_adamw_table_size(self.rows, len(sizes)))
        self.host = np.zeros(max(1, (self.size + 7) // 8), dtype=np.int64)
        self.info = B.AdamwPlanInfo()
        self.status = B.lib.w4a16_adamw_table(self.rows, len(sizes), bits, param, grad, copy, self.host.ctypes.data,
                                              self.size, ctypes.byref(self.info))


@pytest.mark.parametrize("sizes", [[1], [0, 5, 0], [256, 257, 255], [4096 * 25, 8, 0, 1000], [256 * 9000, 3, 256 * 4 * 4 + 1]])
@pytest.mark.parametrize("bits", [8, 32])
def test_table_covers_every_block_once(sizes, bits):
    t = Table(sizes, bits)
    assert t.status == 0
    blocks = [(n + 255) // 256 for n in sizes]
    assert t.info.tensors == len(sizes) and t.info.blocks == sum(blocks) and t.info.state_bits == bits
    # the chunks: (tensor, first block), up to four waves' blocks each
    per = 4 * (1 if sum(blocks) < 8192 else 4)
    chunks = t.host.view(np.int32)[-2 * t.info.chunks:].reshape(-1, 2)
    assert t.size == t.host.nbytes
    assert chunks.tolist() == [[i, b] for i, n in enumerate(blocks) for b in range(0, n, per)]


@pytest.mark.parametrize("change,status,msg", [
    ({(1, "param"): None}, 1, "NULL"),
    ({(0, "m"): None}, 1, "NULL"),
    ({(1, "n"): -1}, 1, "out of range"),
    ({(1, "n"): 1 << 39}, 1, "out of range"),
    ({(0, "param"): 50 * P + 2}, 3, "not aligned"),
    ({(0, "grad"): 50 * P + 1}, 3, "not aligned"),
    ({(0, "copy"): 50 * P + 1}, 3, "not aligned"),
    ({(0, "m"): 50 * P, (0, "v"): 50 * P + 40}, 1, "overlap"),
    ({(0, "param"): 50 * P, (1, "param"): 50 * P}, 1, "overlap"),      # one tensor twice
    ({(0, "copy"): 50 * P, (1, "v"): 50 * P + 100}, 1, "overlap"),
    ({(0, "grad"): 50 * P, (1, "param"): 50 * P + 100}, 1, "overlap"),  # a gradient read beside a write
    ({(1, "grad"): 50 * P, (1, "param"): 50 * P}, 1, "overlap"),
])
def test_table_refuses(change, status, msg):
    t = Table([300, 300], set=change)
    assert t.status == status and msg in L.w4a16_last_error()
    assert not t.host.any()


def test_table_takes_shared_gradients_and_neighbours():
    # a gradient of two tensors; buffers that touch without overlapping
    assert Table([300, 300], set={(0, "grad"): 50 * P, (1, "grad"): 50 * P}).status == 0
    assert Table([300, 300], set={(0, "m"): 50 * P, (0, "v"): 50 * P + 1200, (1, "param"): 50 * P + 2400}).status == 0


@pytest.mark.parametrize("bits,param,grad,copy", [(16, 2, 2, 1), (32, 3, 2, 1), (32, 2, -1, 1), (32, 2, 2, 2)])
def test_table_refuses_types(bits, param, grad, copy):
    assert Table([8], bits, param, grad, copy).status == 1


def test_step_refuses_before_a_device_is_needed():
    t = Table([300])
    good = dict(lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, wd=0.0, step=1, scale=1.0, seed=0)
    def step(table=8 * P, info=t.info, **kw):
        return B.lib.w4a16_adamw_step(table, ctypes.byref(info), *{**good, **kw}.values(), None)
    inf, nan = float("inf"), float("nan")
    for bad in (dict(b1=1.0), dict(b1=-0.1), dict(b2=nan), dict(eps=-1e-9), dict(eps=inf), dict(lr=nan), dict(wd=inf),
                dict(step=0), dict(scale=nan), dict(scale=inf), dict(table=None), dict(info=B.AdamwPlanInfo())):
        assert step(**bad) == 1, bad
    assert step(table=8 * P + 4) == 3
    # no elements: nothing to do
    empty = Table([0])
    assert step(info=empty.info) == 0
    assert B.lib.w4a16_adamw_moments(8 * P, ctypes.byref(t.info), P, 2 * P, None) == 2
    eight = Table([300], 8)
    assert B.lib.w4a16_adamw_moments(8 * P, ctypes.byref(eight.info), None, P, None) == 1
    assert B.lib.w4a16_adamw_moments(8 * P, ctypes.byref(eight.info), P + 4, 2 * P, None) == 3
    assert B.lib.w4a16_adamw_moments(8 * P, ctypes.byref(eight.info), P, P + 16, None) == 1
