"""Sizes that w4a16_lora_linear's kernels do not take are refused before anything
runs: on a host without a GPU the refusal itself comes back, not the missing
device (CPU only; fake pointers, never dereferenced)."""
import pytest

import int4_weight_only_linear_amd as L
from test_adapters_host import P, forward

FAR = 1 << 44  # outputs, past every input's extent


@pytest.mark.parametrize("kw,msg", [
    (dict(M=1 << 22, K=512), "M*K*2 must be below 4 GiB"),
    (dict(M=4, N=1 << 21, K=1 << 14), "N*K/2 must be below 4 GiB"),
    (dict(M=17, N=1 << 21, K=1 << 14), "N*K/2 and"),
])
@pytest.mark.parametrize("u", [None, FAR + (1 << 43)])
def test_sizes(kw, msg, u):
    assert forward(y=FAR, u=u, n=1 << 62, **kw) == 2, L.w4a16_last_error()
    assert msg in L.w4a16_last_error()


def test_forced_decode_kernel(monkeypatch):
    monkeypatch.setenv("W4A16_FORCE_PATH", "gemv")
    L.w4a16_reload_tuning()
    try:
        assert forward(M=17, u=20 * P, n=1 << 62) == 2
        assert "M <= 16" in L.w4a16_last_error()
    finally:
        monkeypatch.delenv("W4A16_FORCE_PATH")
        L.w4a16_reload_tuning()
