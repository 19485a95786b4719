"""An N whose 256 rows of dy pass 32-bit byte offsets in the input gradient is
refused before a device is needed (CPU only; fake pointers, never
dereferenced)."""
import pytest

import int4_weight_only_linear_amd as L
from test_adapters_host import backward


@pytest.mark.parametrize("N", [(1 << 23) - 63, 1 << 23, (1 << 26) + 5])
def test_too_many_features(N):
    assert backward(N=N, K=32, g=32, M=256) == 2, L.w4a16_last_error()
    assert "N above" in L.w4a16_last_error()


@pytest.mark.parametrize("N", [(1 << 23) - 64, (1 << 23) - 100])
def test_the_most_features_pass(N):
    # up to the next check, which these pointers fail
    assert backward(N=N, K=32, g=32, M=256, dla=(1 << 40) + 8) == 3
    assert "16-byte" in L.w4a16_last_error()
