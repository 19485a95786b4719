"""The workspace sizes that the binding keeps (CPU only): asked for once per
sizes, and bounded however many token counts a process meets."""
import contextlib

import pytest

from int4_weight_only_linear_amd import _binding as B

torch = pytest.importorskip("torch")


def test_kept_sizes_are_bounded(monkeypatch):
    monkeypatch.setattr(torch.cuda, "device", lambda device: contextlib.nullcontext())
    asked = []

    def entry_point(M, N):
        asked.append(M)
        return 256 * M + N

    B._sizes.clear()
    device = torch.device("cuda", 0)
    try:
        for M in range(1, 20001):
            assert B._size_of(device, entry_point, M, 7) == 256 * M + 7
            assert B._size_of(device, entry_point, M, 7) == 256 * M + 7
        assert len(asked) == 20000
        assert len(B._sizes) <= 4096
    finally:
        B._sizes.clear()
