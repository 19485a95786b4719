"""Layers and references of the 8-bit products' GPU tests at sizes whose tiles
are 64, 96 and 128 tokens high: references for a sample of the outputs, and the
plan that a call ran with, from the library's log."""
import re

import numpy as np
import pytest

from oracle import experts_ref as X

torch = pytest.importorskip("torch")
import int4_weight_only_linear_amd as L  # noqa: E402

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
_PLAN = re.compile(r"\[w4a16\] minifloat_\w+ slots=.* (?:decode|tile=(\d+)x128 splits=(\d+) steps=\d+)\n")


@pytest.fixture
def planned(monkeypatch, capfd):
    """planned(call): call(), and (tile height, K ranges) of the product that it ran, None for decode."""
    monkeypatch.setenv("W4A16_LOG", "1")
    L.w4a16_reload_tuning()

    def run(call):
        capfd.readouterr()
        out = call()
        found = _PLAN.findall(capfd.readouterr().err)
        assert len(found) == 1, found
        return out, tuple(map(int, found[0])) if found[0][0] else None
    yield run
    monkeypatch.undo()
    L.w4a16_reload_tuning()


class Weights:
    """Codes and block scales of one layer (E None) or of E experts: w [N, K], transposed [K, N].  scales: the fp32
    block scales, or e8m0 bytes, or None for ordinary ones."""

    def __init__(self, rng, N, K, transpose, e8m0, E=None, bias=None, scales=None):
        self.N, self.K, self.tr, self.E = N, K, transpose, E
        lead = () if E is None else (E,)
        shape = lead + ((K, N) if transpose else (N, K))
        blocks = lead + tuple((n + 127) // 128 for n in shape[-2:])
        # normal values, drawn from a table of them: these are many
        table = X.to_e4m3(np.clip(rng.normal(0, 107, 4096), -448, 448))
        self.w = table[rng.integers(0, 4096, shape, dtype=np.uint16)]
        if scales is None:
            scales = rng.integers(110, 118, blocks).astype(np.uint8) if e8m0 else (rng.uniform(0.5, 1.5, blocks) * 2e-4).astype(np.float32)
        self.set_scales(scales)
        self.tw = torch.from_numpy(self.w).view(torch.float8_e4m3fn).cuda()
        self.bias = None if bias is None else torch.from_numpy(rng.normal(0, 0.5, lead + (N,))).to(TYPES[bias]).cuda()

    def set_scales(self, s):
        self.e8m0 = s.dtype == np.uint8
        if self.e8m0:
            self.ws = np.where(s == 255, np.nan, 2.0 ** (s.astype(np.float64) - 127))
            self.ts = torch.from_numpy(s).view(torch.float8_e8m0fnu).cuda()
        else:
            self.ws, self.ts = s.astype(np.float64), torch.from_numpy(s).cuda()

    def of(self, cols, e=None):
        """(codes of the features `cols` of a layer or of expert e, each one's scales)."""
        w, ws = (self.w, self.ws) if e is None else (self.w[e], self.ws[e])
        return (w[:, cols], ws[:, np.asarray(cols) // 128]) if self.tr else (w[cols], ws[np.asarray(cols) // 128])

    def reference(self, codes, scales, cols, e=None):
        """fp8_linear_ref of some rows of codes and features."""
        w, ws = self.of(cols, e)
        y, slack = np.empty((len(codes), len(cols))), np.empty((len(codes), len(cols)))
        for b in np.unique(np.asarray(cols) // 128):
            at = np.nonzero(np.asarray(cols) // 128 == b)[0]
            for i in range(0, len(at), 128):
                j = at[i:i + 128]
                part = (w[:, j], ws[:, j[:1]]) if self.tr else (w[j], ws[j[:1]])
                y[:, j], slack[:, j] = X.fp8_linear_ref(codes, scales, *part, self.K, self.tr)
        return y, slack

    def dense(self, e=None):
        """The scaled weights [K, N] in fp32 on the device."""
        w, s = (self.tw, self.ts) if e is None else (self.tw[e], self.ts[e])
        s = s.float().repeat_interleave(128, -1)[:, :w.shape[1]].repeat_interleave(128, 0)[:w.shape[0]]
        w = w.float() * s
        return w if self.tr else w.T


def edges(rng, n, tile, more):
    """Places at the edges of tiles, at the ends, and `more` others, of 0 .. n - 1."""
    at = {0, n - 1, n // tile * tile, n // tile * tile - 1, tile - 1, tile, tile // 2, n - n % 16}
    at |= set(rng.integers(0, n, more).tolist())
    return np.array(sorted(i for i in at if 0 <= i < n))


def values(rng, M, K, dtype):
    x = rng.normal(size=(M, K)) * np.exp(rng.normal(0, 0.7, K))
    return torch.from_numpy(x).to(TYPES[dtype])
