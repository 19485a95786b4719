"""A layer of routed 8-bit experts at sizes of tall tiles: captured into graphs and
replayed, and on two streams at once.  Tolerance: none, every result has the bits
of the eager call on one stream."""
import numpy as np
import pytest

from fp8_cases import Weights, planned, values  # noqa: F401  (planned: a fixture)
from gpu_util import note

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import int4_weight_only_linear_amd as L  # noqa: E402

E, TOPK, H, F = 8, 4, 1024, 1280


@pytest.fixture(autouse=True)
def _need_gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    note(f"[gpu] {request.node.nodeid}")


class Chain:
    """Router, up, down and the two gradients, into buffers and with a workspace of its own."""

    def __init__(self, seed, M):
        rng = np.random.default_rng(seed)
        self.rng, self.M = rng, M
        self.up, self.down = Weights(rng, F, H, False, False, E=E), Weights(rng, H, F, False, True, E=E)
        self.x, self.dy = values(rng, M, H, "bf16").cuda(), values(rng, M * TOPK, H, "bf16").cuda()
        self.logits = torch.from_numpy(rng.normal(0, 1.5, (M, E)).astype(np.float32)).cuda()
        self.dw = torch.from_numpy(rng.normal(size=(M, TOPK)).astype(np.float32)).cuda()
        new = lambda shape, dtype=torch.bfloat16: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
        self.out = dict(w=new((M, TOPK), torch.float32), ids=new((M, TOPK), torch.int32), h=new((M * TOPK, F)), y=new((M * TOPK, H)),
                        dh=new((M * TOPK, F)), dl=new((M, E), torch.float32))
        bf16 = L.W4A16_BF16
        need = max(L.w4a16_minifloat_moe_workspace_size(M, TOPK, E, F, H, bf16),
                   L.w4a16_minifloat_moe_workspace_size(M, TOPK, E, H, F, bf16, x_per_slot=True),
                   L.w4a16_minifloat_moe_workspace_size(M, TOPK, E, F, H, bf16, transpose=True, x_per_slot=True))
        self.ws = torch.zeros(need, dtype=torch.uint8, device="cuda")

    def run(self):
        o, kw = self.out, dict(score="sigmoid", renormalize=True, scale=0.1)
        L.w4a16_route(self.logits, TOPK, out=(o["w"], o["ids"]), **kw)
        L.w4a16_minifloat_moe_linear(self.x, self.up.tw, self.up.ts, o["ids"], out=o["h"], workspace=self.ws)
        L.w4a16_minifloat_moe_linear(o["h"], self.down.tw, self.down.ts, o["ids"], o["w"], x_per_slot=True, out=o["y"], workspace=self.ws)
        L.w4a16_minifloat_moe_linear(self.dy, self.down.tw, self.down.ts, o["ids"], o["w"], transpose=True, x_per_slot=True, out=o["dh"],
                                     workspace=self.ws)
        L.w4a16_route_backward(self.dw, self.logits, o["ids"], out=o["dl"], **kw)

    def take(self):
        return {k: v.clone() for k, v in self.out.items()}

    def new_inputs(self, seed):
        rng = np.random.default_rng(seed)
        self.x.copy_(values(rng, self.M, H, "bf16"))
        self.logits.copy_(torch.from_numpy(rng.normal(0, 1.5, (self.M, E)).astype(np.float32)))

    def clear(self):
        for k, v in self.out.items():
            v.fill_(0 if k == "ids" else float("nan"))


def same(a, b):
    return all(torch.equal(a[k].view(torch.int16) if a[k].element_size() == 2 else a[k].view(torch.int32),
                           b[k].view(torch.int16) if b[k].element_size() == 2 else b[k].view(torch.int32)) for k in a)


def test_the_chain_runs_tall_tiles(planned):  # noqa: F811
    c = Chain(0, 3000)
    c.run()
    for call in (lambda: L.w4a16_minifloat_moe_linear(c.x, c.up.tw, c.up.ts, c.out["ids"]),
                 lambda: L.w4a16_minifloat_moe_linear(c.dy, c.down.tw, c.down.ts, c.out["ids"], transpose=True, x_per_slot=True)):
        assert planned(call)[1][0] >= 96


def test_captured_and_replayed():
    a, b = Chain(1, 3000), Chain(2, 2500)
    graphs = []
    for c in (a, b):
        c.run()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run()
        graphs.append(g)
    for seed in range(3):
        want = []
        for c in (a, b):
            c.new_inputs(10 + seed)
            c.run()
            want.append(c.take())
            c.clear()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert same(a.take(), want[0]) and same(b.take(), want[1])


def test_two_streams_at_once():
    chains = [Chain(3, 3000), Chain(4, 2700)]
    want = []
    for c in chains:
        c.run()
        want.append(c.take())
        c.clear()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in chains]
    for _ in range(4):
        for c, s in zip(chains, streams):
            with torch.cuda.stream(s):
                c.run()
    torch.cuda.synchronize()
    assert all(same(c.take(), w) for c, w in zip(chains, want))
