"""AdamW with copies of some of the parameters only, in every arrangement."""
import pytest

from gpu_util import note
from test_adamw_gpu import L, step, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    note(f"[gpu] {request.node.nodeid}")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("has", [(True, False, True), (False, True, False), (False, False, True), (False, False, False), None])
def test_some_copies(has, dtype):
    sizes = [300, 77, 1024]
    make = lambda k: [torch.randn(n, generator=torch.Generator().manual_seed(n + k)).cuda() for n in sizes]  # noqa: E731
    P, G, Ms, Vs = make(0), make(1), make(2), [v.square() for v in make(3)]
    C = None if has is None else [torch.full((n,), 9.0, dtype=dtype, device="cuda") if h else None for n, h in zip(sizes, has)]
    ref_p = [p.clone() for p in P]
    step(L.w4a16_adamw_plan(ref_p, G, [m.clone() for m in Ms], [v.clone() for v in Vs]))
    step(L.w4a16_adamw_plan(P, G, Ms, Vs, copies=C))
    assert all(torch.equal(a, b) for a, b in zip(P, ref_p))
    for c, p in zip(C or [], P):
        assert c is None or torch.equal(c, p.to(dtype))


def test_copies_of_two_types_are_refused():
    z = lambda dt=torch.float32: torch.zeros(8, dtype=dt, device="cuda")  # noqa: E731
    for kinds in ((torch.float16, torch.bfloat16), (None, torch.float32)):
        copies = [None if k is None else z(k) for k in kinds]
        with pytest.raises(TypeError):
            L.w4a16_adamw_plan([z(), z()], [z(), z()], [z(), z()], [z(), z()], copies=copies)
