"""Arrays of the chunk operators that are columns of wider ones."""
import numpy as np
import pytest

from chunk_testlib import Paged, put
from mla_testlib import ensure_built
from oracle import chunk as C
from test_gpu_chunk import Case

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def m():
    ensure_built()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import head_latent_attention_paged_gb300 as mod
    return mod


def test_columns_that_end_where_another_array_begins(m):
    """Two requests of at most 128 slots, their weights 400 elements apart: what stands
    behind the second one's slots may be another array."""
    rng = np.random.default_rng(1)
    paged = Paged(rng, [128, 100], 64, "bf16")
    w = rng.random((2, 128), dtype=np.float32)
    arena = torch.zeros(2 * (400 + 128), device="cuda")
    weights = arena[:528].as_strided((2, 128), (400, 1))
    positions = arena[528:].view(torch.int32).as_strided((2, 128), (400, 1))
    weights.copy_(torch.from_numpy(w))
    positions.copy_(torch.arange(128, dtype=torch.int32).expand(2, 128))
    lens = put(paged.lens, np.int32)
    plan = m.mla_evict_make_plan(paged.problem(m), 60)
    ws = torch.zeros(int(plan.workspace_bytes), dtype=torch.uint8, device="cuda")
    before = paged.cache.clone()
    m.mla_cache_evict(plan, paged.cache, put(paged.table), lens, weights, positions, ws, stride=400)
    torch.cuda.synchronize()
    assert lens.tolist() == [60, 60]
    flat, old = paged.cache.view(-1, 576).cpu().numpy(), before.view(-1, 576).cpu().numpy()
    for b, n in enumerate((128, 100)):
        _, origin = C.evict(w[b, :n], np.arange(n), 60)
        assert np.array_equal(flat[paged.slots[b][:60]], old[paged.slots[b][origin]])
        assert np.array_equal(positions[b, :60].cpu().numpy(), origin)
        assert np.array_equal(weights[b, :60].cpu().numpy(), w[b, origin])
    assert float(arena[128:400].abs().max()) == 0 and float(arena[528 + 128:528 + 400].abs().max()) == 0


def test_weights_in_columns_beside_their_lse(m):
    case = Case(m, [(3, 128), (2, 90)], 4, 64, "bf16")
    case.attend()
    whole = torch.zeros(2, 128, device="cuda")
    case.weigh(case.lse, whole)
    arena = torch.zeros(528 + case.lse.numel(), device="cuda")
    arena[528:] = case.lse.view(-1)
    out = arena[:528].as_strided((2, 128), (400, 1))
    m.mla_cache_weights(case.plan, case.q, arena[528:], case.starts_gpu, case.paged.cache, case.table, case.lens,
                        case.workspace, out, stride=400)
    torch.cuda.synchronize()
    assert torch.equal(out, whole) and torch.equal(arena[528:], case.lse.view(-1))
    assert float(arena[128:400].abs().max()) == 0
