"""A quantised cache's rows as the chunk operators set them aside (include/mla_chunk.h),
where the plan's room is far more than the rows there are."""
import numpy as np
import pytest

from chunk_testlib import f64
from mla_testlib import ensure_built
from oracle import chunk as C
from test_gpu_chunk import SCALE, Case

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def m():
    ensure_built()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import head_latent_attention_paged_gb300 as mod
    return mod


@pytest.mark.parametrize("sm_count", [2, 152])
@pytest.mark.parametrize("kv", ["fp8", "fp4"])
def test_room_for_more_rows_than_there_are(m, kv, sm_count):
    """The same bits whether the room is that of the rows or many times it (the warps of
    two multiprocessors' blocks then take several rows' turns each)."""
    case = Case(m, [(3, 1500), (40, 700), (0, 90), (1, 1301)], 4, 64, kv, seed=2, lead=1, pad=2)
    got = []
    for room in (3591, 3600, 5000, 1 << 20):
        case.plan = m.mla_chunk_make_plan(case.problem, case.tokens, context_tokens=room, sm_count=sm_count)
        case.workspace = torch.full((int(case.plan.workspace_bytes),), 0xFF, dtype=torch.uint8, device="cuda")
        case.o.fill_(7.0)
        case.lse.fill_(7.0)
        case.attend()
        case.check_attention()
        out = torch.full((4, 1500), 9.0, device="cuda")
        case.weigh(case.lse, out)
        torch.cuda.synchronize()
        assert int(case.status) == 0
        got.append((case.o.clone(), case.lse.clone(), out))
    for o, lse, out in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(lse, got[0][1]) and torch.equal(out, got[0][2])
    lse = f64(case.lse)
    for b, n in enumerate(case.paged.lens):
        w, t = C.weights(case.queries(b), lse[case.starts[b]:case.starts[b + 1]], case.paged.rows(b), SCALE)
        assert np.all(np.abs(f64(got[0][2][b, :n]) - w) <= t + 2 * C.U * w)
