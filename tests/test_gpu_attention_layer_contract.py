"""runner.AttentionLayer on the GPU: what its calls leave behind (the prompt's
cache rows from their own projection, a residual stream that is the layer's own
output)."""
import numpy as np
import pytest

from oracle import layer as L
from mla_testlib import ensure_built
from test_gpu_attention_layer import EPS, HIDDEN, Q_RANK, _f64, _layer

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def m():
    ensure_built()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import head_latent_attention_paged_gb300 as mod
    return mod


def test_decode_of_its_own_output_without_a_residual(m):
    """Fed its last output as hidden states and no residual, decode() returns
    those hidden states as the residual stream, not the output it writes."""
    g = torch.Generator(device="cuda").manual_seed(5)
    layer, _, _ = _layer(m, g, 4, 3, 1, m.MLA_KV_BF16, "pairs", "none")
    bt = torch.arange(18, dtype=torch.int32, device="cuda").view(3, 6)
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    hidden = torch.randn(3, HIDDEN, generator=g, device="cuda", dtype=torch.bfloat16)
    out, res = layer.decode(hidden, None, pos, bt, pos + 1)
    assert res.data_ptr() == hidden.data_ptr()
    before = out.clone()
    again, res = layer.decode(out, None, pos + 1, bt, pos + 2)
    torch.cuda.synchronize()
    assert torch.equal(res, before) and not torch.equal(again, before)
    other, _, _ = _layer(m, torch.Generator(device="cuda").manual_seed(5), 4, 3, 1, m.MLA_KV_BF16, "pairs", "none")
    other.decode(hidden, None, pos, bt, pos + 1)
    want, _ = other.decode(before, None, pos + 1, bt, pos + 2)
    assert torch.equal(again, want)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("layout,scaling", [("pairs", "none"), ("halves", "yarn")])
def test_prompt_caches_its_own_projection(m, kv, layout, scaling):
    """The rows that prompt() leaves in the pool, chunk by chunk: the layer's
    projection of its normed input (the same product on the same chunk), its
    latent normed, its key rotated, quantised; every other slot as it was."""
    kind = {"bf16": m.MLA_KV_BF16, "fp8": m.MLA_KV_FP8_E4M3_E8M0, "fp4": m.MLA_KV_FP4_E2M1_E8M0}[kv]
    row = {"bf16": 1152, "fp8": 594, "fp4": 324}[kv]
    g = torch.Generator(device="cuda").manual_seed(6)
    rng = np.random.default_rng(6)
    layer, freq, amplitude = _layer(m, g, 4, 3, 1, kind, layout, scaling)
    P, max_pages, pages = layer.problem.page_size, layer.problem.max_pages_per_seq, layer.problem.num_pages
    table = rng.permutation(pages)[:3 * max_pages].reshape(3, max_pages).astype(np.int32)
    put = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    lens = np.array([0, P, 217])
    req = np.repeat(np.arange(3), lens).astype(np.int32)
    pos = np.concatenate([np.arange(n) for n in lens]).astype(np.int32)
    order = rng.permutation(len(req))
    req, pos = req[order], pos[order]
    hidden = torch.randn(len(req), HIDDEN, generator=g, device="cuda", dtype=torch.bfloat16)
    slots = L.slots_of(pos, req, table, P, pages)
    assert (slots >= 0).all()
    for part in (slice(0, 70), slice(70, 70), slice(70, None)):
        layer.prompt(hidden[part], put(pos[part]), put(req[part]), put(table))
        n = len(pos[part])
        if n == 0:
            continue
        x = torch.empty_like(hidden[part])
        m.mla_rms_norm(m.make_norm_problem(n, HIDDEN, eps=EPS), hidden[part], layer.hidden_norm, x)
        _, want, t = L.rms_norm(_f64(hidden[part]), weight=_f64(layer.hidden_norm), eps=np.float32(EPS))
        L.assert_rounded(_f64(x), want, t, "bf16", "prompt norm")
        rows = _f64(torch.matmul(x, layer.w_qkv_a))[:, Q_RANK:]
        y, t = L.row_values(rows, pos[part], _f64(layer.kv_norm), np.float32(EPS), freq, amplitude, layout)
        raw = layer.cache.view(-1, row)[put(slots[part])].cpu().numpy()
        if kv == "bf16":
            raw = (raw.view(np.uint16).astype(np.uint32) << 16).view(np.float32)
        L.assert_cache_rows(raw, y, t, kv, "prompt rows")
    rest = np.setdiff1d(np.arange(pages * P), slots)
    assert int(layer.cache.view(-1, row)[put(rest)].max()) == 0
    assert layer.status() == 0
