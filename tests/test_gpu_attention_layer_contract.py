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
