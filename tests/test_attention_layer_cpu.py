"""What runner.AttentionLayer refuses before a kernel is launched: kernels take
addresses, so tensors that are not what their shapes and types have to be are
read wrongly or past their end.  The layer's tensors are on the host here and no
call gets as far as a launch."""
import pytest

torch = pytest.importorskip("torch")

HIDDEN, Q_RANK, HEADS, BATCH, MAX_PAGES = 96, 64, 3, 2, 4


def _weights():
    def w(*shape):
        return torch.zeros(shape, dtype=torch.bfloat16)

    return dict(hidden_norm=w(HIDDEN), w_qkv_a=w(HIDDEN, Q_RANK + 576), q_norm=w(Q_RANK), kv_norm=w(512),
                w_q_b=w(Q_RANK, HEADS * 256), w_uk=w(HEADS, 512, 192), w_uv=w(HEADS, 512, 256), w_o=w(HEADS * 256, HIDDEN))


def _make(**kw):
    from head_latent_attention_paged_gb300 import _build
    _build.build()
    import head_latent_attention_paged_gb300 as m
    from head_latent_attention_paged_gb300.runner import AttentionLayer
    return AttentionLayer(**dict(dict(_weights(), batch=BATCH, num_pages=9, max_pages=MAX_PAGES, rope=m.mla_rope_plan(),
                                      sm_count=152), **kw))


@pytest.fixture(scope="module")
def layer():
    return _make()


def _int(*shape, dtype=torch.int32):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("name,bad", [
    ("positions", _int(5, dtype=torch.int64)), ("positions", _int(10)[::2]), ("positions", _int(5).float()),
    ("requests", _int(4)), ("requests", _int(6)), ("requests", _int(5, dtype=torch.int64)), ("requests", _int(10)[::2]),
    ("requests", torch.zeros(5, dtype=torch.int32, device="meta")),
    ("block_table", _int(BATCH, MAX_PAGES - 1)), ("block_table", _int(BATCH, MAX_PAGES, dtype=torch.int64)),
    ("block_table", _int(MAX_PAGES, BATCH).T),
])
def test_context_refuses(layer, name, bad):
    a = dict(positions=_int(5), requests=_int(5), block_table=_int(BATCH, MAX_PAGES))
    a[name] = bad
    with pytest.raises(ValueError, match=name):
        layer.context(**a)


@pytest.mark.parametrize("name,bad", [
    ("hidden states", torch.zeros(5, HIDDEN)), ("hidden states", torch.zeros(5, HIDDEN, dtype=torch.bfloat16, device="meta")),
    ("hidden states", torch.zeros(4, HIDDEN, dtype=torch.bfloat16)), ("positions", torch.zeros(5, dtype=torch.int32, device="meta")),
    ("requests", _int(4)), ("block_table", _int(BATCH, MAX_PAGES + 1)),
])
def test_prompt_refuses(layer, name, bad):
    a = dict(hidden=torch.zeros(5, HIDDEN, dtype=torch.bfloat16), positions=_int(5), requests=_int(5),
             block_table=_int(BATCH, MAX_PAGES))
    a["hidden" if name == "hidden states" else name] = bad
    with pytest.raises(ValueError, match=name):
        layer.prompt(**a)


@pytest.mark.parametrize("name,bad", [
    ("hidden states", torch.zeros(BATCH, HIDDEN)), ("hidden states", torch.zeros(HIDDEN, BATCH, dtype=torch.bfloat16).T),
    ("positions", _int(BATCH + 1)), ("seq_lens", _int(BATCH, dtype=torch.int64)),
    ("seq_lens", torch.zeros(BATCH, dtype=torch.int32, device="meta")), ("block_table", _int(BATCH, MAX_PAGES)[:, ::2]),
])
@pytest.mark.parametrize("with_residual", [False, True])
def test_decode_refuses(layer, name, bad, with_residual):
    hidden = torch.zeros(BATCH, HIDDEN, dtype=torch.bfloat16)
    a = dict(hidden=hidden, residual=hidden.clone() if with_residual else None, positions=_int(BATCH),
             seq_lens=_int(BATCH), block_table=_int(BATCH, MAX_PAGES))
    a["hidden" if name == "hidden states" else name] = bad
    with pytest.raises(ValueError, match=name):
        layer.decode(**a)
    if with_residual and name == "hidden states":
        with pytest.raises(ValueError, match=name):
            layer.decode(**dict(a, hidden=hidden, residual=bad))


@pytest.mark.parametrize("name", list(_weights()))
@pytest.mark.parametrize("how", ["type", "short", "device", "dims"])
def test_weights_are_refused(name, how):
    good = _weights()[name]
    bad = {"type": good.float(), "short": good[:-1], "device": good.to("meta"), "dims": good[None]}[how]
    # sizes come from three of the weights: one that is short is told from the others by none
    with pytest.raises(ValueError, match="must be a|multiple of 8" if how in ("short", "device") else name):
        _make(**{name: bad})


@pytest.mark.parametrize("name", ["hidden_norm", "q_norm", "kv_norm", "w_uk", "w_uv"])
def test_unpacked_weights_are_refused(name):
    """Those that kernels read by their address; the library products take strides."""
    good = _weights()[name]
    with pytest.raises(ValueError, match=name):
        _make(**{name: torch.zeros(*good.shape[:-1], 2 * good.shape[-1], dtype=good.dtype)[..., ::2]})
    for name in ("w_qkv_a", "w_q_b", "w_o"):
        _make(**{name: torch.zeros_like(_weights()[name].T).T})


def test_ranks_and_rotations_are_refused():
    import head_latent_attention_paged_gb300 as m

    def w(*shape):
        return torch.zeros(shape, dtype=torch.bfloat16)

    with pytest.raises(ValueError, match="multiple of 8"):      # cache rows start behind the query latent
        _make(q_norm=w(60), w_qkv_a=w(HIDDEN, 60 + 576), w_q_b=w(60, HEADS * 256))
    with pytest.raises(ValueError, match="64"):
        _make(rope=m.mla_rope_plan(rope_dim=32))


def test_calls_are_made_on_the_layers_device(monkeypatch):
    """The library works on the current device: with another one current, a
    layer's calls make its own current around every launch.  (Recorded calls in
    place of the library's; no second GPU is needed.)"""
    from head_latent_attention_paged_gb300 import runner
    layer = _make()
    current, seen = [None], []

    class Device:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            current.append(self.device)

        def __exit__(self, *_):
            current.pop()

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: None)
    calls = ("mla_rms_norm", "mla_rope", "mla_cache_append_tokens", "mla_cache_gather", "mla_decode_step", "mla_get_status")
    for name in calls:
        monkeypatch.setattr(runner, name, lambda *a, name=name, **k: seen.append((name, current[-1])) or 0)
    hidden, table = torch.zeros(BATCH, HIDDEN, dtype=torch.bfloat16), _int(BATCH, MAX_PAGES)
    layer.decode(hidden, None, _int(BATCH), table, _int(BATCH))
    layer.prompt(hidden, _int(BATCH), _int(BATCH), table)
    layer.context(_int(BATCH), _int(BATCH), table)
    assert layer.status() == 0
    assert {name for name, _ in seen} == set(calls)
    assert all(device == layer.device for _, device in seen) and current == [None]
