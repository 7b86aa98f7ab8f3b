"""What a tracking runner.AttentionLayer notes of the tokens it caches (the slots'
positions and weights), with the layer's tensors on the host and recorded calls in
place of the library's."""
import pytest

from test_attention_layer_cpu import BATCH, HIDDEN, MAX_PAGES, _int, _make

torch = pytest.importorskip("torch")

SLOTS = MAX_PAGES * 64


class _Nowhere:
    def __init__(self, device):
        pass

    def __enter__(self):
        pass

    def __exit__(self, *_):
        pass


@pytest.fixture
def calls(monkeypatch):
    """[(name, arguments, keywords)] of the library's calls, none of which is made."""
    from head_latent_attention_paged_gb300 import runner
    seen = []
    monkeypatch.setattr(torch.cuda, "device", _Nowhere)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: None)
    for name in ("mla_rms_norm", "mla_rope", "mla_cache_append_tokens", "mla_q_absorb", "mla_decode_step",
                 "mla_chunk_attend", "mla_cache_weights"):
        monkeypatch.setattr(runner, name, lambda *a, name=name, **k: seen.append((name, a, k)))
    return seen


def _i32(*values):
    return torch.tensor(values, dtype=torch.int32)


def _live(layer):
    """The slots' entries, without the one of padding."""
    return layer.slot_positions[:, :SLOTS], layer.weights[:, :SLOTS]


def _hidden(n):
    return torch.zeros(n, HIDDEN, dtype=torch.bfloat16)


def test_requests_outside_the_batch_note_nothing(calls):
    """The append reports them and writes no row; neither is anything noted."""
    layer = _make(track=True)
    table = _int(BATCH, MAX_PAGES)
    bad = [-1, BATCH, BATCH + 1, 2**31 - 1, -2**31]
    positions, requests = _i32(5, *[7] * len(bad), 6), _i32(1, *bad, 0)
    n = len(bad) + 2
    want = torch.full((BATCH, SLOTS), -1, dtype=torch.int32)
    want[1, 5], want[0, 6] = 5, 6
    layer.prompt(_hidden(n), positions, requests, table)
    assert torch.equal(_live(layer)[0], want)
    layer.slot_positions.fill_(-1)
    layer.prefill(_hidden(n), None, positions, requests, _i32(0, 1, n), table, _i32(7, 6), context_tokens=0)
    assert torch.equal(_live(layer)[0], want)
    # slots of their own, and positions and slots out of range
    layer.slot_positions.fill_(-1)
    layer.prefill(_hidden(n), None, positions, requests, _i32(0, 1, n), table, _i32(7, 6), context_tokens=0,
                  slots=_i32(5, *[2] * len(bad), SLOTS))
    want[0, 6] = -1
    assert torch.equal(_live(layer)[0], want)


def test_a_layer_of_no_requests_notes_nothing(calls):
    """Every request is outside its batch."""
    layer = _make(track=True, batch=0)
    layer.prompt(_hidden(2), _i32(0, 1), _i32(0, -1), _int(0, MAX_PAGES))
    assert calls[-1][0] == "mla_cache_append_tokens" and layer.slot_positions.numel() == 0


def test_padding_with_slots_caches_nothing(calls):
    """A token of position -1 is padding whatever its slot says: the append, whose
    positions are the slots, gets a negative one for it."""
    layer = _make(track=True)
    table, requests = _int(BATCH, MAX_PAGES), _i32(0, 1, 0, 1)
    positions, slots = _i32(9, 12, -1, -1), _i32(3, 4, 0, 7)
    layer.prefill(_hidden(4), None, positions, requests, _i32(0, 1, 2), table, _i32(4, 5), context_tokens=0, slots=slots)
    layer.decode(_hidden(BATCH), None, _i32(-1, 13), table, _i32(0, 6), slots=_i32(0, 5))
    appends = [a for name, a, _ in calls if name == "mla_cache_append_tokens"]
    assert [a[3].tolist() for a in appends] == [[3, 4, -1, -1], [-1, 5]]
    where = torch.full((BATCH, SLOTS), -1, dtype=torch.int32)
    where[0, 3], where[1, 4], where[1, 5] = 9, 12, 13
    assert torch.equal(_live(layer)[0], where) and slots.tolist() == [3, 4, 0, 7]


def test_a_slot_written_again_starts_without_weight(calls):
    """A rejected draft's slot, or one of an earlier request's: what its token got is
    not the new one's."""
    layer = _make(track=True)
    table = _int(BATCH, MAX_PAGES)
    layer.weights.copy_(torch.arange(layer.weights.numel()).view_as(layer.weights) + 1.0)
    want = _live(layer)[1].clone()
    layer.prompt(_hidden(3), _i32(5, 6, -1), _i32(0, 1, 1), table)
    want[0, 5] = want[1, 6] = 0
    assert torch.equal(_live(layer)[1], want)
    layer.decode(_hidden(BATCH), None, _i32(9, -1), table, _i32(10, 0))
    want[0, 9] = 0
    assert torch.equal(_live(layer)[1], want)
    layer.prefill(_hidden(4), None, _i32(30, 31, 32, -1), _i32(1, 1, BATCH, 0), _i32(0, 0, 2), table, _i32(9, 4),
                  context_tokens=0, slots=_i32(2, 3, 4, 1))
    want[1, 2] = want[1, 3] = 0
    assert torch.equal(_live(layer)[1], want)
    # before the weights of the call's queries are added
    names = [name for name, _, _ in calls]
    assert names.index("mla_cache_append_tokens") < names.index("mla_cache_weights")


def test_forget_clears_one_request(calls):
    layer = _make(track=True)
    layer.weights.fill_(3.0)
    layer.slot_positions.fill_(8)
    layer.forget(1)
    assert float(layer.weights[0].min()) == 3.0 and int(layer.slot_positions[0].min()) == 8
    assert float(layer.weights[1].abs().max()) == 0 and int(layer.slot_positions[1].max()) == -1
    _make().forget(0)                                  # a layer that does not track has nothing to forget


@pytest.mark.parametrize("track", [False, True])
def test_prefill_of_no_tokens(monkeypatch, track):
    """A step of the program in which no request has new tokens: nothing is launched."""
    monkeypatch.setattr(torch.cuda, "device", _Nowhere)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: None)
    layer = _make(track=track)
    none, table = _i32(), _int(BATCH, MAX_PAGES)
    for residual in (None, _hidden(0)):
        out, summed = layer.prefill(_hidden(0), residual, none, none, _int(BATCH + 1), table, _i32(3, 4))
        assert out.shape == summed.shape == (0, HIDDEN) and out.dtype == torch.bfloat16


def _room(layer, calls):
    """Expanded rows that the plans of a layer's calls have room for."""
    return [a[0].context_tokens for name, a, _ in calls if name == "mla_chunk_attend"]


def test_room_for_requests_that_share_pages(calls):
    """Over a quantised cache each request's rows are set aside by themselves: more than
    the pool holds where requests share pages."""
    import head_latent_attention_paged_gb300 as m
    kw = dict(kv_dtype=m.MLA_KV_FP8_E4M3_E8M0, num_pages=MAX_PAGES)
    layer = _make(track=True, **kw)
    assert layer.step_plan.context_tokens == BATCH * SLOTS
    table = _int(BATCH, MAX_PAGES)

    def prefill(layer, n, **more):
        layer.prefill(_hidden(n), None, _int(n), _int(n), _int(BATCH + 1), table, _int(BATCH), **more)
        return _room(layer, calls)[-1]

    # a call of one token has new tokens of one request at most
    assert prefill(layer, 1) == SLOTS and prefill(layer, 5) == BATCH * SLOTS
    assert prefill(layer, 5, context_tokens=77) == 77
    # what the program knows of its requests' lengths, for the layer's life
    layer = _make(track=True, context_tokens=100, **kw)
    assert layer.step_plan.context_tokens == 100 and prefill(layer, 5) == 100
    assert prefill(layer, 5, context_tokens=77) == 77
    assert prefill(_make(context_tokens=0, **kw), 5) == 0
    for bad in (-1, 2**31):
        with pytest.raises(m.MlaError):
            _make(track=True, context_tokens=bad, **kw)
