"""The binding of include/mla_chunk.h takes a stride from its tensors' shapes where none
is given: arrays that this one stride does not describe are refused, as every row but
the first would be read and written elsewhere, or past its end."""
import pytest

from test_chunk_cpu import A, _code, _evict, _problem, _weigh, m  # noqa: F401

torch = pytest.importorskip("torch")


def _f32(*shape):
    return torch.zeros(shape)


def _i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


@pytest.mark.parametrize("kw", [
    dict(out=_f32(4, 200)[:, :100]), dict(out=_f32(100, 4).T), dict(into=_f32(4, 99)), dict(into=_f32(4, 200)[:, :100]),
    dict(into=_f32(4, 200)[:, ::2])])
def test_weights_of_other_strides(m, kw):  # noqa: F811
    with pytest.raises(ValueError, match="stride"):
        _weigh(m, **dict(dict(out=_f32(4, 100), into=None, stride=None), **kw))


@pytest.mark.parametrize("kw", [
    dict(w=_f32(4, 101)[:, :100]), dict(pos=_i32(4, 99)), dict(pos=_i32(100, 4).T), dict(wo=_f32(4, 101)),
    dict(po=_i32(4, 200)[:, :100]), dict(po=_i32(4, 90))])
def test_evictions_of_other_strides(m, kw):  # noqa: F811
    with pytest.raises(ValueError, match="stride"):
        _evict(m, **dict(dict(w=_f32(4, 100), pos=_i32(4, 100), wo=None, po=None, lo=None, stride=None), **kw))


def test_packed_tensors_get_as_far_as_the_library(m):  # noqa: F811
    """And a given stride is taken as it is (the workspace's size is refused behind it)."""
    assert _code(m, _weigh, m, out=_f32(4, 100), into=_f32(4, 100), stride=None, size=1) == m.MLA_ERR_WORKSPACE_TOO_SMALL
    assert _code(m, _weigh, m, out=_f32(4, 200)[:, :100], into=A[8], stride=200, size=1) == m.MLA_ERR_WORKSPACE_TOO_SMALL
    assert _code(m, _evict, m, w=_f32(4, 100), pos=_i32(4, 100), wo=None, po=None, lo=None, stride=None,
                 size=1) == m.MLA_ERR_WORKSPACE_TOO_SMALL
    assert _code(m, _evict, m, w=_f32(4, 200)[:, :100], pos=_i32(4, 200)[:, :100], wo=None, po=None, lo=None, stride=200,
                 size=1) == m.MLA_ERR_WORKSPACE_TOO_SMALL
