"""Which queries a step retrieves its pages by, on a machine without a GPU (its kernels' calls are replaced)."""
import warnings

import pytest

from hybrid_sparse_attention_hkv_b200 import step as module


class Retrieved(Exception):
    pass


@pytest.fixture
def step(monkeypatch):
    st = module.HkvHsaStep.__new__(module.HkvHsaStep)
    st.store, st.out, st.rope = None, None, None
    st.kbar_pages = st.Kp = st.sel = st.ws = st.scores = None

    def select(kbar, Q, *a):
        raise Retrieved(Q)
    monkeypatch.setattr(module, "hkv_select_pages", select)
    return st


CALLS = [lambda st, **kw: st("rotated", None, None, None, None, None, None, **kw), lambda st, **kw: st.prepare_chunk("rotated", None, None, **kw)]


@pytest.mark.parametrize("call", CALLS)
def test_rotated_queries_in_the_place_of_unrotated_ones_are_told_of(step, call):
    """The summaries are of the keys before their rotation: retrieving by the chunk's rotated queries is not silent."""
    step.rope = object()
    with pytest.warns(UserWarning, match="q_pages"):
        with pytest.raises(Retrieved, match="rotated"):
            call(step)


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("rope,kw,used", [(None, {}, "^rotated"), (None, dict(q_pages="before"), "^before"), (object(), dict(q_pages="before"), "^before"),
                                          (object(), dict(q_pages="rotated"), "^rotated")])
def test_queries_that_are_given_are_used_without_a_word(step, call, rope, kw, used):
    step.rope = rope
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(Retrieved, match=used):
            call(step, **kw)
