"""The calls for several candidates a sequence at the C boundary, without a GPU: what they refuse before they touch one."""
import pytest

import gqa_decode_attention_paged_gb300 as pkv


@pytest.fixture(scope="module")
def lib():
    return pkv.load()


def test_calls_without_a_pool_fail_cleanly(lib):
    assert lib.paged_tree_attention(None, None, 1, 8, None, None, 1, None, 1, None, 1, 1.0, None, None) == 1
    assert lib.paged_tree_reserve_workspace(None, 1, 8) == 1
    assert lib.paged_tree_commit(None, None, None, 1, None, None, 1, None, 1, None, None) == 1
    assert lib.paged_beam_select(None, None, 0, 10, None, 1, 1, 10, 1, None, None, None, None) == 1
    assert lib.paged_beam_reserve_workspace(None, 1, 1, 10, 1) == 1
    assert lib.paged_beam_reorder(None, None, 1, 1, 1, None, 1, None, None, None, None, None) == 1
    assert b"NULL pool" in lib.pkv_last_error_message()


def test_the_names_are_public():
    for name in ("paged_tree_attention", "paged_tree_commit", "paged_beam_select", "paged_beam_reorder"):
        assert name in pkv.__all__ and callable(getattr(pkv, name))
    assert pkv.DEVERR_NAN == 16


def test_arguments_that_are_no_tensors_are_refused_by_name():
    for call in (lambda: pkv.paged_beam_select(None, [[0.0]], None, 1), lambda: pkv.paged_beam_reorder(None, [[0]], None, None, None),
                 lambda: pkv.paged_tree_attention(None, [[0.0]], None, None, None, None, 1.0)):
        with pytest.raises(TypeError):
            call()
