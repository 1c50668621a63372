"""The paged layer's own checks: what it refuses, and that a refused call leaves it as it was (no GPU)."""
import pytest
import torch

import compressed_sparse_attention_13_b200 as K
from compressed_sparse_attention_13_b200.paged import PagedLayer


def layer(n_seq=3, n_pages=6, max_pages=4):
    return PagedLayer(K.gqa_params(8, 2, 128, 0.1, page_size=4), n_seq=n_seq, n_pages=n_pages, max_pages=max_pages, device="cpu")


def state(lay):
    return list(lay.lens), [list(h) for h in lay._held], sorted(lay._free), lay.table.tolist(), lay.pos.tolist()


@pytest.mark.parametrize("lens", [[5, 4, 2], [0, 0, 11], [11, 0, 0]])
def test_a_prefill_of_more_tokens_than_rows_is_refused(lens):
    lay = layer()
    q, k, v = (torch.zeros(10, h, 128, dtype=torch.bfloat16) for h in (8, 2, 2))
    before = state(lay)
    with pytest.raises(ValueError, match="11 tokens in 10 rows"):
        lay.prefill(lens, q, k, v, None, torch.zeros_like(q))
    assert state(lay) == before


@pytest.mark.parametrize("lens,match", [([1, 2], "3 lengths"), ([1, 2, 3, 0], "3 lengths"), ([4, -1, 2], "at least 0"),
                                        ([0, 3, 0], "holds tokens")])
def test_a_prefill_of_wrong_lengths_is_refused(lens, match):
    lay = layer()
    lay.reserve(1, 3)
    lay.lens[1] = 3
    q, k, v = (torch.zeros(10, h, 128, dtype=torch.bfloat16) for h in (8, 2, 2))
    before = state(lay)
    with pytest.raises(ValueError, match=match):
        lay.prefill(lens, q, k, v, None, torch.zeros_like(q))
    assert state(lay) == before


@pytest.mark.parametrize("active", [[1, 1], [0, 2, 0], [3], [-1], [2, -1]])
def test_a_step_of_a_sequence_named_twice_or_of_none_is_refused(active):
    """Named twice, a sequence would move on by two tokens with room for one, and only one of them would be written."""
    lay = layer()
    for s in range(3):
        lay.reserve(s, 4)
        lay.lens[s] = 4
    before = state(lay)
    with pytest.raises(ValueError, match="each once"):
        lay.advance(active)
    assert state(lay) == before
    lay.advance([2, 0])
    assert lay.lens == [5, 4, 5] and lay.pos.tolist() == [4, -1, 4]


def test_prompts_that_find_no_room_take_no_pages():
    """The pool holds the first two prompts and not the third: none of its pages stays with an empty sequence."""
    lay = layer()
    q, k, v = (torch.zeros(30, h, 128, dtype=torch.bfloat16) for h in (8, 2, 2))
    before = state(lay)
    for lens in ([8, 8, 9], [8, 0, 17]):   # 2 + 2 + 3 of 6 pages; 5 pages of a table of 4
        with pytest.raises(RuntimeError, match="sequence 2: no room"):
            lay.prefill(lens, q, k, v, None, torch.zeros_like(q))
        assert state(lay) == before
    for s, n in ((0, 8), (1, 8), (2, 8)):
        lay.reserve(s, n)
        lay.lens[s] = n
    lay.release(2)
    lay.reserve(2, 3)
    lay.lens[2] = 3
    before = state(lay)
    with pytest.raises(RuntimeError, match="sequence 1: no room"):
        lay.advance()      # one page is left for the two that need one
    assert state(lay) == before
