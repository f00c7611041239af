"""Host-side checks of the page pool's calls, without a GPU: move lists that do not belong together."""
import pytest
import torch

from bit_block_scaled_nvfp4_b200 import api, paged


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


@pytest.mark.parametrize("src,dst,count,error,what", [
    (i32(3), i32(2), None, ValueError, "moves.dst"), (i32(3).long(), i32(3), None, TypeError, "moves.src"),
    (i32(3), i32(3).long(), None, TypeError, "moves.dst"), (i32(3), i32(3, 1), None, ValueError, "moves.dst"),
    (i32(3), i32(3), i32(2), ValueError, "moves.count"), (i32(3), i32(3), i32(1).long(), TypeError, "moves.count")])
def test_page_copies_check_their_lists(src, dst, count, error, what):
    """Lists of two lengths, or of 64-bit numbers, would be read past their end or as other pages."""
    cache = paged.empty_cache4(30, 2, 128, 1.0, 1.0, "cpu")
    with pytest.raises(error, match=what):
        api.kv_pages_copy(cache, api.PageMoves(src, dst, 30, count))
    if count is None:
        with pytest.raises(error, match=what):
            api.kv_tails_copy(torch.zeros(4, 1, 128, 32), api.PageMoves(i32(3), i32(3), 30, None, src, dst))
