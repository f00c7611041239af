"""Host-side checks of the 4-bit cache's and the page pool's calls, without a GPU: move lists that do not
belong together, and the device a workspace is sized for."""
import contextlib

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


def test_the_workspace_is_sized_for_the_tensors_device(monkeypatch):
    """Its size goes with the device's SMs: the library answers for the current device, so the tensors' is entered."""
    entered, asked = [0], []

    @contextlib.contextmanager
    def device(d):
        entered.append(torch.device("cuda", d).index if isinstance(d, int) else d.index)
        yield
        entered.pop()

    class Lib:
        @staticmethod
        def attn_kv4_paged_workspace_size(p):
            asked.append(entered[-1])
            return 64

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: entered[-1])
    monkeypatch.setattr(api._lib, "load", lambda: Lib)
    with pytest.raises(ValueError):                       # (no GPU here: the workspace is refused after that)
        api._kv4_workspace(api._lib.Kv4AttnParams(), torch.empty(64, dtype=torch.uint8), torch.device("cuda", 1))
    assert asked == [1] and entered == [0]
