"""GPU: the page pool where lengths and tables do not fit its state (refused as a whole), and the way to take
tokens back."""
import pytest
import torch

from bit_block_scaled_nvfp4_b200 import api, paged
from test_gpu_kv4_attention import Case, KTS, VTS
from test_gpu_pages import DEV, Pair, _state, i32

pytestmark = pytest.mark.gpu


@pytest.mark.status_checked
@pytest.mark.parametrize("fault", ["negative length", "length past the table", "no such page", "negative page", "page that nobody holds"])
@pytest.mark.parametrize("seqs", [4, 300])
def test_refused_compactions_change_nothing(fault, seqs):
    p = Pair(5 * seqs, seqs, 4)
    p.grow([200 - s % 70 for s in range(seqs)])
    p.free(list(range(0, seqs, 2)))
    bad = seqs - 1                                        # the last row, with rows to move before it
    if "length" in fault:
        p.lens[bad] = -1 if fault == "negative length" else 257
    else:
        free = int((p.pool.refs == 0).nonzero()[0])
        p.table[bad, 1] = {"no such page": 5 * seqs, "negative page": -1, "page that nobody holds": free}[fault]
    before = _state(p)
    api.check_status()
    moves = api.kv_pages_compact(p.pool, p.table, p.lens)
    assert api.check_status() == 5
    assert all(torch.equal(a, b) for a, b in zip(_state(p), before))
    assert int(moves.count) == 0 and (moves.src == -1).all() and (moves.dst == -1).all()


@pytest.mark.status_checked
@pytest.mark.parametrize("cut,new", [(100, 101), (100, 130), (127, 128), (1, 400)])
def test_a_page_that_two_sequences_hold_is_not_given_for_appending(cut, new):
    """A fork cut back into a page it shares: what it would append there is another sequence's."""
    p = Pair(20, 3, 7)
    p.grow([128, 30, 0])
    p.fork([0], [2])
    p.lens[2] = cut
    before = _state(p)
    api.check_status()
    api.kv_pages_alloc(p.pool, p.table, p.lens, i32([128, 31, new]))
    assert api.check_status() == 5
    assert all(torch.equal(a, b) for a, b in zip(_state(p), before))
    api.kv_pages_alloc(p.pool, p.table, p.lens, i32([128, 31, cut]))      # not growing, it is nobody's concern
    assert api.check_status() == 0


def test_taking_tokens_back():
    """Proposals stored, attended to and refused, over page boundaries and after a fork: the pool's lens stay
    what has been allocated, the tokens' own lengths fall; no page is lost."""
    hq, hkv, S, W, P = 8, 2, 3, 6, 16
    g = torch.Generator(device=DEV).manual_seed(41)
    cache, pool = paged.empty_cache4(P, hkv, 128, KTS, VTS, DEV), paged.empty_pool(P, DEV)
    table, held = torch.full((S, W), -1, dtype=torch.int32, device=DEV), i32([0] * S)
    have = [0] * S
    hist = [torch.zeros(2, 0, hkv, 128, device=DEV) for _ in range(S)]

    def feed(new):
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        T, start = cu[-1], i32(have)
        k, v = torch.randn(2, T, hkv, 128, generator=g, device=DEV, dtype=torch.bfloat16)
        q = torch.randn(T, hq, 128, generator=g, device=DEV, dtype=torch.bfloat16)
        after = torch.maximum(held, i32([a + n for a, n in zip(have, new)]))
        api.kv_pages_alloc(pool, table, held, after)
        held.copy_(after)
        api.kv4_append_paged(cache, k, v, i32(cu), start, table)
        rk, rv = api.kv4_read_paged(cache, i32(cu), start, table, T, dtype=torch.float32)
        for s, n in enumerate(new):
            hist[s] = torch.cat([hist[s], torch.stack([rk, rv])[:, cu[s]:cu[s + 1]]], 1)
            have[s] += n
        out, lse = api.attn_kv4_paged(q, cache, table, i32(have), W * 64, cu_q=i32(cu), max_q=max(new), want_lse=True)
        c = Case.__new__(Case)
        c.new, c.ctx, c.hq, c.hkv, c.dtype, c.q = new, list(have), hq, hkv, q.dtype, q
        c.cu, c.values = cu, lambda s: (hist[s][0].double(), hist[s][1].double())
        c.check(out, lse)

    def back(counts):
        for s, n in enumerate(counts):
            have[s] -= n
            hist[s] = hist[s][:, :have[s]]

    def pages():
        assert int(pool.refs.sum()) == sum((n + 63) // 64 for n in held.tolist())

    feed([62, 130, 0])
    feed([5, 70, 0])                                      # proposals past a page's end
    back([5, 70, 0])
    feed([2, 1, 0])
    feed([70, 3, 0])
    pages()
    assert held.tolist() == [134, 200, 0]
    assert have[0] >= held[0] // 64 * 64                  # its tokens reach its last page: it can be forked
    api.kv_pages_copy(cache, api.kv_pages_fork(pool, table, held, i32([0]), i32([2])))
    have[2], hist[2] = have[0], hist[0]
    feed([1, 1, 4])
    back([0, 1, 3])                                       # no further than position 128, up to which pages are shared
    feed([3, 2, 9])
    pages()
    for s in range(S):
        k, v = api.kv4_read_paged(cache, i32([0, have[s]]), i32([0]), table[s:s + 1].contiguous(), have[s], dtype=torch.float32)
        assert torch.equal(torch.stack([k, v]), hist[s])
    api.kv_pages_free(pool, table, held, i32([0, 1, 2]))
    assert not pool.refs.any()
