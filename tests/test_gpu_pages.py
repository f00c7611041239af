"""GPU parity of the page pool against the oracle's lists: allocation, forks, frees, compaction
and the page copies they ask for, in runs as a server makes them, and the calls that are
refused as a whole."""
import random

import numpy as np
import pytest
import torch

from bit_block_scaled_nvfp4_b200 import api, paged
from oracle import kv4 as OK

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Pair:
    """The pool on the GPU next to the oracle's, and the page contents as one number a page."""

    def __init__(self, pages, seqs, width):
        self.want = OK.Pool(pages, seqs, width)
        self.pool = paged.empty_pool(pages, DEV)
        self.table = torch.full((seqs, width), -1, dtype=torch.int32, device=DEV)
        self.lens = torch.zeros(seqs, dtype=torch.int32, device=DEV)

    def same(self):
        assert self.pool.refs.tolist() == self.want.refs
        assert self.lens.tolist() == self.want.lens
        for s, n in enumerate(self.want.lens):
            k = self.want.pages_of(n)
            assert self.table[s, :k].tolist() == self.want.table[s][:k], s

    def grow(self, new):
        self.want.alloc(new)
        api.kv_pages_alloc(self.pool, self.table, self.lens, i32(new))
        k = [self.want.pages_of(n) for n in new]
        for s in range(len(new)):
            assert self.table[s, :k[s]].tolist() == self.want.table[s][:k[s]]
        self.want.lens = list(new)
        self.lens.copy_(i32(new))
        self.same()

    def fork(self, src, dst):
        moves = self.want.fork(src, dst)
        got = api.kv_pages_fork(self.pool, self.table, self.lens, i32(src), i32(dst))
        assert list(zip(got.src.tolist(), got.dst.tolist())) == moves
        assert got.seq_src.tolist() == src and got.seq_dst.tolist() == dst
        self.same()
        return got

    def free(self, seqs):
        self.want.free(seqs)
        api.kv_pages_free(self.pool, self.table, self.lens, i32(seqs))
        self.same()

    def compact(self):
        moves = self.want.compact()
        got = api.kv_pages_compact(self.pool, self.table, self.lens)
        n = int(got.count)
        assert n == len(moves) and list(zip(got.src.tolist(), got.dst.tolist()))[:n] == moves
        assert (got.src[n:] == -1).all() and (got.dst[n:] == -1).all()
        self.same()
        return got


@pytest.mark.parametrize("pages,seqs,width,longest", [(40, 5, 6, 300), (1, 2, 1, 64), (9001, 90, 40, 2500), (4096, 3, 700, 40000)])
def test_runs_of_pool_calls_match_the_oracle(pages, seqs, width, longest):
    r = random.Random(pages)
    p = Pair(pages, seqs, width)
    for step in range(14):
        new = [min(n + r.choice([0, 1, 1, r.randint(0, longest)]), longest, 64 * width) for n in p.want.lens]
        new = [max(a, b) for a, b in zip(new, p.want.lens)]
        free = p.want.refs.count(0)
        for s in range(seqs):                                     # as far as the pool reaches
            need = p.want.pages_of(new[s]) - p.want.pages_of(p.want.lens[s])
            if need > free:
                new[s] = p.want.lens[s]
            else:
                free -= need
        p.grow(new)
        empty = [s for s in range(seqs) if p.want.lens[s] == 0]
        if empty:
            dst = r.sample(empty, r.randint(1, len(empty)))
            src = [r.choice([s for s in range(seqs) if s != d]) for d in dst]
            if sum(p.want.lens[s] % 64 != 0 for s in src) <= p.want.refs.count(0):
                p.fork(src, dst)
        if r.random() < 0.7:
            p.free(r.sample(range(seqs), r.randint(0, seqs // 2 + 1)))
        if step % 3 == 2:
            p.compact()
    p.free(list(range(seqs)))
    assert not p.pool.refs.any()


@pytest.mark.parametrize("hkv,kind", [(1, "4"), (3, "4"), (8, "4"), (2, "8")])
def test_copies_of_page_contents(hkv, kind):
    pages = 57
    cache = paged.empty_cache4(pages, hkv, 128, 1.0, 1.0, DEV) if kind == "4" else paged.empty_cache(pages, hkv, 128, 1.0, DEV)
    arrays = [cache.k_pages, cache.k_scales, cache.v_pages, cache.v_scales]
    for a in arrays:
        a.random_(0, 256)
    want = [a.clone() for a in arrays]
    r = random.Random(hkv)
    ids = r.sample(range(pages), 30)
    src, dst = [r.choice(ids[:10]) for _ in range(20)], ids[10:]
    for a in want:
        for s, d in zip(src, dst):
            a[d] = a[s]
    moves = paged.page_moves(src, dst, pages, DEV)
    api.kv_pages_copy(cache, moves)
    assert all(torch.equal(a, b) for a, b in zip(arrays, want))
    # entries of -1 are skipped; with a count only the first ones are made
    moves.src[3] = moves.dst[3] = -1
    moves.count = i32([7])
    for a, b in zip(arrays, want):
        a.random_(0, 256)
        b.copy_(a)
        for i in (0, 1, 2, 4, 5, 6):
            b[dst[i]] = b[src[i]]
    api.kv_pages_copy(cache, moves)
    assert all(torch.equal(a, b) for a, b in zip(arrays, want))


def test_forked_cache_reads_the_same_and_grows_apart():
    """Append, fork, copy, append different tokens: each sequence reads back its own history."""
    hkv, S = 2, 4
    cache = paged.empty_cache4(24, hkv, 128, 2.0 ** -6, 2.0 ** -6, DEV)
    p = Pair(24, S, 5)
    g = torch.Generator().manual_seed(1)

    def put(counts):
        old = list(p.want.lens)
        p.grow([a + b for a, b in zip(old, counts)])
        cu = np.concatenate([[0], np.cumsum(counts)]).tolist()
        k = torch.randn(cu[-1], hkv, 128, generator=g).bfloat16().to(DEV)
        api.kv4_append_paged(cache, k, -k, i32(cu), i32(old), p.table)

    def text(s):
        n = p.want.lens[s]
        return api.kv4_read_paged(cache, i32([0, n]), i32([0]), p.table[s:s + 1].contiguous(), n)[0]

    put([150, 64, 0, 0])
    first = text(0), text(1)
    api.kv_pages_copy(cache, p.fork([0, 1], [2, 3]))
    assert torch.equal(text(2), first[0]) and torch.equal(text(3), first[1])
    put([1, 1, 1, 1])
    put([40, 3, 90, 7])
    assert torch.equal(text(0)[:150], first[0]) and torch.equal(text(2)[:150], first[0])
    assert not torch.equal(text(0)[150:191], text(2)[150:191])
    before = [text(s) for s in range(S)]
    p.free([1])
    api.kv_pages_copy(cache, p.compact())
    for s in (0, 2, 3):
        assert torch.equal(text(s), before[s])


def test_forked_tails_of_the_8_bit_v_cache():
    """kv_append_paged's incomplete V groups follow a fork."""
    hkv, d = 1, 128
    cache, tail = paged.empty_cache(8, hkv, d, 2.0 ** -6, DEV), paged.empty_tail(3, hkv, d, torch.bfloat16, DEV)
    p = Pair(8, 3, 3)
    k = torch.randn(71, hkv, d, dtype=torch.bfloat16, device=DEV)
    p.grow([70, 0, 0])
    api.kv_append_paged(cache, k[:70], k[:70], i32([0, 70, 70, 70]), i32([0, 0, 0]), p.table, tail, max_new=70)
    moves = p.fork([0], [2])
    api.kv_pages_copy(cache, moves)
    api.kv_tails_copy(tail, moves)
    p.grow([71, 0, 71])
    api.kv_append_paged(cache, torch.cat([k[70:], k[70:]]), torch.cat([k[70:], k[70:]]), i32([0, 1, 1, 2]),
                        i32([70, 0, 70]), p.table, tail, max_new=1)
    assert p.table[0, 1] != p.table[2, 1]
    for a in (cache.k_pages, cache.k_scales, cache.v_pages, cache.v_scales):
        assert torch.equal(a[p.table[0, 1].item()], a[p.table[2, 1].item()])
    assert torch.equal(tail[0], tail[2])


def _state(p):
    return p.pool.refs.clone(), p.table.clone(), p.lens.clone()


@pytest.mark.status_checked
@pytest.mark.parametrize("src,dst", [([0], [1]), ([0], [0]), ([0, 0], [3, 3]), ([0], [7]), ([-1], [3]), ([4], [3]),
                                     ([0, 0, 0, 0], [3, 5, 6, 2])])
def test_refused_forks_change_nothing(src, dst):
    """A destination in use, its own source, given twice, out of range; too few free pages."""
    p = Pair(9, 7, 4)
    p.grow([100, 70, 0, 0, 130, 0, 0])
    tail = torch.zeros(7, 1, 128, 32, dtype=torch.bfloat16, device=DEV).random_(-5, 5)
    if src == [4]:
        p.table[4, 1] = 99                                        # a page that does not exist
    before, kept = _state(p), tail.clone()
    moves = api.kv_pages_fork(p.pool, p.table, p.lens, i32(src), i32(dst))
    api.kv_tails_copy(tail, moves)
    assert api.check_status() == 5
    assert all(torch.equal(a, b) for a, b in zip(_state(p), before))
    assert (moves.src == -1).all() and (moves.dst == -1).all() and (moves.seq_dst == -1).all()
    assert torch.equal(tail, kept)


@pytest.mark.status_checked
@pytest.mark.parametrize("new", [[100, 1000], [99, 64], [100, 257], [2 ** 31 - 1, 2 ** 31 - 1]])
def test_refused_allocations_change_nothing(new):
    p = Pair(5, 2, 4)
    p.grow([100, 64])
    before = _state(p)
    api.kv_pages_alloc(p.pool, p.table, p.lens, i32(new))
    assert api.check_status() == 5
    assert all(torch.equal(a, b) for a, b in zip(_state(p), before))


@pytest.mark.status_checked
def test_frees_named_twice_or_out_of_range():
    p = Pair(12, 4, 4)
    p.grow([100, 64, 10, 0])
    p.want.free([1])
    api.kv_pages_free(p.pool, p.table, p.lens, i32([1, 1, 3, 1]))
    assert api.check_status() == 0
    p.same()
    p.want.free([0])
    p.table[2, 0] = 50
    p.want.lens[2] = 0
    api.kv_pages_free(p.pool, p.table, p.lens, i32([4, 0, -1, 2]))
    assert api.check_status() == 5
    assert p.pool.refs.tolist() == p.want.refs and p.lens.tolist() == p.want.lens


def test_pool_calls_in_a_graph():
    """Fork, copy and free captured once and replayed: the state comes back each time."""
    cache = paged.empty_cache4(30, 2, 128, 1.0, 1.0, DEV)
    cache.k_pages.random_(0, 256)
    p = Pair(30, 6, 4)
    p.grow([130, 200, 64, 0, 0, 0])
    src, dst = i32([0, 1, 1]), i32([3, 4, 5])
    before = _state(p)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        moves = api.kv_pages_fork(p.pool, p.table, p.lens, src, dst)
        api.kv_pages_copy(cache, moves)
        lens = p.lens.clone()
        api.kv_pages_free(p.pool, p.table, p.lens, dst)
    for _ in range(3):
        cache.k_pages.random_(0, 256)
        graph.replay()
        assert lens.tolist() == [130, 200, 64, 130, 200, 200]
        assert torch.equal(cache.k_pages[moves.src.long()], cache.k_pages[moves.dst.long()])
        assert torch.equal(p.pool.refs, before[0]) and torch.equal(p.lens, before[2])
