"""GPU parity of the 4-bit cache's appends and reads against the oracle: codes and scales bit for
bit, values as code * scale * tensor scale rounded once; nothing but the appended tokens' codes
and scales is written."""
import numpy as np
import pytest
import torch

from bit_block_scaled_nvfp4_b200 import api, paged
from oracle import kv4 as OK
from helpers import f32

pytestmark = pytest.mark.gpu
DEV = "cuda"
KTS, VTS = 2.0 ** -6 * 1.37, 2.0 ** -7 * 1.11


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _pair(seed, pages, hkv, fill=None):
    """A cache on the GPU and the oracle's; `fill`: random bytes beforehand."""
    cache = paged.empty_cache4(pages, hkv, 128, KTS, VTS, DEV)
    want = OK.Cache(pages, hkv, 128, KTS, VTS)
    if fill:
        g = torch.Generator().manual_seed(seed)
        for t, w in ((cache.k_pages, want.kp), (cache.k_scales, want.ks), (cache.v_pages, want.vp), (cache.v_scales, want.vs)):
            b = torch.randint(0, 256, t.shape, generator=g, dtype=torch.uint8)
            t.copy_(b)
            w[:] = b.numpy()
    return cache, want


def _same(cache, want):
    for name, t, w in (("K codes", cache.k_pages, want.kp), ("K scales", cache.k_scales, want.ks),
                       ("V codes", cache.v_pages, want.vp), ("V scales", cache.v_scales, want.vs)):
        t = t.cpu().numpy()
        assert np.array_equal(t, w), f"{name} differ at {np.argwhere(t != w)[:4].tolist()}"


def _tokens(g, n, hkv, dtype):
    k = torch.randn(n, hkv, 128, generator=g) * torch.exp2(torch.randint(-6, 4, (n, hkv, 1), generator=g).float())
    v = torch.randn(n, hkv, 128, generator=g)
    v[torch.rand(n, generator=g) < 0.05] = 0.0                 # all-zero blocks
    return k.to(dtype), v.to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("hkv,plan", [
    (2, [[1, 1, 1]] * 4 + [[63, 64, 65], [0, 2, 0], [130, 1, 61]]),
    (1, [[1]] * 3 + [[200]]),
    (5, [[0, 0, 7, 0], [1, 0, 0, 1], [0, 70, 1, 0]]),
    (8, [[300, 0, 129], [1, 1, 1]])])
def test_append_and_read_match_the_oracle(dtype, hkv, plan):
    g = torch.Generator().manual_seed(hkv)
    S = len(plan[0])
    total = [sum(c[s] for c in plan) for s in range(S)]
    width = max((n + 63) // 64 for n in total) + 1
    pages = S * width + 2
    perm = torch.randperm(pages, generator=g)[:S * width].view(S, width).int()
    cache, want = _pair(3, pages, hkv, fill=True)
    lens = [0] * S
    for call in plan:
        n = sum(call)
        k, v = _tokens(g, n, hkv, dtype)
        cu = np.concatenate([[0], np.cumsum(call)]).tolist()
        api.kv4_append_paged(cache, k.to(DEV), v.to(DEV), i32(cu), i32(lens), perm.to(DEV))
        for s in range(S):
            want.append(f32(k[cu[s]:cu[s + 1]]), f32(v[cu[s]:cu[s + 1]]), lens[s], perm[s].tolist())
        _same(cache, want)
        for out in (dtype, torch.float32):
            kr, vr = api.kv4_read_paged(cache, i32(cu), i32(lens), perm.to(DEV), n, dtype=out)
            for s in range(S):
                ko, vo = want.read(call[s], perm[s].tolist(), lens[s])
                for got, ref in ((kr, ko), (vr, vo)):
                    # the tensor scale's product rounded to float32, then once to the type
                    ref = torch.from_numpy(ref.astype(np.float32)).to(out)
                    assert torch.equal(got[cu[s]:cu[s + 1]].cpu(), ref)
        lens = [a + b for a, b in zip(lens, call)]


def test_strided_tokens_and_rows_behind_the_last_sequence():
    g = torch.Generator().manual_seed(5)
    hkv, T = 3, 90
    wide = torch.randn(T, 2 * hkv * 128 + 200, generator=g).bfloat16().to(DEV)
    k = wide[:, 8:8 + hkv * 128].view(T, hkv, 128)
    v = wide[:, 200 + hkv * 128:].view(T, hkv, 128)
    assert not k.is_contiguous()
    row = [4, 2]
    cache, want = _pair(9, 5, hkv, fill=True)
    cu, lens, table = i32([0, 71]), i32([13]), i32([row])        # rows 71.. belong to nobody
    api.kv4_append_paged(cache, k, v, cu, lens, table)
    want.append(f32(k[:71]), f32(v[:71]), 13, row)
    _same(cache, want)
    out = torch.full((2, T, hkv * 128 + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    ko, vo = (o[:, :hkv * 128].view(T, hkv, 128) for o in out)
    api.kv4_read_paged(cache, cu, lens, table, T, out=(ko, vo))
    a, b = api.kv4_read_paged(cache, cu, lens, table, 71)
    assert torch.equal(ko[:71], a) and torch.equal(vo[:71], b)
    assert (out[:, 71:] == 7).all() and (out[:, :, hkv * 128:] == 7).all()


def test_values_past_the_scale_and_special_values():
    """Saturation, subnormal blocks and signed zeros, as the quantizer itself encodes them."""
    x = torch.zeros(6, 1, 128)
    x[0] = torch.linspace(-60000, 60000, 128)
    x[1] = torch.linspace(-1e-7, 1e-7, 128)
    x[2, 0, ::2] = -0.0
    x[3, 0, 0] = 2688 * KTS
    x[4] = torch.linspace(-3, 3, 128)
    x[5, 0, 5] = 6e-8
    x = x.half()
    cache, want = _pair(0, 2, 1)
    api.kv4_append_paged(cache, x.to(DEV), x.to(DEV), i32([0, 6]), i32([63]), i32([[1, 0]]))
    want.append(f32(x), f32(x), 63, [1, 0])
    _same(cache, want)


def test_no_tokens_is_no_work():
    cache, want = _pair(1, 3, 2, fill=True)
    e = torch.empty(0, 2, 128, dtype=torch.bfloat16, device=DEV)
    api.kv4_append_paged(cache, e, e, i32([0, 0, 0]), i32([5, 0]), i32([[0], [1]]))
    k, v = api.kv4_read_paged(cache, i32([0, 0, 0]), i32([5, 0]), i32([[0], [1]]), 0)
    assert k.shape == v.shape == (0, 2, 128)
    _same(cache, want)


def test_many_sequences_and_a_page_past_32_bit_offsets():
    """More sequences than a CTA counts at once; pages whose byte offset is past 2^32."""
    S, hkv = 700, 8
    g = torch.Generator().manual_seed(2)
    pages = (1 << 32) // (hkv * 4096) + S + 10
    cache = paged.empty_cache4(pages, hkv, 128, KTS, VTS, DEV)
    counts = torch.randint(0, 4, (S,), generator=g).tolist()
    cu = np.concatenate([[0], np.cumsum(counts)]).tolist()
    k, v = _tokens(g, cu[-1], hkv, torch.bfloat16)
    lens = torch.randint(0, 60, (S,), generator=g)
    table = (pages - 1 - torch.randperm(S, generator=g)).int().view(S, 1)
    api.kv4_append_paged(cache, k.to(DEV), v.to(DEV), i32(cu), lens.int().to(DEV), table.to(DEV))
    kr, vr = api.kv4_read_paged(cache, i32(cu), lens.int().to(DEV), table.to(DEV), cu[-1], dtype=torch.float32)
    small = OK.Cache(1, hkv, 128, KTS, VTS)
    for s in range(0, S, 37):
        small.append(f32(k[cu[s]:cu[s + 1]]), f32(v[cu[s]:cu[s + 1]]), int(lens[s]), [0])
        a, b = small.read(counts[s], [0], int(lens[s]))
        assert np.array_equal(f32(kr[cu[s]:cu[s + 1]]), a.astype(np.float32))
        assert np.array_equal(f32(vr[cu[s]:cu[s + 1]]), b.astype(np.float32))
    assert not cache.k_pages[:pages - S].any()


@pytest.mark.status_checked
@pytest.mark.parametrize("start,table,written", [
    ([0], [[0, 9]], 64), ([0], [[0, -1]], 64), ([100], [[0, 1]], 28), ([-3], [[0, 1]], 0),
    ([2 ** 31 - 20], [[0, 1]], 0)])
def test_places_out_of_range_are_reported_and_skipped(start, table, written):
    cache, _ = _pair(0, 4, 1)
    k = torch.ones(100, 1, 128, dtype=torch.bfloat16, device=DEV)
    api.kv4_append_paged(cache, k, k, i32([0, 100]), i32(start), i32(table))
    assert api.check_status() == 5
    assert int((cache.k_scales != 0).all(-1).sum()) == written
    out = torch.full((2, 100, 1, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    api.kv4_read_paged(cache, i32([0, 100]), i32(start), i32(table), 100, out=(out[0], out[1]))
    assert api.check_status() == 5
    assert int((out[0] != 7).all(-1).sum()) == written


def test_append_and_read_in_a_graph_on_another_stream():
    g = torch.Generator().manual_seed(8)
    cache, want = _pair(0, 8, 2)
    k, v = _tokens(g, 3, 2, torch.float16)
    kd, vd, lens = k.to(DEV), v.to(DEV), i32([60, 0, 5])
    cu, table = i32([0, 1, 2, 3]), i32([[0, 1], [2, 3], [4, 5]])
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        api.kv4_append_paged(cache, kd, vd, cu, lens, table)
        kr, vr = api.kv4_read_paged(cache, cu, lens, table, 3, dtype=torch.float32)
        lens += 1
    for step in range(6):                                       # across a page boundary
        k, v = _tokens(g, 3, 2, torch.float16)
        kd.copy_(k)
        vd.copy_(v)
        graph.replay()
        for s, n in enumerate((60, 0, 5)):
            row = table[s].tolist()
            want.append(f32(k[s:s + 1]), f32(v[s:s + 1]), n + step, row)
            a, b = want.read(1, row, n + step)
            assert np.array_equal(f32(kr[s:s + 1]), a.astype(np.float32))
            assert np.array_equal(f32(vr[s:s + 1]), b.astype(np.float32))
    _same(cache, want)
