"""GPU: the ways attention over the 4-bit cache is called (views, plans, graphs, streams), what it does
with rows and pages that are not there, and a run of all of the cache's calls together. Tolerances as
derived in test_gpu_kv4_attention.py; where the same work is done twice the results are equal."""
import math

import pytest
import torch

from bit_block_scaled_nvfp4_b200 import api, paged
from test_gpu_kv4_attention import Case, DEV, KTS, VTS, i32

pytestmark = pytest.mark.gpu
# decoding steps; two tokens; chunks; both kinds
KINDS = {"steps": ([1, 1, 1, 1], [70, 0, 500, 63], 8, 2), "two": ([2, 1, 2], [64, 5, 300], 8, 2),
         "chunks": ([100, 40, 7], [30, 0, 200], 10, 2), "mixed": ([1, 150, 1, 3], [900, 10, 64, 77], 8, 1)}
kinds = pytest.mark.parametrize("kind", list(KINDS))


def case(kind, dtype=torch.bfloat16, **kw):
    return Case(*KINDS[kind], dtype, **kw)


@kinds
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_strided_queries_and_rows_behind_the_last_sequence(kind, dtype):
    c = case(kind, dtype, seed=5)
    out, lse = c.run()
    T, hq = c.q.shape[:2]
    wide = torch.full((T + 5, hq + 3, 128), math.nan, dtype=dtype, device=DEV)      # a slice of a projection, padded
    wide[:T, 2:2 + hq] = c.q
    to = torch.full((T + 5, hq, 128), 7.0, dtype=dtype, device=DEV)
    c.q = wide[:, 2:2 + hq]
    got, lse2 = c.run(out=to)
    assert got is to and torch.equal(got[:T], out) and torch.equal(lse2[:T], lse)
    assert (to[T:] == 7).all()


@kinds
def test_runs_repeat_exactly_and_plans_give_the_same(kind):
    c = case(kind, seed=6)
    out, lse = c.run()
    again, lse2 = c.run(workspace=torch.full((1 << 26,), 255, dtype=torch.uint8, device=DEV))
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    T, hq = c.q.shape[:2]
    plan = api.KV4AttentionPlan(c.cache, c.table, i32(c.ctx), max(c.ctx), hq, max_q=max(c.new), max_tokens=T + 9,
                                dtype=c.dtype, want_lse=True)
    a, b = plan.run(c.q, i32(c.cu))
    assert a.data_ptr() == plan.out.data_ptr() and torch.equal(a, out) and torch.equal(b, lse)
    if max(c.new) == 1:
        a, b = plan.run(c.q)
        assert torch.equal(a, out) and torch.equal(b, lse)
    else:
        with pytest.raises(ValueError):
            plan.run(c.q)
    with pytest.raises(ValueError):
        plan.run(c.q.half())
    with pytest.raises(ValueError):
        plan.run(c.q[:, :-1])
    with pytest.raises(ValueError):
        plan.run(c.q, i32(c.cu)[:-1])
    with pytest.raises(ValueError):
        plan.run(c.q, i32(c.cu).cpu())


@kinds
def test_no_tokens(kind):
    c = case(kind, seed=7)
    S = len(c.new)
    hq, T = c.hq, len(c.q)
    c.q = c.q[:0]
    out, lse = c.run(cu_q=i32([0] * (S + 1)))
    assert out.shape == (0, hq, 128) and lse.shape == (0, hq)
    to = torch.full((T, hq, 128), 7.0, dtype=c.dtype, device=DEV)
    c.q = torch.zeros_like(to)
    c.run(cu_q=i32([0] * (S + 1)), out=to)               # rows, but none of them a sequence's
    assert (to == 7).all()


@kinds
@pytest.mark.parametrize("q_scale,scale", [(1.0, 1.0), (2.0 ** 20, 2.0 ** -24), (2.0 ** -30, 2.0 ** 27), (0.0, 0.1)])
def test_scales_of_queries_and_scores(kind, q_scale, scale):
    c = case(kind, seed=8, q_scale=q_scale)               # (bf16: queries past fp16's range on either side)
    c.check(*c.run(softmax_scale=scale), scale=scale)


@kinds
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_a_row_of_nan_or_infinity_stays_alone(kind, dtype):
    c = case(kind, dtype, seed=9)
    out, lse = c.run()
    bad = torch.zeros(c.q.shape[:2], dtype=torch.bool, device=DEV)
    for i, value in enumerate((math.nan, math.inf, -math.inf)):
        t, h = (i * 37 + 1) % len(c.q), (i * 3 + 1) % c.hq
        c.q[t, h, i * 50] = value
        bad[t, h] = True
    out2, lse2 = c.run()
    assert torch.equal(out[~bad], out2[~bad]) and torch.equal(lse[~bad], lse2[~bad])


@pytest.mark.status_checked
@kinds
@pytest.mark.parametrize("page", [-1, 10 ** 6, -(2 ** 31)])
def test_missing_pages_are_left_out_and_reported(kind, page):
    """As if the sequence's keys were the others alone: page 0 of a sequence with more is taken away."""
    c = case(kind, seed=10)
    s = max(range(len(c.ctx)), key=lambda i: c.ctx[i] - c.new[i])
    assert c.ctx[s] - c.new[s] > 64
    want, want_lse = c.run()
    other = c.table.clone()
    other[s, :-1] = c.table[s, 1:]
    keep = c.ctx[s]
    c.ctx[s] = keep - 64
    c.table, table = other, c.table
    ref, ref_lse = c.run()
    c.ctx[s], c.table = keep, table.clone()
    c.table[s, 0] = page
    assert api.check_status() == 0
    out, lse = c.run()
    assert api.check_status() == 5
    rows = slice(c.cu[s], c.cu[s + 1])
    rest = torch.ones(len(c.q), dtype=torch.bool, device=DEV)
    rest[rows] = False
    assert torch.equal(out[rest], want[rest]) and torch.equal(lse[rest], want_lse[rest])
    # the same keys in other tiles: two roundings of the weights and of the output apart
    a = VTS * 2688
    assert ((out[rows].double() - ref[rows].double()).abs() <= 2 * (2.0 ** -11 + 2.0 ** -12) * a + 2.0 ** -8 * ref[rows].double().abs()).all()
    assert (lse[rows] - ref_lse[rows]).abs().max() < 1e-3
    c.table[s] = page                                     # and with none of its pages: nothing to attend to
    out, lse = c.run()
    assert api.check_status() == 5
    assert (out[rows] == 0).all() and (lse[rows] == -math.inf).all()
    assert torch.equal(out[rest], want[rest]) and torch.equal(lse[rest], want_lse[rest])


@pytest.mark.status_checked
@kinds
@pytest.mark.parametrize("what", ["short", "long", "negative"])
def test_sequences_out_of_range_are_left_out_and_reported(kind, what):
    c = case(kind, seed=11)
    s = 1
    limit = max(c.ctx)
    c.ctx[s] = {"short": c.new[s] - 1, "long": limit + 1, "negative": -5}[what]
    to = torch.full_like(c.q, 7.0)
    api.check_status()
    out, lse = c.run(out=to, max_context=limit)
    assert api.check_status() == 5
    assert (out[c.cu[s]:c.cu[s + 1]] == 7).all()
    c.new[s] = 0                                          # (the others are cut among the SMs in other places)
    c.check(out, lse)


@kinds
def test_graphs_on_other_streams_with_their_own_workspaces(kind):
    """Two captured steps over one cache, replayed at the same time, queries changing between replays."""
    a, b = case(kind, seed=12), case(kind, seed=13)
    cases, jobs = (a, b), []
    for c in cases:
        c.static = c.q.clone()
        ctx, cu = i32(c.ctx), i32(c.cu)
        plan = api.KV4AttentionPlan(c.cache, c.table, ctx, max(c.ctx), c.hq, max_q=max(c.new), max_tokens=len(c.q),
                                    dtype=c.dtype, want_lse=True)
        plan.run(c.static, cu)                            # before the capture: the one-time set-up
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out, lse = plan.run(c.static, cu)
        jobs.append((graph, stream, out, lse, plan, ctx, cu))
    for step in range(4):
        want = []
        for c in cases:
            c.q = torch.randn_like(c.q)
            c.static.copy_(c.q)
            want.append(c.run())
        torch.cuda.synchronize()
        for _ in range(5):
            for graph, stream, *_ in jobs:
                with torch.cuda.stream(stream):
                    graph.replay()
        torch.cuda.synchronize()
        for (o, l), (_, _, out, lse, *_) in zip(want, jobs):
            assert torch.equal(o, out) and torch.equal(l, lse)


@pytest.mark.parametrize("new", [1, 40])
def test_pages_past_32_bit_offsets(new):
    pages, hkv = 140_000, 8                               # K and V 4.6 GB each
    cache = paged.empty_cache4(pages, hkv, 128, KTS, VTS, DEV)
    small = paged.empty_cache4(8, hkv, 128, KTS, VTS, DEV)
    g = torch.Generator(device=DEV).manual_seed(14)
    k, v = torch.randn(2, 200, hkv, 128, generator=g, device=DEV, dtype=torch.bfloat16)
    q = torch.randn(new, 16, 128, generator=g, device=DEV, dtype=torch.bfloat16)
    outs = []
    for c, table in ((cache, [[139_999, 3, 131_072, 70_001]]), (small, [[1, 3, 0, 2]])):
        api.kv4_append_paged(c, k, v, i32([0, 200]), i32([0]), i32(table))
        outs.append(api.attn_kv4_paged(q, c, i32(table), i32([200]), 200, cu_q=i32([0, new]), max_q=new))
    assert torch.equal(outs[0], outs[1])


def test_a_run_of_them_together():
    """Prompts, steps, forks, frees and a compaction, as a server goes through them: every call's attention against
    float64 of the values read back when they were stored, and the cache unchanged by what moves its pages."""
    hq, hkv, S, W, P = 8, 2, 6, 8, 40
    g = torch.Generator(device=DEV).manual_seed(15)
    cache, pool = paged.empty_cache4(P, hkv, 128, KTS, VTS, DEV), paged.empty_pool(P, DEV)
    table, lens = torch.full((S, W), -1, dtype=torch.int32, device=DEV), i32([0] * S)
    hist = [torch.zeros(2, 0, hkv, 128, device=DEV) for _ in range(S)]

    def feed(new):
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        T = cu[-1]
        cu = i32(cu)
        k, v = torch.randn(2, T, hkv, 128, generator=g, device=DEV, dtype=torch.bfloat16)
        q = torch.randn(T, hq, 128, generator=g, device=DEV, dtype=torch.bfloat16)
        after = lens + i32(new)
        api.kv_pages_alloc(pool, table, lens, after)
        api.kv4_append_paged(cache, k, v, cu, lens, table)
        rk, rv = api.kv4_read_paged(cache, cu, lens, table, T, dtype=torch.float32)
        at = 0
        for s, n in enumerate(new):
            hist[s] = torch.cat([hist[s], torch.stack([rk[at:at + n], rv[at:at + n]])], 1)
            at += n
        lens.copy_(after)
        out, lse = api.attn_kv4_paged(q, cache, table, lens, W * 64, cu_q=cu, max_q=max(new), want_lse=True)
        c = Case.__new__(Case)
        c.new, c.ctx, c.hq, c.hkv, c.dtype, c.q = new, lens.tolist(), hq, hkv, q.dtype, q
        c.cu, c.values = cu.tolist(), lambda s: (hist[s][0].double(), hist[s][1].double())
        assert c.ctx == [h.shape[1] for h in hist]
        c.check(out, lse)

    def same():
        for s, h in enumerate(hist):
            n = h.shape[1]
            if n:
                k, v = api.kv4_read_paged(cache, i32([0, n]), i32([0]), table[s:s + 1].contiguous(), n, dtype=torch.float32)
                assert torch.equal(torch.stack([k, v]), h)

    feed([130, 64, 0, 33, 0, 0])                          # prompts
    feed([1, 1, 0, 1, 0, 0])                              # a step
    api.kv_pages_copy(cache, api.kv_pages_fork(pool, table, lens, i32([0, 0, 3]), i32([2, 4, 5])))
    for s, d in ((0, 2), (0, 4), (3, 5)):
        hist[d] = hist[s]
    same()
    feed([1] * S)                                         # the forks grow apart
    feed([2, 1, 70, 0, 1, 3])
    same()
    api.kv_pages_free(pool, table, lens, i32([0, 3]))
    hist[0], hist[3] = hist[0][:, :0], hist[3][:, :0]
    api.kv_pages_copy(cache, api.kv_pages_compact(pool, table, lens))
    live = int((pool.refs > 0).sum())
    assert (pool.refs[:live] > 0).all() and (pool.refs[live:] == 0).all()
    same()
    feed([90, 1, 1, 0, 1, 1])                             # a new prompt beside the steps
    same()
