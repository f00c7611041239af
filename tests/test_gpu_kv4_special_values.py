"""GPU: attention over the 4-bit cache where a cached value is NaN, and where scores vanish. A query's output is a
function of the keys it sees alone, so a NaN behind them changes no bit of it; where it sees the NaN the formula says
which outputs are NaN: those of a V block's 16 channels, or all of a row's for a key. Scores: tolerances as derived in
test_gpu_kv4_attention.py."""
import math

import pytest
import torch

from test_gpu_kv4_attention import Case, DEV

pytestmark = pytest.mark.gpu
# few rows a KV head, of several tokens; many, within a CTA and cut among several; both kinds in one call
KINDS = {"steps": ([1, 1, 1], [70, 0, 500], 8, 2), "few": ([4, 1, 3], [61, 5, 700], 4, 1),
         "few, two tiles": ([2, 2, 1], [62, 3000, 9], 16, 2), "chunks": ([100, 40, 7], [30, 0, 200], 10, 2),
         "long chunk": ([300], [2000], 8, 2), "mixed": ([1, 150, 1, 3], [900, 10, 64, 77], 8, 1)}
kinds = pytest.mark.parametrize("kind", list(KINDS))
NAN = (0x7F, 0xFF)                                        # E4M3's two NaN codes


def place(c, s, pos):
    return int(c.table[s, pos // 64]), pos % 64


def seen_by(c, s, pos):
    """Which rows of q see position `pos` of sequence s."""
    rows = torch.zeros(len(c.q), dtype=torch.bool, device=DEV)
    n = c.new[s]
    rows[c.cu[s] + max(0, pos - (c.ctx[s] - n)):c.cu[s + 1]] = True
    return rows


def positions(c):
    """Of each sequence: its last token, one in the middle of the new ones, the last cached one."""
    for s, (n, ctx) in enumerate(zip(c.new, c.ctx)):
        yield from {(s, ctx - 1), (s, ctx - 1 - n // 2), (s, max(0, ctx - n - 1))}


@kinds
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_a_nan_value_reaches_the_queries_that_see_it_and_no_others(kind, dtype):
    c = Case(*KINDS[kind], dtype, seed=21)
    out, lse = c.run()
    g = c.hq // c.hkv
    for i, (s, pos) in enumerate(sorted(positions(c))):
        page, slot = place(c, s, pos)
        h, blocks = i % c.hkv, [i % 8, (3 * i + 5) % 8]
        kept = c.cache.v_scales.clone()
        for k, b in enumerate(blocks):
            c.cache.v_scales[page, h, b, slot] = NAN[(i + k) % 2]
        if pos + 1 < c.ctx[s]:                            # a second one behind it changes nothing
            page, slot = place(c, s, pos + 1)
            c.cache.v_scales[page, h, blocks[0], slot] = NAN[0]
        got, got_lse = c.run()
        c.cache.v_scales.copy_(kept)
        want = out.clone()
        for b in blocks:
            want[seen_by(c, s, pos), h * g:(h + 1) * g, 16 * b:16 * b + 16] = math.nan
        assert torch.equal(got.isnan(), want.isnan()), (s, pos)
        assert torch.equal(got.nan_to_num(), want.nan_to_num()) and torch.equal(got_lse, lse), (s, pos)


@kinds
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_a_nan_key_reaches_the_queries_that_see_it_and_no_others(kind, dtype):
    c = Case(*KINDS[kind], dtype, seed=22)
    out, lse = c.run()
    g = c.hq // c.hkv
    for i, (s, pos) in enumerate(sorted(positions(c))):
        page, slot = place(c, s, pos)
        h = i % c.hkv
        kept = c.cache.k_scales.clone()
        c.cache.k_scales[page, h, slot, i % 8] = NAN[i % 2]
        got, got_lse = c.run()
        c.cache.k_scales.copy_(kept)
        bad = torch.zeros(c.q.shape[:2], dtype=torch.bool, device=DEV)
        bad[seen_by(c, s, pos), h * g:(h + 1) * g] = True
        assert got[bad].isnan().all() and got_lse[bad].isnan().all(), (s, pos)
        assert torch.equal(got[~bad], out[~bad]) and torch.equal(got_lse[~bad], lse[~bad]), (s, pos)


@kinds
@pytest.mark.parametrize("dtype,q_scale,scale", [(torch.bfloat16, 2.0 ** -120, 2.0 ** -24), (torch.bfloat16, 1.0, 2.0 ** -146),
                                                 (torch.float16, 1.0, 2.0 ** -146)])
def test_scores_too_small_for_float32_are_zero(kind, dtype, q_scale, scale):
    """The factor from products to scores leaves float32's range at the bottom: every key that a row sees has
    the same weight, the others none."""
    c = Case(*KINDS[kind], dtype, seed=23, q_scale=q_scale)
    c.check(*c.run(softmax_scale=scale), scale=scale)
