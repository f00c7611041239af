"""GPU attention over the 4-bit cache against a plain float64 softmax of the cached values.

Tolerance, element by element, from the arithmetic: with w the weights, A = sum_j w_j |v_j| and
B = max_j scale * sum_c |q_c k_jc| of the row,
  * the weights are rounded to fp16, half a step of 2^-10: at most 2^-11 A; as P = 2^(s - m + 6) with m at
    most the row's maximum, its largest is at least 2^6, and one below 2^-14 is rounded to half a step
    of 2^-24: 2^-31 of the largest weight at most, each: 2^-31 max w sum_j |v_j|;
  * a score is 128 products summed in float32 by the tensor cores and scaled: at most
    136 * 2^-23 B off, numerator and denominator each: 2 * 136 * 2^-23 B A;
  * exponentials (2 ulp), sums, rescaling and the splits' joining: within 2^-18 A;
  * the output rounding: half a step of its type, relative to the value.
lse: the scores' error, 2^-18, and float32 rounding of the result (2^-22 |lse|)."""
import math

import numpy as np
import pytest
import torch

from bit_block_scaled_nvfp4_b200 import api, paged
from oracle import kv4 as OK
from helpers import f32

pytestmark = pytest.mark.gpu
DEV = "cuda"
KTS, VTS = 2.0 ** -5, 2.0 ** -7


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Case:
    """Sequences with `past` tokens cached before their new ones, all appended to a shuffled cache."""

    def __init__(self, new, past, hq, hkv, dtype, seed=0, q_scale=1.0, spare=3):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.new, self.ctx = list(new), [n + p for n, p in zip(new, past)]
        self.hq, self.hkv, self.dtype = hq, hkv, dtype
        S = len(new)
        need = [(c + 63) // 64 for c in self.ctx]
        pages = sum(need) + spare
        ids = torch.randperm(pages, generator=g, device=DEV).int()
        self.table = torch.full((S, max(need) + 1), -1, dtype=torch.int32, device=DEV)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = ids[at:at + n]
            at += n
        self.cache = paged.empty_cache4(pages, hkv, 128, KTS, VTS, DEV)
        # stale contents: every code, and NaN scales, in the slots behind each context
        for t in (self.cache.k_pages, self.cache.v_pages):
            t.random_(0, 256, generator=g)
        self.cache.k_scales.fill_(0x7F)
        self.cache.v_scales.fill_(0x7F)
        cu = np.concatenate([[0], np.cumsum(self.ctx)]).tolist()
        shape = torch.ones(1, hkv, 128, device=DEV)
        shape[..., ::31] = 8.0
        k = ((torch.randn(cu[-1], hkv, 128, generator=g, device=DEV) + 0.3) * shape).to(dtype)
        v = torch.randn(cu[-1], hkv, 128, generator=g, device=DEV).to(dtype)
        api.kv4_append_paged(self.cache, k, v, i32(cu), i32([0] * S), self.table)
        self.cu = np.concatenate([[0], np.cumsum(new)]).tolist()
        self.q = (torch.randn(self.cu[-1], hq, 128, generator=g, device=DEV) * q_scale).to(dtype)

    def run(self, **kw):
        kw.setdefault("max_q", max(max(self.new), 1))
        kw.setdefault("want_lse", True)
        kw.setdefault("cu_q", i32(self.cu))
        kw.setdefault("max_context", max(max(self.ctx), 1))
        return api.attn_kv4_paged(self.q, self.cache, self.table, i32(self.ctx), **kw)

    def values(self, s):
        n = self.ctx[s]
        k, v = api.kv4_read_paged(self.cache, i32([0, n]), i32([0]), self.table[s:s + 1].contiguous(), n, dtype=torch.float32)
        return k.double(), v.double()

    def check(self, out, lse, scale=1 / math.sqrt(128)):
        eps = torch.finfo(self.dtype).eps / 2
        for s, (n, ctx) in enumerate(zip(self.new, self.ctx)):
            if n == 0:
                continue
            k, v = self.values(s)
            seen = torch.arange(ctx, device=DEV) <= torch.arange(ctx - n, ctx, device=DEV).unsqueeze(1)
            g = self.hq // self.hkv
            for h in range(self.hq):
                q = self.q[self.cu[s]:self.cu[s + 1], h].double()
                kh, vh = k[:, h // g], v[:, h // g]
                x = ((q @ kh.T) * scale).masked_fill(~seen, -math.inf)
                ref_lse = torch.logsumexp(x, -1)
                w = torch.exp(x - ref_lse.unsqueeze(-1))
                ref, a = w @ vh, w @ vh.abs()
                b = ((q.abs() @ kh.abs().T) * scale).masked_fill(~seen, 0).amax(-1, keepdim=True)
                tol = eps * ref.abs() + (2.0 ** -11 + 2 * 136 * 2.0 ** -23 * b + 2.0 ** -18) * a
                tol += 2.0 ** -31 * w.amax(-1, keepdim=True) * (seen.double() @ vh.abs())
                got = out[self.cu[s]:self.cu[s + 1], h].double()
                d = (got - ref).abs()
                assert (d <= tol).all(), f"seq {s} head {h}: {float((d / tol).max()):.2f} of the tolerance at {int((d / tol).argmax())}"
                if lse is not None:
                    d = (lse[self.cu[s]:self.cu[s + 1], h].double() - ref_lse).abs()
                    assert (d <= 136 * 2.0 ** -23 * b[:, 0] + 2.0 ** -18 + 2.0 ** -22 * ref_lse.abs()).all(), f"lse {float(d.max())}"


DTYPES = [torch.bfloat16, torch.float16]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hq,hkv", [(8, 2), (1, 1), (3, 3), (32, 8), (6, 2), (7, 1), (16, 1), (20, 2), (48, 3)])
def test_one_token_a_sequence(dtype, hq, hkv):
    c = Case([1] * 9, [0, 1, 62, 63, 64, 127, 300, 1000, 777], hq, hkv, dtype, seed=hq)
    out, lse = c.run()
    c.check(out, lse)
    again, lse2 = c.run(cu_q=None)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hq,hkv,new", [(4, 4, [1, 0, 3, 8, 2, 5]), (8, 2, [2, 4, 0, 1]), (8, 1, [4, 1, 3]), (32, 2, [2, 1, 0, 2]), (5, 1, [6, 2])])
def test_a_few_tokens_a_sequence(dtype, hq, hkv, new):
    c = Case(new, [0, 5, 61, 500, 64, 1300][:len(new)], hq, hkv, dtype, seed=len(new))
    c.check(*c.run())


def test_one_long_sequence_over_all_of_the_device():
    c = Case([1], [40000], 8, 2, torch.bfloat16)
    c.check(*c.run())
    c = Case([2], [9000], 32, 8, torch.float16)
    c.check(*c.run())


def test_more_sequences_than_a_block_counts_at_once():
    g = torch.Generator().manual_seed(4)
    past = torch.randint(0, 200, (700,), generator=g).tolist()
    c = Case([0 if i % 7 == 3 else 1 for i in range(700)], past, 2, 1, torch.bfloat16)
    out, lse = c.run(max_q=1)
    c.check(out, lse)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hq,hkv,new,past", [
    (1, 1, [200], [0]), (4, 1, [128], [0]), (2, 2, [129, 33], [0, 0]), (8, 2, [300], [1000]),
    (6, 2, [130, 77, 1], [5, 700, 64]), (7, 1, [90, 0, 40], [63, 9, 1]), (16, 1, [70, 5], [129, 2]),
    (5, 1, [257, 51, 52], [0, 31, 128]), (26, 2, [41, 200], [333, 0])])
def test_prompts_and_chunks(dtype, hq, hkv, new, past):
    c = Case(new, past, hq, hkv, dtype, seed=len(new) + hq)
    c.check(*c.run())


def test_a_long_prompt():
    c = Case([3000], [0], 8, 2, torch.bfloat16)
    c.check(*c.run())


def test_a_chunk_far_into_a_long_context():
    c = Case([100], [20000], 8, 2, torch.float16)
    c.check(*c.run())


def test_steps_and_chunks_together():
    c = Case([1, 150, 1, 0, 1, 2, 90, 1], [700, 100, 64, 5, 2000, 0, 0, 127], 16, 4, torch.bfloat16)
    c.check(*c.run())
