"""GPU attention over the 4-bit cache in the cuts of its work: more sequences than a CTA counts at once in both
kernels, and bounds on the tokens a sequence far above what it has. Tolerances as derived in
test_gpu_kv4_attention.py."""
import pytest
import torch

from bit_block_scaled_nvfp4_b200 import api
from test_gpu_kv4_attention import Case, i32

pytestmark = pytest.mark.gpu


def test_more_sequences_than_a_block_counts_at_once_in_both_kernels():
    """One token each for the kernel of few rows, 3 and 17 of 8 heads for the other, none at all."""
    g = torch.Generator().manual_seed(6)
    past = torch.randint(0, 200, (1100,), generator=g).tolist()
    new = [(0, 1, 3, 17, 1, 3)[i % 6] for i in range(1100)]
    c = Case(new, past, 8, 1, torch.bfloat16, seed=31)
    out, lse = c.run()
    again, lse2 = c.run()
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    c.check(out, lse)


@pytest.mark.parametrize("max_q", [2, 40, 5000])
@pytest.mark.parametrize("new,past,hq,hkv", [([1], [900], 8, 2), ([1], [0], 3, 3), ([2], [70], 16, 1), ([1, 2, 1, 0], [500, 64, 0, 9], 32, 2),
                                             ([1, 1, 1], [63, 2000, 130], 8, 1)])
def test_a_plan_for_more_tokens_than_there_are(new, past, hq, hkv, max_q):
    c = Case(new, past, hq, hkv, torch.float16, seed=32)
    c.check(*c.run(max_q=max_q))
    plan = api.KV4AttentionPlan(c.cache, c.table, i32(c.ctx), c.table.shape[1] * 64, hq, max_q=max_q, max_tokens=len(c.q),
                                dtype=c.dtype, want_lse=True)
    c.check(*plan.run(c.q, i32(c.cu)))
