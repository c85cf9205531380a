"""What the serving operators promise beyond their sums: empty batches, buffers that overlap, capture into graphs,
contexts with long pages, and a serving step checked stage by stage."""
import pytest
import torch

import dynamic_depth_b200 as T
from test_gpu_operators import F16

pytestmark = pytest.mark.gpu


def test_an_empty_batch_goes_through_every_operator():
    """A step in which no request has a new token: outputs of no rows, the cache as it was."""
    i32 = dict(dtype=torch.int32, device="cuda")
    pool = torch.ones(4, 2, 2, 16, 64, dtype=F16, device="cuda")
    table = torch.zeros(2, 3, **i32)
    lens, fresh, head = torch.tensor([3, 0], **i32), torch.zeros(2, **i32), torch.zeros(1, **i32)
    for words in (0, 1):
        plan = T.plan_batch(lens, fresh, table, torch.arange(4, **i32), head, 16, 0,
                            parents=torch.zeros(0, **i32) if words else None, mask_words=words)
        assert plan.cu.tolist() == [0, 0, 0] and plan.lens.tolist() == [3, 0] and plan.free_head.tolist() == [0]
        q = T.norm_rope_append(torch.zeros(0, 8 * 64, dtype=F16, device="cuda"), 4, pool, plan.slots, plan.positions,
                               T.rope_table(8, 64))
        out, lse = T.tree_attention(q, pool, table, lens, plan.cu, 4, masks=plan.masks, return_lse=True)
        assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
        lp = T.token_logprobs(out.reshape(0, 256), torch.zeros(0, **i32), n_top=3)
        assert lp.top_ids.shape == (0, 3) and lp.logprob.shape == (0,)
    assert bool((pool == 1).all())
