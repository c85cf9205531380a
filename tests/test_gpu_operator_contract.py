"""What the serving operators promise beyond their sums: empty batches, buffers that overlap, capture into graphs,
contexts with long pages, and a serving step checked stage by stage."""
import math

import numpy as np
import pytest
import torch

import dynamic_depth_b200 as T
import operator_refs as R
import synthetic as S
from gpu_helpers import gpu_model, oracle_weights, status_clean
from oracle import decode as D
from test_gpu_operators import BF16, F16, gen, random_tree, run_tree, tree_case
from test_gpu_speculate_tree import nodes_of, stop_at

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


@pytest.mark.parametrize("page", [4096, 8192, 1 << 15])
def test_tree_speculation_on_a_context_with_long_pages(page):
    W, widths, n_new = oracle_weights("tiny"), [2, 2], 7
    P = S.prompts(1, 11, 512, seed=141)[0]
    m = gpu_model("tiny", None, max_lanes=nodes_of(widths), max_seq=32, L_max=3, max_prefill_tokens=16,
                  kv_page_tokens=page)
    plain = D.generate_lane(W, P, 3, n_new)
    stop = stop_at(plain)
    assert stop > 1
    m.prefill(0, P, 3)
    chain, _ = m.speculate(0, n_new, 1, 3, 2)
    assert chain[:stop].tolist() == plain.tokens[:stop].tolist()
    m.prefill(0, P, 3)
    tok, _ = m.speculate_tree(0, n_new, 1, 3, widths)
    status_clean(m)
    assert tok[:stop].tolist() == plain.tokens[:stop].tolist()


def test_tree_speculation_across_position_4096():
    """Prompts that end before and behind the end of a planning page, nodes on both sides of it; the tokens are those of
    a chain of drafts."""
    n_new, widths = 10, [2, 2]
    m = gpu_model("tiny", None, max_lanes=nodes_of(widths), max_seq=4096 + 64, L_max=2, max_prefill_tokens=4200)
    for T_ in (4089, 4096, 4099):
        P = S.prompts(1, T_, 512, seed=143)[0]
        m.prefill(0, P, 2)
        chain, _ = m.speculate(0, n_new, 1, 2, 2)
        m.prefill(0, P, 2)
        tok, _ = m.speculate_tree(0, n_new, 1, 2, widths)
        status_clean(m)
        assert tok.tolist() == chain.tolist()


@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("nodes", [3, 12, 70])
def test_outputs_in_the_queries_own_place(hd, nodes):
    """dev_out may be dev_q: whole row blocks, and blocks cut over several CTAs."""
    c = tree_case([2500, 40, 0, 700], [nodes, 2, nodes, 1], 8, 2, hd, BF16, 32, seed=hd + nodes)
    want, wl, _ = run_tree(c)
    o, lse, st = run_tree(c, out=c["q"])
    assert st == 0 and o.data_ptr() == c["q"].data_ptr()
    assert torch.equal(o, want) and torch.equal(lse, wl)


def test_queries_and_outputs_side_by_side_in_one_buffer():
    c = tree_case([300, 9], [5, 8], 4, 2, 64, F16, 16, seed=20)
    want, _, _ = run_tree(c)
    wide = torch.zeros(13, 2, 4, 64, dtype=F16, device="cuda")
    wide[:, 0] = c["q"]
    c["q"] = wide[:, 0]
    assert torch.equal(run_tree(c, out=wide[:, 1])[0], want)


@pytest.mark.parametrize("rows,vocab", [(1300, 9000), (4000, 16000)])
def test_the_cost_of_many_best_tokens_has_no_step(rows, vocab):
    """Ordinary (normal) rows: 64 best tokens cost a few times what 40 do, not a pass over the row for each of them."""
    x = (torch.randn(rows, vocab, generator=gen(vocab), device="cuda") * 3).bfloat16()
    cost = {}
    for n in (40, 57, 60, 64):
        T.token_logprobs(x, n_top=n)
        best = math.inf
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            o = T.token_logprobs(x, n_top=n)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        cost[n] = best
        assert torch.equal(o.top_logprobs, o.top_logprobs.sort(1, descending=True).values)
    assert max(cost.values()) < 8 * cost[40], cost


def test_a_serving_step_checked_stage_by_stage():
    """Plan, append, attention and log probabilities of a prompt, a tree of drafts and a block of single tokens, captured
    in one graph a step; each stage is checked on what the one before it left, so its bound is its own rounding alone."""
    g, rng = gen(30), np.random.default_rng(30)
    H, Hk, hd, page, n_pages, base, V = 8, 2, 64, 16, 64, 1e4, 999
    i32 = dict(dtype=torch.int32, device="cuda")
    n64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    pool = torch.zeros(n_pages, 2, Hk, page, hd, dtype=BF16, device="cuda")
    table = torch.full((3, 12), -1, **i32)
    free = torch.from_numpy(rng.permutation(n_pages).astype(np.int32)).cuda()
    head, lens = torch.zeros(1, **i32), torch.zeros(3, **i32)
    rope = T.rope_table(256, hd, base)
    gq, gk = (1 + 0.1 * torch.randn(hd, generator=g, device="cuda") for _ in range(2))
    w = torch.randn(H * hd, V, generator=g, device="cuda") / 20
    half, fp = R.HALF_STEP[BF16], (hd / 16 + 12) * 2.0 ** -24
    for fresh, tree in (([40, 7, 90], False), ([9, 1, 14], True), ([1, 1, 1], False)):
        total = sum(fresh)
        parents = sum((random_tree(rng, f) for f in fresh), []) if tree else None
        x = torch.randn(total, (H + 2 * Hk) * hd, generator=g, device="cuda").to(BF16)
        ins = (lens.clone(), torch.tensor(fresh, **i32), head.clone(), torch.tensor(parents, **i32) if tree else None,
               torch.zeros(total, **i32))
        np_table, ctx, old_head = table.cpu().numpy(), lens.tolist(), int(head)
        before = pool.clone()

        def step():
            plan = T.plan_batch(ins[0], ins[1], table, free, ins[2], page, total, parents=ins[3],
                                mask_words=1 if tree else 0)
            q = T.norm_rope_append(x, H, pool, plan.slots, plan.positions, rope, q_gain=gq, k_gain=gk)
            out, lse = T.tree_attention(q, pool, table, ins[0], plan.cu, max(fresh), masks=plan.masks, return_lse=True)
            logits = (out.reshape(total, -1).float() @ w).contiguous()
            return plan, q, out, lse, logits, T.token_logprobs(logits, ins[4], n_top=3)
        torch.mm(torch.zeros(2, 2, device="cuda"), torch.zeros(2, 2, device="cuda"))  # the library's handle, before capture
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            plan, q, out, lse, logits, lp = step()
        assert torch.equal(pool, before)  # captured, not run
        graph.replay()
        torch.cuda.synchronize()
        # the plan, exactly
        want = R.plan(ctx, fresh, np_table, free.cpu().numpy(), old_head, page, parents, 1 if tree else 0)
        assert np.array_equal(table.cpu().numpy(), np_table) and plan.slots.tolist() == want["slots"]
        assert plan.positions.tolist() == want["positions"] and plan.lens.tolist() == want["lens"]
        # norm, rotation and append
        wq, wk, wv, sq, sk = R.norm_rope(n64(x), H, Hk, hd, np.array(want["positions"]), base, n64(gq), n64(gk))
        flat = n64(pool.permute(0, 3, 1, 2, 4).reshape(-1, 2, Hk, hd)[plan.slots])
        assert (np.abs(n64(q) - wq) <= half * np.abs(wq) + fp * sq).all()
        assert (np.abs(flat[:, 0] - wk) <= half * np.abs(wk) + fp * sk).all() and np.array_equal(flat[:, 1], wv)
        # attention, on the queries and the cache as they are, masks from the parents by hand
        see = None
        if tree:
            see = np.zeros((total, 32), bool)
            for r in range(3):
                for j in range(fresh[r]):
                    row = want["cu"][r] + j
                    if parents[row] >= 0:
                        see[row] = see[want["cu"][r] + parents[row]]
                    see[row, j] = True
        wo, wl, tol, ltol = R.tree_attention(n64(q), n64(pool), np_table, ctx, want["cu"], see, hd ** -0.5, BF16)
        assert (np.abs(n64(out) - wo) <= tol).all() and (np.abs(n64(lse) - wl) <= ltol).all()
        # log probabilities of the logits as they are
        for r in range(total):
            p, rank, ent, ls, ids, top = R.logprobs_row(n64(logits[r]), 0, 3)
            e = 2 * R.sum_bound(V / 256 + 8)
            assert int(lp.rank[r]) == rank and lp.top_ids[r].tolist() == ids.tolist()
            assert abs(float(lp.logprob[r]) - p) <= e + 2.0 ** -23 * abs(p)
            assert abs(float(lp.lse[r]) - ls) <= e + 2.0 ** -23 * abs(ls)
            assert abs(float(lp.entropy[r]) - ent) <= e * (1 + ent) + 2.0 ** -23 * ent
        lens, head = plan.lens.clone(), plan.free_head.clone()
    assert lens.tolist() == [50, 9, 105]


@pytest.mark.parametrize("name,widths", [("tiny", [3, 3]), ("m407", [4, 2, 2])])
def test_tree_speculation_with_split_activations(name, widths):
    """More than 8 nodes a pass, so the projections run on the tensor cores and read the attention's output as high
    and low fp16 halves."""
    sh, W, n = S.SHAPES[name], oracle_weights(name), nodes_of(widths)
    P, n_new = S.prompts(1, 17, sh.vocab, seed=142)[0], 7
    m = gpu_model(name, None, max_lanes=n, max_seq=17 + n_new + n, L_max=4, max_prefill_tokens=32, act_split=1)
    plain = D.generate_lane(W, P, 4, n_new)
    stop = stop_at(plain)
    assert stop > 1
    m.prefill(0, P, 4)
    tok, _ = m.speculate_tree(0, n_new, 2, 4, widths)
    status_clean(m)
    assert tok[:stop].tolist() == plain.tokens[:stop].tolist()


@pytest.mark.parametrize("tree", [False, True])
def test_a_padded_batch_stores_nothing_for_its_empty_rows(tree):
    """A batch of a fixed number of rows of which the last hold no token, in memory that an earlier plan has used."""
    i32 = dict(dtype=torch.int32, device="cuda")
    rows, H, hd, page = 40, 2, 64, 16
    pool = torch.zeros(8, 2, 1, page, hd, dtype=F16, device="cuda")
    table, free, rope = torch.full((2, 4), -1, **i32), torch.arange(8, **i32), T.rope_table(64, hd)
    lens, head = torch.zeros(2, **i32), torch.zeros(1, **i32)
    x = torch.ones(rows, (H + 2) * hd, dtype=F16, device="cuda")
    for fresh in ([25, 15], [3, 4], [0, 1], [0, 0]):
        n = sum(fresh)
        parents = torch.tensor([-1] * rows, **i32) if tree else None
        plan = T.plan_batch(lens, torch.tensor(fresh, **i32), table, free, head, page, rows, parents=parents,
                            mask_words=2 if tree else 0)
        assert bool((plan.slots[n:] == -1).all()) and bool((plan.positions[n:] == 0).all())
        assert not tree or bool((plan.masks[n:] == 0).all())
        st = torch.zeros(1, **i32)
        before = pool.clone()
        T.norm_rope_append(x, H, pool, plan.slots, plan.positions, rope, status=st)
        changed = (pool != before).permute(0, 3, 1, 2, 4).reshape(8 * page, -1).any(1).nonzero()[:, 0].tolist()
        assert int(st) == 0 and changed == sorted(plan.slots[:n].tolist())
        lens, head = plan.lens.clone(), plan.free_head.clone()
        x = x + 1
        del plan
