"""Self-speculative greedy decode with a tree of drafts, and prompt scoring, on the GPU path against the fp64 oracle.
With greedy choices a tree of drafts gives the tokens of a plain decode at the verify depth, whatever its shape; the
GPU must emit them up to the first position where the oracle's top-1/top-2 margin is at most 1e-3."""
import numpy as np
import pytest

import synthetic as S
from oracle import decode as D
from oracle import model as M

import operator_refs as R
from gpu_helpers import MARGIN, gpu_model, oracle_weights, status_clean

pytestmark = pytest.mark.gpu


def stop_at(plain):
    for t in range(len(plain.tokens)):
        if M.top2_margin(plain.logits[t]) <= MARGIN:
            return t
    return len(plain.tokens)


def nodes_of(widths):
    n, level = 1, 1
    for w in widths:
        level *= w
        n += level
    return n


def tree_rounds(W, prompt, Ld, Lv, widths, n_new):
    """Rounds of the tree speculation, every node drafted by its own run of the oracle over its whole path."""
    tokens = [int(D.generate_lane(W, prompt, Lv, 1).tokens[0])]
    rounds = 0
    while len(tokens) < n_new:
        rounds += 1
        path = []
        plain = D.generate_lane(W, prompt, Lv, len(tokens) + len(widths) + 1).tokens
        node = list(tokens)
        taken = 1
        for w in widths[:n_new - len(tokens) - 1]:
            x, _ = M.forward(W, np.concatenate([prompt, node]), Ld)
            lg = M.head_logits(W, x[-1])
            best = np.lexsort((np.arange(len(lg)), -lg))[:w]
            nxt = int(plain[len(tokens) + len(path)])
            if nxt not in best:
                break
            path.append(nxt)
            node.append(nxt)
            taken += 1
        tokens += [int(t) for t in plain[len(tokens):len(tokens) + taken]]
    return rounds


@pytest.mark.parametrize("name,Ld,Lv,widths", [("tiny", 4, 4, [2, 2]), ("tiny", 1, 4, [3, 2, 1]), ("tiny", 2, 8, [4]),
                                               ("tiny", 2, 8, [1, 1, 1]), ("tiny", 1, 2, [8, 3, 1]),
                                               ("m407", 2, 8, [3, 2]), ("m1b4_mini", 1, 3, [4, 2, 2])])
def test_tree_matches_plain_decode(name, Ld, Lv, widths):
    sh = S.SHAPES[name]
    W = oracle_weights(name)
    T, n_new, n = 13, 9, nodes_of(widths)
    P = S.prompts(2, T, sh.vocab, seed=131)
    m = gpu_model(name, None, max_lanes=max(2, n), max_seq=T + n_new + n, L_max=8, max_prefill_tokens=max(T, n))
    for i in range(2):
        plain = D.generate_lane(W, P[i], Lv, n_new)
        m.prefill(i, P[i], Lv)
        tok, rounds = m.speculate_tree(i, n_new, Ld, Lv, widths)
        status_clean(m)
        stop = stop_at(plain)
        assert tok[:stop].tolist() == plain.tokens[:stop].tolist(), (i, tok, plain.tokens)
        if stop == n_new and Ld == Lv:  # every level is accepted: the greedy choice is among a node's best
            assert rounds == -(-(n_new - 1) // (len(widths) + 1))
        assert -(-(n_new - 1) // (len(widths) + 1)) <= rounds <= n_new - 1


def test_tree_rounds_match_the_oracle_and_a_chain_matches_speculate():
    W = oracle_weights("tiny")
    T, n_new = 10, 8
    P = S.prompts(1, T, 512, seed=132)[0]
    m = gpu_model("tiny", None, max_lanes=16, max_seq=48, L_max=8, max_prefill_tokens=16)
    plain = D.generate_lane(W, P, 4, n_new)
    if stop_at(plain) < n_new:
        pytest.skip("a near-tie in the oracle's run")
    for widths in ([3, 2], [1, 1, 1], [6]):
        m.prefill(0, P, 4)
        tok, rounds = m.speculate_tree(0, n_new, 1, 4, widths)
        assert tok.tolist() == plain.tokens.tolist()
        assert rounds == tree_rounds(W, P, 1, 4, widths, n_new)
    # the lane goes on from where the call left it, by either call
    m.prefill(0, P, 4)
    a, _ = m.speculate_tree(0, 3, 1, 4, [2, 2])
    b, _ = m.speculate(0, 3, 1, 4, 2)
    c, _ = m.speculate_tree(0, 4, 2, 4, [3])
    status_clean(m)
    assert a.tolist() + b.tolist()[1:] + c.tolist()[1:] == plain.tokens.tolist()


def test_tree_after_a_shared_prefix_and_beside_decode():
    """A lane on shared pages speculates; its donor's and the other lanes' caches stay as they were."""
    sh, W = S.SHAPES["m1b4_mini"], oracle_weights("m1b4_mini")
    pre, n_new = 64, 6
    P = S.prompts(3, pre + 9, sh.vocab, seed=133)
    P[1:, :pre] = P[0, :pre]
    m = gpu_model("m1b4_mini", None, max_lanes=16, max_seq=pre + 40, L_max=3, max_prefill_tokens=128)
    m.prefill(0, P[0], 3)
    m.prefill(1, P[1], 3, share_from=0, shared_tokens=pre)
    m.prefill(2, P[2], 3, share_from=0, shared_tokens=pre)
    for lane in (1, 0):
        plain = D.generate_lane(W, P[lane], 3, n_new)
        tok, _ = m.speculate_tree(lane, n_new, 1, 3, [3, 3])
        stop = stop_at(plain)
        assert tok[:stop].tolist() == plain.tokens[:stop].tolist()
    plain = D.generate_lane(W, P[2], 3, n_new)
    tok, _ = m.speculate(2, n_new, 1, 3, 4)
    status_clean(m)
    stop = stop_at(plain)
    assert tok[:stop].tolist() == plain.tokens[:stop].tolist()


def test_tree_refusals():
    from dynamic_depth_b200 import TlError
    m = gpu_model("tiny", None, max_lanes=8, max_seq=32, L_max=8, max_prefill_tokens=16)
    P = S.prompts(1, 8, 512, seed=134)
    m.prefill(0, P[0], 4)

    def status(*a):
        with pytest.raises(TlError) as e:
            m.speculate_tree(*a)
        return e.value.status
    assert status(0, 5, 2, 8, [2]) == -4          # verify deeper than the lane's cache
    assert status(1, 5, 2, 4, [2]) == -3          # lane never prefilled
    assert status(0, 5, 4, 2, [2]) == -1          # draft deeper than verify
    assert status(0, 5, 2, 4, []) == -1
    assert status(0, 5, 2, 4, [0]) == -1
    assert status(0, 5, 2, 4, [65]) == -1
    assert status(0, 5, 2, 4, [2, 3]) == -1       # 9 nodes for 8 lanes
    assert status(0, 22, 2, 4, [4]) == -1         # 8 + 22 + 5 - 2 > 32 positions
    assert status(8, 5, 2, 4, [2]) == -1
    tok, rounds = m.speculate_tree(0, 1, 2, 4, [2])  # one token: the prompt's own
    assert rounds == 0 and len(tok) == 1


@pytest.mark.parametrize("name,T,L,lanes", [("tiny", 23, 3, 4), ("m407", 20, 2, 8), ("m1b4_mini", 70, 2, 16)])
def test_score_matches_oracle(name, T, L, lanes):
    sh, W = S.SHAPES[name], oracle_weights(name)
    P = S.prompts(1, T, sh.vocab, seed=135)[0]
    m = gpu_model(name, None, max_lanes=lanes, max_seq=T + 2, L_max=L, max_prefill_tokens=T)
    o = m.score(1, P, L, n_top=4)
    status_clean(m)
    x, _ = M.forward(W, P, L)
    assert len(o.logprob) == T
    for t in range(T):
        lg = M.head_logits(W, x[t])
        tgt = int(P[t + 1]) if t + 1 < T else -1
        lp, rank, ent, lse, ids, top = R.logprobs_row(lg, tgt, 4)
        # the parity bar of the logits (max-abs 1e-2) bounds all of them: log-sum-exp and log probabilities move by
        # at most one and two of it, the entropy by the spread of the logits times it
        assert abs(float(o.lse[t]) - lse) <= 1e-2
        assert abs(float(o.logprob[t]) - lp) <= 2e-2
        assert abs(float(o.entropy[t]) - ent) <= 2e-2 * (1 + lg.max() - lg.min())
        assert np.abs(o.top_logprobs[t].cpu().numpy() - top).max() <= 2e-2
        gap = np.sort(lg)[::-1][:5]
        if (gap[:-1] - gap[1:]).min() > 2e-2:
            assert o.top_ids[t].tolist() == ids.tolist()
    # the lane is prefilled as by prefill
    plain = D.generate_lane(W, P, L, 2)
    tok, _ = m.speculate(1, 2, 1, L, 1)
    assert int(tok[0]) == int(plain.tokens[0]) or stop_at(plain) == 0


def test_score_on_a_shared_prefix():
    sh = S.SHAPES["tiny"]
    P = S.prompts(2, 90, sh.vocab, seed=136)
    P[1, :64] = P[0, :64]
    m = gpu_model("tiny", None, max_lanes=4, max_seq=96, L_max=3, max_prefill_tokens=96)
    whole = m.score(2, P[1], 3, n_top=1)
    m.score(0, P[0], 3)
    part = m.score(1, P[1], 3, n_top=1, share_from=0, shared_tokens=64)
    status_clean(m)
    assert len(part.logprob) == 90 - 64 and len(whole.logprob) == 90
    # the same kernels on the same positions; only the widths of the passes differ
    assert np.abs(part.logprob.cpu().numpy() - whole.logprob[64:].cpu().numpy()).max() <= 2e-2
