"""The serving operators on the GPU against plain 64-bit implementations (operator_refs.py)."""
import math

import numpy as np
import pytest
import torch

import dynamic_depth_b200 as T
from dynamic_depth_b200 import _lib
import operator_refs as R

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ------------------------------------------------------------ log probabilities --
def check_logprobs(x, targets, n_top):
    o = T.token_logprobs(x, targets, n_top=n_top)
    xs = x.double().cpu().numpy()
    V = x.shape[1]
    tol = R.sum_bound(V / 256 + 8)  # a lane sums at most vocab / 256 terms
    for r in range(x.shape[0]):
        t = -1 if targets is None else int(targets[r])
        lp, rank, ent, lse, ids, top = R.logprobs_row(xs[r], t, n_top)
        z = abs(lse) if math.isfinite(lse) else 0.0
        got = [float(o.entropy[r]), float(o.lse[r])] + ([float(o.logprob[r])] if targets is not None else [])
        want = [ent, lse] + ([lp] if targets is not None else [])
        for g, w in zip(got, want):
            # entropy = ln S - T / S: the errors of S and of T, whose terms all have one sign
            assert np.allclose(g, w, rtol=2.0 ** -23, atol=2 * tol * (1 + abs(ent)) if math.isfinite(w) else 0,
                               equal_nan=True), (r, g, w, z)
        if targets is not None:
            assert int(o.rank[r]) == rank, (r, int(o.rank[r]), rank)
        if n_top:
            assert o.top_ids[r].tolist() == ids.tolist(), r
            assert np.allclose(o.top_logprobs[r].cpu().double().numpy(), top, rtol=2.0 ** -23, atol=2 * tol,
                               equal_nan=True)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,vocab,n_top", [(1, 1, 1), (3, 2, 2), (2, 7, 0), (5, 255, 3), (4, 256, 64), (3, 513, 20),
                                              (2, 4097, 5), (1, 50257, 8), (9, 50257, 64), (700, 1003, 12)])
def test_logprobs_sizes(dtype, rows, vocab, n_top):
    g = gen(rows * 7 + vocab)
    x = (torch.randn(rows, vocab, generator=g, device="cuda") * 4).to(dtype)
    t = torch.randint(-1, vocab, (rows,), generator=g, device="cuda").int()
    check_logprobs(x, t, n_top)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_logprobs_structured_rows(dtype):
    V = 6000
    x = torch.zeros(9, V, device="cuda")
    x[1] = -math.inf                                        # nothing left
    x[2] = -math.inf
    x[2, [5, 17, 5999]] = torch.tensor([1.0, 2.0, 1.0], device="cuda")   # a few tokens left
    x[3] = torch.arange(V, device="cuda") / 1000            # ascending
    x[4] = -torch.arange(V, device="cuda") / 1000           # descending
    x[5] = torch.finfo(dtype).min                           # the type's lowest value everywhere
    x[6] = torch.finfo(dtype).min
    x[6, 4000] = 3.0
    x[7, ::2] = -0.0                                        # equals +0
    x[8, 100:5000] = 50.0
    x = x.to(dtype)
    for n_top in (1, 20, 64):
        check_logprobs(x, torch.tensor([5999, 7, 17, 300, 0, 12, 4000, 301, 4999], device="cuda").int(), n_top)
    check_logprobs(x, torch.tensor([0, -1, 3, 5999, 5999, 0, 0, 302, 0], device="cuda").int(), 3)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,vocab", [(3, 40000), (1500, 9000)])
def test_logprobs_masks_of_the_lowest_value(dtype, rows, vocab):
    """Masked stretches (the type's lowest value, or -inf) before and after the tokens that are left, in every order
    that a pass over the row can meet them; a warp a row and a cluster a row."""
    g = gen(vocab)
    x = (torch.randn(rows, vocab, generator=g, device="cuda") * 4).to(dtype)
    low = torch.finfo(dtype).min
    x[0, :vocab * 3 // 4] = low
    x[1, vocab // 8:] = low
    x[2, :vocab // 2] = -math.inf
    x[2, vocab // 2:-3] = low
    pick = torch.tensor([vocab - 1, 5, vocab - 2] + [vocab // 2] * (rows - 3), device="cuda").int()
    o = T.token_logprobs(x, pick, n_top=7)
    check_logprobs(x[:3], pick[:3], 7)
    small = T.token_logprobs(x[:3].contiguous(), pick[:3].contiguous(), n_top=7)
    for u, v in zip(o, small):  # either way of sharing the rows out: the same ids, sums to rounding
        assert torch.equal(u[:3], v) if v.dtype == torch.int32 else torch.allclose(u[:3], v, rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("n_top", [1, 20, 21, 64])
def test_logprobs_many_short_rows(n_top):
    """A warp a row: random rows, and rows whose values are all equal, ascending, or mostly masked."""
    V, rows = 3001, 1300
    x = torch.randn(rows, V, generator=gen(n_top), device="cuda") * 3
    x[0] = 1.0
    x[1] = torch.arange(V, device="cuda")
    x[2] = -torch.arange(V, device="cuda")
    x[3] = -math.inf
    x[4, 7:] = -math.inf
    x[5] = (torch.arange(V, device="cuda") // 300).float()
    x[6, 2990:] = math.nan
    t = torch.randint(0, V, (rows,), generator=gen(1), device="cuda").int()
    keep = list(range(12)) + [rows - 1]
    for dtype in (F32, BF16):
        y = x.to(dtype)
        o = T.token_logprobs(y, t, n_top=n_top)
        tol = R.sum_bound(V / 32 + 8)  # a lane sums at most vocab / 32 terms
        for r in keep:
            lp, rank, ent, lse, ids, top = R.logprobs_row(y[r].double().cpu().numpy(), int(t[r]), n_top)
            assert o.top_ids[r].tolist() == ids.tolist() and int(o.rank[r]) == rank
            for got, want in ((o.logprob[r], lp), (o.lse[r], lse), (o.entropy[r], ent)):
                assert np.allclose(float(got), want, rtol=2.0 ** -23, equal_nan=True,
                                   atol=2 * tol * (1 + abs(ent)) if math.isfinite(want) else 0)
            assert np.allclose(o.top_logprobs[r].cpu().double().numpy(), top, rtol=2.0 ** -23, atol=2 * tol,
                               equal_nan=True)


def test_logprobs_nan_and_infinity():
    x = torch.randn(5, 3001, generator=gen(3), device="cuda")
    x[0, 17] = math.nan
    x[1, 2999] = math.inf
    x[2, [4, 9]] = math.inf
    x[3, 8] = -math.nan
    x[3, 2000] = math.inf
    check_logprobs(x, torch.tensor([3, 4, 9, 7, 3000], device="cuda").int(), 5)
    o = T.token_logprobs(x, torch.tensor([3001, -7, 3001, 2 ** 30, -2], device="cuda").int())  # no such token
    assert torch.isnan(o.logprob).all() and (o.rank == -1).all() and o.top_ids is None


def test_logprobs_strided_rows_and_no_target():
    g = gen(5)
    wide = torch.randn(6, 4000, generator=g, device="cuda")
    for lo, hi in ((0, 3999), (1, 3000), (3, 2001), (5, 2054)):
        check_logprobs(wide[:, lo:hi], None, 4)
        check_logprobs(wide.bfloat16()[::2, lo:hi], None, 4)
    t = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert T.token_logprobs(wide[:0], t, n_top=2).top_ids.shape == (0, 2)


def test_logprobs_are_the_same_every_time_and_in_a_graph():
    x = torch.randn(3, 50257, generator=gen(6), device="cuda")
    t = torch.tensor([1, 2, 50256], device="cuda").int()
    a = T.token_logprobs(x, t, n_top=6)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        b = T.token_logprobs(x, t, n_top=6)
    for _ in range(2):
        gr.replay()
    torch.cuda.synchronize()
    for u, v in zip(a, b):
        assert torch.equal(u, v)


# ------------------------------------------------------------------ batch plans --
def run_plan(cached, fresh, page, max_pages, n_free, head, parents=None, words=0, n_rows=None, seed=0):
    rng = np.random.default_rng(seed)
    n = len(cached)
    ids = rng.permutation(300000).astype(np.int32)
    table, at = np.full((n, max_pages), -1, np.int32), 0
    for r, c in enumerate(cached):
        h = min(max_pages, -(-c // page)) if c > 0 else 0
        table[r, :h] = ids[at:at + h]
        at += h
    free = ids[at:at + n_free]
    total = sum(f for f, c in zip(fresh, cached) if 0 <= f <= 1 << 24 and c >= 0)
    rows = total if n_rows is None else n_rows
    dt = torch.from_numpy(table.copy()).cuda()
    par = None
    if parents is not None:
        par = torch.tensor((list(parents) + [0] * rows)[:rows], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = T.plan_batch(torch.tensor(cached, dtype=torch.int32, device="cuda"),
                     torch.tensor(fresh, dtype=torch.int32, device="cuda"), dt, torch.from_numpy(free).cuda(),
                     torch.tensor([head], dtype=torch.int32, device="cuda"), page, rows, parents=par,
                     mask_words=words, status=status)
    want = R.plan(cached, fresh, table, free, head, page, parents, words)
    k = min(rows, total)
    assert o.cu.tolist() == want["cu"]
    assert o.lens.tolist() == want["lens"]
    assert o.granted.tolist() == want["granted"]
    assert o.free_head.tolist() == [want["free_head"]]
    assert o.slots[:k].tolist() == want["slots"][:k]
    assert o.positions[:k].tolist() == want["positions"][:k]
    assert np.array_equal(dt.cpu().numpy(), table)
    if words:
        got = o.masks[:k].cpu().numpy().astype(np.int64) & 0xFFFFFFFF
        assert got.tolist() == [list(m) for m in want["masks"][:k]]
    return o, int(status)


def random_tree(rng, n):
    return [-1 if j == 0 or rng.random() < 0.1 else int(rng.integers(0, j)) for j in range(n)]


@pytest.mark.parametrize("page", [1, 16, 64])
@pytest.mark.parametrize("n", [1, 5, 255, 257, 1000])
def test_plan_lengths(page, n):
    rng = np.random.default_rng(n + page)
    cached = rng.integers(0, 200, n).tolist()
    fresh = rng.integers(0, 90, n).tolist()
    cached[0] = 0
    run_plan(cached, fresh, page, 400, 60000, 2)
    run_plan(cached, [1] * n, page, 400, 60000, 0)


def test_plan_without_new_tokens():
    run_plan([5, 0, 64], [0, 0, 0], 16, 8, 4, 1)


@pytest.mark.parametrize("words", [1, 2, 8])
def test_plan_trees(words):
    rng = np.random.default_rng(words)
    fresh = [1, 32 * words, 0, 32 * words - 1, 5]
    parents = sum((random_tree(rng, f) for f in fresh), [])
    _, st = run_plan([7, 0, 3, 500, 64], fresh, 16, 64, 100, 0, parents, words)
    assert st == 0
    run_plan([7, 0, 3, 500, 64], fresh, 16, 64, 100, 0, None, words)  # masks of a draft without branches
    chain = sum((list(range(-1, f - 1)) for f in fresh), [])
    run_plan([7, 0, 3, 500, 64], fresh, 16, 64, 100, 0, chain, words)


def test_plan_refusals_on_the_device():
    # the list runs out at the third request; the fourth needs no page; the table's row ends before the fifth's end
    o, st = run_plan([16, 10, 5, 3, 100], [40, 30, 60, 2, 40], 16, 8, 7, 1)
    assert o.granted.tolist() == [1, 1, 0, 1, 0] and st == _lib.TL_BAD_LENGTH
    o, st = run_plan([16, -3, 5], [4, 2, -1], 16, 8, 7, 0)
    assert o.granted.tolist() == [1, 0, 0] and st == _lib.TL_BAD_LENGTH
    # a parent that is not an earlier node counts as none
    _, st = run_plan([3], [4], 16, 8, 7, 0, [-1, 1, 5, 2], 1)
    assert st == _lib.TL_BAD_PARENT
    # more nodes than mask bits; fewer rows than tokens
    _, st = run_plan([3, 4], [40, 2], 16, 8, 9, 0, None, 1)
    assert st == _lib.TL_BAD_LENGTH
    _, st = run_plan([3, 4], [20, 20], 16, 8, 9, 0, None, 1, n_rows=25)
    assert st == _lib.TL_BAD_LENGTH


def test_plan_leaves_rows_behind_the_batch():
    dev = "cuda"
    slots = torch.full((10,), 77, dtype=torch.int64, device=dev)
    pos = torch.full((10,), 88, dtype=torch.int32, device=dev)
    z = torch.zeros(8, dtype=torch.int32, device=dev)
    table = torch.full((1, 4), -1, dtype=torch.int32, device=dev)
    i = torch.tensor([3, 4, 9, 8, 0, 0, 0, 0], dtype=torch.int32, device=dev)  # cached 3, fresh 4, free pages 9, 8
    _lib.check(_lib.lib().tl_plan_batch(i.data_ptr(), i.data_ptr() + 4, 1, 4, table.data_ptr(), 4, i.data_ptr() + 8, 2,
                                        i.data_ptr() + 16, None, 10, 0, z.data_ptr(), z.data_ptr() + 8,
                                        z.data_ptr() + 12, z.data_ptr() + 16, slots.data_ptr(), pos.data_ptr(), None,
                                        None, torch.cuda.current_stream().cuda_stream), "plan")
    assert slots.tolist() == [-1, 36, 37, 38] + [77] * 6 and pos.tolist() == [3, 4, 5, 6] + [88] * 6
    assert table.tolist() == [[-1, 9, -1, -1]] and z.tolist()[:5] == [0, 4, 7, 1, 1]


# ------------------------------------------------------ norm, rotation and append --
@pytest.mark.parametrize("din,dcache", [(F32, F16), (F32, BF16), (F16, F16), (BF16, BF16), (BF16, F16), (F16, BF16)])
@pytest.mark.parametrize("heads,kv_heads,hd", [(4, 4, 32), (6, 2, 64), (8, 1, 128), (5, 5, 128)])
@pytest.mark.parametrize("norm", [False, True])
def test_norm_rope(din, dcache, heads, kv_heads, hd, norm):
    rows, page, n_pages, base, length = 37, 16, 6, 1e4, 100003
    g = gen(hd + heads)
    x = torch.randn(rows, (heads + 2 * kv_heads) * hd, generator=g, device="cuda").to(din)
    x[3] = 0  # a row that a norm must not divide by
    gq, gk = (1 + 0.2 * torch.randn(2, hd, generator=g, device="cuda")).unbind(0) if norm else (None, None)
    pool = torch.randn(n_pages, 2, kv_heads, page, hd, generator=g, device="cuda").to(dcache)
    before = pool.clone()
    slots = torch.randperm(n_pages * page, generator=g, device="cuda")[:rows].contiguous()
    slots[5] = -1
    pos = torch.randint(0, length, (rows,), generator=g, device="cuda").int()
    pos[:3] = torch.tensor([0, 1, length - 1])
    rope = T.rope_table(length, hd, base)
    gq, gk = (None, None) if not norm else (gq.contiguous(), gk.contiguous())
    q = T.norm_rope_append(x, heads, pool, slots, pos, rope, q_gain=gq, k_gain=gk, eps=1e-5)
    n64 = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    wq, wk, wv, sq, sk = R.norm_rope(n64(x), heads, kv_heads, hd, pos.cpu().numpy(), base, n64(gq), n64(gk), 1e-5)
    half = R.HALF_STEP[dcache]
    # fp32: the table, the norm's sum of hd terms and square root, three roundings of the rotation
    fp = (hd / 16 + 12) * 2.0 ** -24
    tiny = 2.0 ** -25 if dcache == F16 else 0.0
    assert (np.abs(n64(q) - wq) <= half * np.abs(wq) + fp * sq + tiny).all()
    flat = pool.permute(0, 3, 1, 2, 4).reshape(-1, 2, kv_heads, hd)
    keep = [i for i in range(rows) if i != 5]
    got = n64(flat[slots[keep]])
    assert (np.abs(got[:, 0] - wk[keep]) <= half * np.abs(wk[keep]) + fp * sk[keep] + tiny).all()
    assert (np.abs(got[:, 1] - wv[keep]) <= half * np.abs(wv[keep]) + tiny).all()
    if din == dcache:
        assert np.array_equal(got[:, 1], wv[keep])
    untouched = torch.ones(n_pages * page, dtype=torch.bool, device="cuda")
    untouched[slots[keep]] = False
    old = before.permute(0, 3, 1, 2, 4).reshape(-1, 2, kv_heads, hd)
    assert torch.equal(flat[untouched], old[untouched])


def test_norm_rope_bad_rows_and_strides():
    g = gen(1)
    wide = torch.randn(9, 8 * 64, generator=g, device="cuda").half()
    x = wide[:, 64:64 * 5]  # rows of 4 heads in a wider array
    pool = torch.zeros(2, 2, 1, 16, 64, dtype=F16, device="cuda")
    slots = torch.tensor([0, 1, 2, 32, -2, 5, 2 ** 40, 7, 31], device="cuda")
    pos = torch.tensor([0, 1, -1, 3, 4, 50, 6, 7, 49], device="cuda").int()
    rope = T.rope_table(50, 64)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = torch.full((9, 2, 64), 9.0, dtype=F16, device="cuda")
    T.norm_rope_append(x, 2, pool, slots, pos, rope, q_out=q, status=st)
    assert int(st) == _lib.TL_BAD_POSITION | _lib.TL_BAD_SLOT
    assert (q[[2, 5]] == 9.0).all()  # rows left out
    flat = pool.permute(0, 3, 1, 2, 4).reshape(-1, 2, 64)
    filled = [i for i in range(32) if bool((flat[i] != 0).any())]
    assert filled == [0, 1, 7, 31]
    dense = T.norm_rope_append(x.contiguous(), 2, torch.zeros_like(pool), slots, pos, rope, q_out=q.clone())
    assert torch.equal(q, dense)
    empty = T.norm_rope_append(x[:0], 2, pool, slots[:0], pos[:0], rope)
    assert empty.shape == (0, 2, 64)


# --------------------------------------------------------------- tree attention --
def tree_case(ctx, nodes, H, Hk, hd, dtype, page, masks="tree", seed=0, extra_rows=0, n_pages=None):
    """Inputs of a call: q, pool, table, ctx, cu, mask words (or None) and booleans, total rows."""
    g, rng = gen(seed), np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    total = int(cu[-1]) + extra_rows
    need = [-(-(c + n) // page) for c, n in zip(ctx, nodes)]
    max_pages = max(need + [1]) + 1
    n_pages = sum(need) + 3
    pool = torch.randn(n_pages, 2, Hk, page, hd, generator=g, device="cuda").to(dtype)
    ids = rng.permutation(n_pages).astype(np.int32)
    table, at = np.full((len(ctx), max_pages), -1, np.int32), 0
    for r, k in enumerate(need):
        table[r, :k] = ids[at:at + k]
        at += k
    q = torch.randn(total, H, hd, generator=g, device="cuda").to(dtype)
    most = max(list(nodes) + [1])
    words, see = (most + 31) // 32, None
    if masks is not None:
        see = np.zeros((total, 32 * words), bool)
        for r, n in enumerate(nodes):
            par = random_tree(rng, n)
            for j in range(n):
                row = cu[r] + j
                if masks == "random":
                    see[row, :n] = rng.random(n) < 0.4
                else:
                    if par[j] >= 0:
                        see[row] = see[cu[r] + par[j]]
                    see[row, j] = True
    return dict(q=q, pool=pool, table=table, ctx=np.array(ctx, np.int32), cu=cu, see=see, words=words, most=most)


def mask_tensor(see):
    if see is None:
        return None
    rows, bits = see.shape
    w = (see.reshape(rows, bits // 32, 32).astype(np.uint64) << np.arange(32, dtype=np.uint64)).sum(-1)
    return torch.from_numpy(w.astype(np.uint32).view(np.int32)).cuda()


def run_tree(c, scale=0.0, out=None, **kw):
    d = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = T.tree_attention(c["q"], c["pool"], d(c["table"]), d(c["ctx"]), d(c["cu"]), c["most"],
                              masks=mask_tensor(c["see"]), scale=scale, out=out, return_lse=True, status=st, **kw)
    return o, lse, int(st)


def check_tree(c, scale=0.0, status=0, out=None):
    o, lse, st = run_tree(c, scale, out)
    assert st == status
    sc = scale or c["q"].shape[2] ** -0.5
    pool = c["pool"].double().cpu().numpy()
    wo, wl, tol, ltol = R.tree_attention(c["q"].double().cpu().numpy(), pool, c["table"], c["ctx"], c["cu"], c["see"],
                                         sc, c["q"].dtype)
    n = int(c["cu"][-1])
    go, gl = o[:n].double().cpu().numpy(), lse[:n].double().cpu().numpy()
    assert np.array_equal(np.isinf(gl), np.isinf(wl[:n]))
    bad = ~(np.abs(go - wo[:n]) <= tol[:n])
    assert not bad.any(), (np.argwhere(bad)[:4].tolist(), go[bad][:4], wo[:n][bad][:4], tol[:n][bad][:4])
    fin = np.isfinite(wl[:n])
    assert (np.abs(gl - wl[:n])[fin] <= ltol[:n][fin]).all(), np.abs(gl - wl[:n])[fin].max()
    return o, lse


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("H,Hk", [(1, 1), (4, 4), (8, 2), (5, 1)])
def test_tree_heads(dtype, hd, H, Hk):
    check_tree(tree_case([100, 0, 17], [7, 3, 1], H, Hk, hd, dtype, 16, seed=hd + H))


@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_tree_pages_and_tile_ends(hd, page):
    ctx = [0, 1, 63, 64, 65, 127, 128, 129, 255, 256, 300]
    check_tree(tree_case(ctx, [2, 1, 1, 3, 1, 1, 2, 1, 1, 1, 5], 2, 1, hd, F16, page, seed=page + hd))


@pytest.mark.parametrize("nodes", [1, 4, 5, 8, 9, 16, 17, 33, 64, 100, 256])
@pytest.mark.parametrize("masks", ["tree", "random", None])
def test_tree_node_counts(nodes, masks):
    check_tree(tree_case([70, 0], [nodes, (nodes + 1) // 2], 4, 1, 64, BF16, 32, masks, seed=nodes))


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_tree_long_contexts_are_cut_and_joined(dtype):
    check_tree(tree_case([9000], [3], 4, 1, 128, dtype, 64, seed=1))     # one row block over every SM
    check_tree(tree_case([5000, 17, 2300], [20, 1, 40], 4, 2, 64, dtype, 16, seed=2))
    check_tree(tree_case([4100], [70], 2, 1, 32, dtype, 128, seed=3))


def test_tree_many_requests():
    rng = np.random.default_rng(4)
    n = 700
    check_tree(tree_case(rng.integers(0, 60, n).tolist(), rng.integers(0, 3, n).tolist(), 2, 1, 32, F16, 16, seed=4))


def test_tree_rows_that_see_nothing_and_rows_behind():
    c = tree_case([0, 40, 0], [6, 5, 0], 4, 2, 64, F16, 16, "random", seed=5, extra_rows=4)
    c["see"][:6] = False
    c["see"][2, 1] = True
    out = torch.full_like(c["q"], 7.0)
    o, lse = check_tree(c, out=out)
    assert (o[[0, 1, 3, 4, 5]] == 0).all() and torch.isinf(lse[[0, 1, 3, 4, 5]]).all()
    assert (o[11:] == 7.0).all()


def test_tree_scales_strides_and_fp32_output():
    c = tree_case([333, 60], [9, 12], 4, 2, 64, BF16, 16, seed=6)
    check_tree(c, scale=0.37)
    base, _ = check_tree(c)
    wide = torch.zeros(c["q"].shape[0], 3, 4, 64, dtype=BF16, device="cuda")
    wide[:, 1] = c["q"]
    c["q"] = wide[:, 1]
    out = torch.zeros(c["q"].shape[0], 2, 4, 64, dtype=BF16, device="cuda")
    o, _, _ = run_tree(c, out=out[:, 1])
    assert torch.equal(o, base) and (out[:, 0] == 0).all()
    f32, _, _ = run_tree(c, out=torch.zeros(c["q"].shape[0], 4, 64, device="cuda"))
    assert torch.equal(f32.bfloat16(), base)


@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("nodes", [6, 40])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_tree_ignores_what_a_row_does_not_see(hd, nodes, dtype):
    c = tree_case([50, 0], [nodes, nodes], 2, 1, hd, dtype, 16, "random", seed=7)
    c["see"][:, 3] = False                     # node 3 is seen by nobody, node 2 by one row of each request
    c["see"][:, 2] = False
    c["see"][[1, nodes + 1], 2] = True
    P = 16
    want, wl, _ = run_tree(c)
    pool = c["pool"].clone()
    for r, base in ((0, 50), (1, 0)):
        def put(j, k, v):
            pg, off = c["table"][r][(base + j) // P], (base + j) % P
            c["pool"][pg, 0, :, off], c["pool"][pg, 1, :, off] = k, v
        put(3, math.nan, math.inf)
        put(2, 0.5, math.nan)
        # and whatever lies behind the last node on its page
        end = base + nodes
        if end % P:
            pg = c["table"][r][end // P]
            c["pool"][pg, :, :, end % P:] = math.nan
    got, gl, st = run_tree(c)
    rows = torch.ones(2 * nodes, dtype=torch.bool, device="cuda")
    rows[[1, nodes + 1]] = False
    assert st == 0 and torch.isfinite(got[rows].float()).all()
    assert torch.isnan(got[[1, nodes + 1]].float()).all()
    # the rows that do not see them: as before, within the rounding of probabilities on either path
    tol = 4 * R.HALF_STEP[dtype]
    assert (got[rows].float() - want[rows].float()).abs().max() <= tol * want.float().abs().max() * 2
    assert torch.allclose(gl[rows], wl[rows], atol=1e-5, equal_nan=False)
    c["pool"].copy_(pool)


def test_tree_bad_pages_and_lengths():
    c = tree_case([100, 70, 90], [3, 2, 4], 2, 2, 64, F16, 16, seed=8)
    c["table"][0, 2] = -1
    c["table"][1, 0] = 10 ** 6
    check_tree(c, status=_lib.TL_BAD_PAGE)
    c = tree_case([100, 70, 90], [3, 2, 4], 2, 2, 64, F16, 16, seed=9)
    keep, _, _ = run_tree(c)
    c["ctx"][1] = 10 ** 6  # past its table: the request is left out
    out = torch.full_like(c["q"], 5.0)
    o, _, st = run_tree(c, out=out)
    assert st == _lib.TL_BAD_LENGTH and (o[3:5] == 5.0).all()
    assert torch.equal(o[:3], keep[:3]) and torch.equal(o[5:], keep[5:])
    c["ctx"][1] = -1
    o, _, st = run_tree(c, out=torch.full_like(c["q"], 5.0))
    assert st == _lib.TL_BAD_LENGTH and (o[3:5] == 5.0).all() and torch.equal(o[5:], keep[5:])


@pytest.mark.parametrize("nodes", [2, 40])
def test_tree_lengths_near_31_bits_are_left_out(nodes):
    # a table can repeat pages, so it can hold more positions than an index of 31 bits: the request is left out
    page, max_pages = 1024, 1 << 21
    pool = torch.zeros(1, 2, 1, page, 128, dtype=F16, device="cuda")
    table = torch.zeros(1, max_pages, dtype=torch.int32, device="cuda")
    q = torch.ones(nodes, 1, 128, dtype=F16, device="cuda")
    cu = torch.tensor([0, nodes], dtype=torch.int32, device="cuda")
    for ctx in (2 ** 31 - 1, 2 ** 31 - 64, 2 ** 31 - 4095 - nodes):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full_like(q, 5.0)
        T.tree_attention(q, pool, table, torch.tensor([ctx], dtype=torch.int32, device="cuda"), cu, nodes, out=out,
                         status=st)
        assert int(st) == _lib.TL_BAD_LENGTH and (out == 5.0).all()


def test_tree_far_pages():
    # a pool whose last pages lie past 2^31 elements
    page, hd, Hk = 64, 128, 8
    n_pages = (2 ** 31) // (2 * Hk * page * hd) + 8
    pool = torch.zeros(n_pages, 2, Hk, page, hd, dtype=F16, device="cuda")
    c = tree_case([150], [2], 8, 8, hd, F16, page, seed=10)
    near, _, _ = run_tree(c)
    for i, pg in enumerate(c["table"][0][:3]):
        pool[n_pages - 1 - i] = c["pool"][pg]
    c["table"][0, :3] = [n_pages - 1, n_pages - 2, n_pages - 3]
    c["pool"] = pool
    far, _, st = run_tree(c)
    assert st == 0 and torch.equal(near, far)
    # and the append reaches them
    x = torch.randn(2, 24 * hd, generator=gen(0), device="cuda").half()
    slots = torch.tensor([n_pages * page - 1, n_pages * page - 70], device="cuda")
    T.norm_rope_append(x, 8, pool, slots, torch.zeros(2, dtype=torch.int32, device="cuda"), T.rope_table(4, hd))
    v = x.view(2, 24, hd)[:, 16:]
    assert torch.equal(pool[n_pages - 1, 1, :, 63], v[0]) and torch.equal(pool[n_pages - 2, 1, :, 58], v[1])


def test_tree_graph_replay_and_other_stream():
    c = tree_case([3000, 45], [12, 7], 8, 2, 128, BF16, 16, seed=11)
    want, wl, _ = run_tree(c)
    d = {k: torch.from_numpy(c[k]).cuda() for k in ("table", "ctx", "cu")}
    m = mask_tensor(c["see"])
    ws = T.tree_attention_workspace(128, 8, 2, c["most"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o = T.tree_attention(c["q"], c["pool"], d["table"], d["ctx"], d["cu"], c["most"], masks=m, workspace=ws)
    s.synchronize()
    assert torch.equal(o, want)
    graphs, outs = [], []
    for _ in range(2):  # two graphs that share a workspace, replayed one after the other
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(T.tree_attention(c["q"], c["pool"], d["table"], d["ctx"], d["cu"], c["most"], masks=m,
                                         workspace=ws))
        graphs.append(g)
    for _ in range(3):
        ws.fill_(0xFF)
        for g, o in zip(graphs, outs):
            o.zero_()
            g.replay()
            assert torch.equal(o, want)
    d["ctx"][0] = 2000  # a replay follows the lengths on the device
    graphs[0].replay()
    c["ctx"][0] = 2000
    assert torch.equal(outs[0], run_tree(c)[0])


def test_tree_calls_on_two_streams_at_once():
    # different widths and row counts share the SMs, their shared memory and their tensor memory
    cases = [tree_case([900, 2100, 64], [40, 33, 9], 4, 4, 128, BF16, 64, seed=12),
             tree_case([1500, 700], [60, 64], 8, 2, 64, BF16, 16, seed=13)]
    want = [run_tree(c)[0] for c in cases]
    dev = [{k: torch.from_numpy(c[k]).cuda() for k in ("table", "ctx", "cu")} for c in cases]
    masks = [mask_tensor(c["see"]) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i, c in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                outs[i].append(T.tree_attention(c["q"], c["pool"], dev[i]["table"], dev[i]["ctx"], dev[i]["cu"], c["most"],
                                                masks=masks[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o in outs[i]:
            assert torch.equal(o, want[i])


def test_tree_one_head_of_a_wider_projection():
    # q and out of one head, cut from rows of more: the heads' stride means nothing
    c = tree_case([75], [3], 1, 1, 64, F16, 16, seed=14)
    want, _, _ = run_tree(c)
    wide = torch.zeros(3, 64 * 5, dtype=F16, device="cuda")
    wide[:, 64:128] = c["q"][:, 0]
    c["q"] = wide[:, 64:128].unsqueeze(1)
    assert torch.equal(run_tree(c)[0], want)


# ------------------------------------------------------------------- together --
def test_a_serving_step():
    """Plan, append and attention of two steps: a prompt, then a tree of drafts, against attention over the same keys
    kept in one array."""
    g, rng = gen(12), np.random.default_rng(12)
    H, Hk, hd, page, n_pages, base = 8, 2, 64, 16, 64, 1e4
    i32 = dict(dtype=torch.int32, device="cuda")
    pool = torch.zeros(n_pages, 2, Hk, page, hd, dtype=BF16, device="cuda")
    table = torch.full((3, 12), -1, **i32)
    free = torch.from_numpy(rng.permutation(n_pages).astype(np.int32)).cuda()
    head, lens = torch.zeros(1, **i32), torch.zeros(3, **i32)
    rope = T.rope_table(256, hd, base)
    gq, gk = (1 + 0.1 * torch.randn(hd, generator=g, device="cuda") for _ in range(2))
    V = 999
    w = torch.randn(H * hd, V, generator=g, device="cuda", dtype=F32) / 20
    kept = [[], [], []]
    for fresh, tree in (([40, 7, 90], False), ([9, 1, 14], True)):
        total = sum(fresh)
        parents = sum((random_tree(rng, f) for f in fresh), []) if tree else None
        pt = torch.tensor(parents, **i32) if tree else None
        x = torch.randn(total, (H + 2 * Hk) * hd, generator=g, device="cuda").to(BF16)
        plan = T.plan_batch(lens, torch.tensor(fresh, **i32), table, free, head, page, total, parents=pt,
                            mask_words=1 if tree else 0)
        q = T.norm_rope_append(x, H, pool, plan.slots, plan.positions, rope, q_gain=gq, k_gain=gk)
        out = T.tree_attention(q, pool, table, lens, plan.cu, max(fresh), masks=plan.masks)
        lp = T.token_logprobs(out.reshape(total, -1).float() @ w, torch.zeros(total, **i32), n_top=3)
        # the same by hand: positions from the parents, keys and values in arrays
        ctx, cu = lens.cpu().numpy(), np.concatenate([[0], np.cumsum(fresh)])
        n64 = lambda t: t.double().cpu().numpy()  # noqa: E731
        see = np.zeros((total, 96), bool)
        pos = np.zeros(total, np.int64)
        for r, f in enumerate(fresh):
            for j in range(f):
                p = parents[cu[r] + j] if tree else j - 1
                see[cu[r] + j] = see[cu[r] + p] if p >= 0 else False
                see[cu[r] + j, j] = True
                pos[cu[r] + j] = ctx[r] + see[cu[r] + j].sum() - 1
        wq, wk, wv, _, _ = R.norm_rope(n64(x), H, Hk, hd, pos, base, n64(gq), n64(gk))
        for r, f in enumerate(fresh):
            for j in range(f):
                kept[r].append((wk[cu[r] + j], wv[cu[r] + j]))
            ks, vs = np.array([k for k, _ in kept[r]]), np.array([v for _, v in kept[r]])
            for j in range(f):
                vis = np.concatenate([np.ones(ctx[r], bool), see[cu[r] + j, :f]])
                for h in range(H):
                    s = ks[vis, h // 4] @ wq[cu[r] + j, h] / 8.0
                    p = np.exp(s - s.max())
                    want = (p / p.sum()) @ vs[vis, h // 4]
                    # q, k, v and p each rounded to bf16: scores off by 2 * 2^-8 of sum |q k| / 8 (about |q| |k| / 8)
                    ds = 2 * 2.0 ** -8 * (np.abs(ks[vis, h // 4]) @ np.abs(wq[cu[r] + j, h])).max() / 8.0
                    tol = (math.expm1(2 * ds) + 3 * 2.0 ** -8) * np.abs(vs[vis, h // 4]).max()
                    assert (np.abs(n64(out[cu[r] + j, h]) - want) <= tol).all()
        assert torch.isfinite(lp.logprob).all() and (lp.top_logprobs[:, 0] >= lp.logprob).all()
        lens, head = plan.lens, plan.free_head
    assert lens.tolist() == [49, 8, 104]
