"""Tree attention where every CTA runs many key tiles and several row blocks, so that rings, buffers, barriers and
running references go round many times, against the definition in 64 bits.

A test counts the tiles of its case (as the kernels deal them: two CTAs an SM share them equally) and asserts that
there are more than enough.  Values change sign from one 64-position stretch to the next, so a tile that is dropped,
read twice or taken from another stage moves the result by more than the bound."""
import math

import numpy as np
import pytest
import torch

import operator_refs as R
from test_gpu_operators import BF16, F16, gen, run_tree, tree_case

pytestmark = pytest.mark.gpu


def geometry(hd, rows_per_head):
    """(rows of a block, positions of a tile, stages of a ring) for a width and the most rows of a key head."""
    if rows_per_head <= 32 or hd == 32:
        return (16 if rows_per_head <= 16 else 32 if rows_per_head <= 32 else 64), (64 if hd == 128 else 128), \
            (4 if hd == 32 else 2)
    return 128, 64, (2 if hd == 128 else 4)


def tiles_per_cta(c):
    Hk, hd = c["pool"].shape[2], c["pool"].shape[4]
    G = c["q"].shape[1] // Hk
    BM, KT, stages = geometry(hd, c["most"] * G)
    units = 0
    for r in range(len(c["ctx"])):
        n = int(c["cu"][r + 1] - c["cu"][r])
        units += -(-(int(c["ctx"][r]) + n) // KT) * -(-n * G // BM) * Hk
    return units / (2 * torch.cuda.get_device_properties(0).multi_processor_count), stages


def positions_of(c, r):
    """(pages, offsets) of a request's positions."""
    P = c["pool"].shape[3]
    pos = torch.arange(int(c["ctx"][r]) + int(c["cu"][r + 1] - c["cu"][r]), device="cuda")
    return torch.from_numpy(c["table"][r]).cuda().long()[pos // P], pos % P


def put(c, r, which, x):
    """Keys (0) or values (1) of a request, [positions, key heads, width]."""
    pg, off = positions_of(c, r)
    c["pool"][pg, which, :, off] = x.to(c["pool"].dtype)


def striped_values(c, seed):
    g = gen(seed)
    Hk, hd = c["pool"].shape[2], c["pool"].shape[4]
    for r in range(len(c["ctx"])):
        n = len(positions_of(c, r)[0])
        sign = torch.randint(0, 2, (n // 64 + 1, Hk, hd), generator=g, device="cuda").float() * 2 - 1
        v = sign.repeat_interleave(64, 0)[:n] * (1 + 0.1 * torch.randn(n, Hk, hd, generator=g, device="cuda"))
        put(c, r, 1, v)


def definition(c, scale):
    """(out, lse, bound on out, bound on lse) in fp64 on the GPU; the bounds are operator_refs.tree_attention's, but
    for what fp16 probabilities lose: they are held 2^7 times larger, so a denormal one is off by 2^-32 of the largest."""
    rows, H, hd = c["q"].shape
    Hk = c["pool"].shape[2]
    G = H // Hk
    half = R.HALF_STEP[c["q"].dtype]
    out = torch.zeros(rows, H, hd, dtype=torch.float64, device="cuda")
    tol, lse, ltol = torch.zeros_like(out), torch.full((rows, H), -math.inf, dtype=torch.float64, device="cuda"), \
        torch.zeros(rows, H, dtype=torch.float64, device="cuda")
    for r in range(len(c["ctx"])):
        a, b, ctx = int(c["cu"][r]), int(c["cu"][r + 1]), int(c["ctx"][r])
        n = b - a
        if n == 0:
            continue
        pg, off = positions_of(c, r)
        k, v = c["pool"][pg, 0, :, off].double(), c["pool"][pg, 1, :, off].double()  # [positions, Hk, hd]
        q = c["q"][a:b].double().view(n, Hk, G, hd)
        see = torch.ones(n, ctx + n, dtype=torch.bool, device="cuda")
        see[:, ctx:] = torch.ones(n, n, device="cuda").tril() > 0 if c["see"] is None else \
            torch.from_numpy(c["see"][a:b, :n]).cuda()
        see = see[None, :, None]  # [1, n, 1, positions]
        s = torch.einsum("nhgd,thd->hngt", q, k) * scale
        size = torch.einsum("nhgd,thd->hngt", q.abs(), k.abs()) * scale
        s = s.masked_fill(~see, -math.inf)
        m = s.amax(-1, keepdim=True)
        e = torch.exp(s - m)
        z = e.sum(-1, keepdim=True)
        p = e / z
        o, mag = torch.einsum("hngt,thd->nhgd", p, v), torch.einsum("hngt,thd->nhgd", p, v.abs())
        keys = see.sum(-1).double()  # [1, n, 1]
        big = torch.where(see, s, torch.zeros_like(s)).abs().amax(-1)
        ds = (hd + 4) * 2.0 ** -24 * torch.where(see, size, torch.zeros_like(size)).amax(-1) + 2.0 ** -22 * big
        rel = (2 * ds + keys * 2.0 ** -23 + 2.0 ** -19).permute(1, 0, 2)[..., None]
        t = (half + rel) * mag + half * o.abs() + 1e-7
        if c["q"].dtype == F16:
            t = t + (keys * 2.0 ** -32 / z[..., 0]).permute(1, 0, 2)[..., None] * v.abs().amax(0)[None, :, None]
        ll = (m + torch.log(z))[..., 0]
        lt = ds + keys * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -23 * ll.abs()
        out[a:b], tol[a:b] = o.reshape(n, H, hd), t.reshape(n, H, hd)
        lse[a:b], ltol[a:b] = ll.permute(1, 0, 2).reshape(n, H), lt.permute(1, 0, 2).reshape(n, H)
    return out, lse, tol, ltol


def check(c, least, scale=None):
    per_cta, stages = tiles_per_cta(c)
    assert per_cta > least * stages, (per_cta, stages)
    scale = scale or c["q"].shape[2] ** -0.5
    wo, wl, tol, ltol = definition(c, scale)
    o, lse, st = run_tree(c, scale=scale)
    assert st == 0
    n = int(c["cu"][-1])
    off = (o[:n].double() - wo[:n]).abs() / tol[:n]
    assert bool((off <= 1).all()), (float(off.nan_to_num(9e9).max()), (~(off <= 1)).nonzero()[:4].tolist())
    loff = (lse[:n].double() - wl[:n]).abs() / ltol[:n]
    assert bool((loff <= 1).all()), float(loff.nan_to_num(9e9).max())
    again, lse2, _ = run_tree(c, scale=scale)
    assert torch.equal(o[:n], again[:n]) and torch.equal(lse[:n], lse2[:n])


@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("nodes,group", [(1, 1), (1, 4), (5, 4), (10, 4), (40, 4)])
def test_rings_go_round_many_times(hd, nodes, group):
    dtype = F16 if (nodes + hd // 32) % 2 else BF16
    rng = np.random.default_rng(hd + nodes)
    ctx = rng.integers(2200, 3800, 24).tolist()
    c = tree_case(ctx, [nodes] * 24, 8 * group, 8, hd, dtype, 16 if hd == 64 else 64, seed=nodes)
    striped_values(c, hd)
    check(c, 2)


@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("nodes,group", [(2, 2), (10, 4)])
def test_many_short_requests_a_cta(hd, nodes, group):
    """Several whole row blocks a CTA, and more requests than a CTA has threads."""
    rng = np.random.default_rng(hd)
    n = 800
    ctx = rng.integers(0, 400, n).tolist()
    fresh = rng.integers(max(1, nodes // 2), nodes + 1, n).tolist()
    fresh[3] = fresh[-2] = 0
    c = tree_case(ctx, fresh, 6 * group, 6, hd, F16 if hd == 64 else BF16, 32, seed=hd + 1)
    striped_values(c, hd + 1)
    check(c, 2)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("nodes", [1, 40])
def test_scores_that_climb(hd, dtype, nodes):
    """Scores rise by 2^9 between stretches of a context, and values fall by as much: every stretch has its share of
    the result, and reaches it only if the sums so far are scaled by the right factor each time the reference moves."""
    levels, R_ = (2 if dtype == F16 else 12), 20
    ctx = [2600 + 64 * r for r in range(R_)]
    c = tree_case(ctx, [nodes] * R_, 8, 8, hd, dtype, 64, seed=nodes)
    g = gen(hd)
    c["q"] = (1 + 0.05 * torch.randn(*c["q"].shape, generator=g, device="cuda")).to(dtype)
    step = 9 * math.log(2) / math.sqrt(hd)  # of each key element
    for r in range(R_):
        n = ctx[r] + nodes
        level = torch.arange(n, device="cuda") * levels // n
        k = level[:, None, None] * step + 0.05 * torch.randn(n, 8, hd, generator=g, device="cuda")
        sign = torch.randint(0, 2, (n // 64 + 1, 8, hd), generator=g, device="cuda").float() * 2 - 1
        v = sign.repeat_interleave(64, 0)[:n] * torch.exp2(9.0 * (levels - 1 - level))[:, None, None]
        put(c, r, 0, k)
        put(c, r, 1, v)
    check(c, 2)


@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("nodes", [1, 40])
@pytest.mark.parametrize("gap", [24.3, 25.5])
def test_probabilities_far_below_the_largest_keep_their_share(hd, nodes, gap):
    """One key of value 0 has 2^gap times the weight of each other, whose values are 1: what is left of the result is
    their share, which fp16 probabilities relative to the largest would lose (below 2^-25) or double (below 2^-24)."""
    n_req, ctx = 24, 6000
    c = tree_case([ctx] * n_req, [nodes] * n_req, 8, 8, hd, F16, 64, seed=hd)
    c["q"] = torch.ones_like(c["q"])
    for r in range(n_req):
        k = torch.zeros(ctx + nodes, 8, hd, device="cuda")
        k[0] = gap * math.log(2) / math.sqrt(hd)
        v = torch.ones(ctx + nodes, 8, hd, device="cuda")
        v[0] = 0
        put(c, r, 0, k)
        put(c, r, 1, v)
    wo, wl, tol, ltol = definition(c, hd ** -0.5)
    assert float(tol.max()) < 0.02 * float(wo.min())  # the bound sees a fiftieth of their share
    o, lse, st = run_tree(c)
    off, loff = float(((o.double() - wo).abs() / tol).max()), float(((lse.double() - wl).abs() / ltol).max())
    assert st == 0 and off <= 1 and loff <= 1, (off, loff)
