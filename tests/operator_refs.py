"""Plain 64-bit implementations of the serving operators, row by row, and the error bounds their tests hold the
kernels to.  A rounding to a type is off by at most half a step, finfo.eps / 2 relative to the value."""
import math

import numpy as np
import torch

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


# ------------------------------------------------------------ log probabilities --
def sort_order(x):
    """Ids in the order (value descending, id ascending), NaN first."""
    x = np.asarray(x, dtype=np.float64)
    key = np.where(np.isnan(x), np.inf, x)
    return np.lexsort((np.arange(len(x)), -key, ~np.isnan(x)))


def logprobs_row(x, target, n_top):
    """(logprob, rank, entropy, lse, top ids, top logprobs) of one row (float64 numpy)."""
    n = len(x)
    order = sort_order(x)
    top = order[:n_top]
    nan, inf = bool(np.isnan(x).any()), bool(np.isposinf(x).any())
    has = 0 <= target < n
    rank = int(np.nonzero(order == target)[0][0]) if has and not nan else -1
    if nan or inf:
        q = float("nan")
        return (0.0 if target == -1 else q), rank, q, q, top, np.full(n_top, q)
    m = x.max()
    if m == -math.inf:
        lp = np.full(n, -math.inf)
        lse, ent = -math.inf, 0.0
    else:
        ln_sum = math.log(np.exp(x - m).sum())
        lse = m + ln_sum
        lp = (x - m) - ln_sum  # where m is the type's lowest value, lse has no digits left for the logarithm
        p = np.exp(lp)
        ent = -float((p * np.where(p > 0, lp, 0.0)).sum())
    return (lp[target] if has else (0.0 if target == -1 else float("nan"))), rank, ent, lse, top, lp[top]


def sum_bound(terms):
    """Relative error of a sum of `terms` positive fp32 terms in one accumulator, each an exponential good to 2^-21
    (2^-22 of the instruction and the rounding of its argument)."""
    return terms * 2.0 ** -24 + 2.0 ** -21


# ------------------------------------------------------------------ batch plans --
def plan(cached, fresh, table, free, head, page, parents=None, words=0, n_rows=None):
    """The plan of a batch, request by request.  table is extended in place."""
    R = len(cached)
    cu, lens, granted, slots, pos, masks = [0], [], [], [], [], []
    left, refused_before, taken = len(free) - head, False, 0
    need_so_far = 0
    for r in range(R):
        c, f = int(cached[r]), int(fresh[r])
        if c < 0 or f < 0 or f > 1 << 24:
            cu.append(cu[-1])
            lens.append(c)
            granted.append(0)
            continue
        held, want = -(-c // page), -(-(c + f) // page)
        fits = want <= table.shape[1]
        need = want - held if fits else 0
        need_so_far += need
        ok = fits and (need == 0 or need_so_far <= left)
        if ok:
            for i in range(need):
                table[r, held + i] = free[head + need_so_far - need + i]
            taken += need
        par = None if parents is None else parents[cu[-1]:cu[-1] + f]
        bits = []
        for j in range(f):
            at = c + j
            s = int(table[r, at // page]) * page + at % page if ok and table[r, at // page] >= 0 else -1
            slots.append(s)
            if par is None:
                b = (1 << (j + 1)) - 1
            else:
                p = int(par[j])
                b = (bits[p] if 0 <= p < j else 0) | 1 << j
            bits.append(b)
            pos.append(c + (j if par is None else bin(b).count("1") - 1))
            if words:
                w = [(b >> 32 * i) & 0xFFFFFFFF if j < 32 * words else 0 for i in range(words)]
                masks.append(w)
        cu.append(cu[-1] + f)
        lens.append(c + f if ok else c)
        granted.append(int(ok))
    return dict(cu=cu, lens=lens, granted=granted, free_head=head + taken, slots=slots, positions=pos, masks=masks)


# ------------------------------------------------------ norm, rotation and append --
def norm_rope(x, heads, kv_heads, hd, positions, base, gq=None, gk=None, eps=1e-6):
    """(q, k, v) in float64 and the bound's scale for q and k: |the two factors| summed, per element."""
    rows = x.shape[0]
    x = x.reshape(rows, heads + 2 * kv_heads, hd).astype(np.float64)
    qk = x[:, :heads + kv_heads].copy()
    if gq is not None:
        inv = 1.0 / np.sqrt((qk ** 2).mean(-1, keepdims=True) + eps)
        g = np.concatenate([np.broadcast_to(gq, (heads, hd)), np.broadcast_to(gk, (kv_heads, hd))])
        qk = qk * inv * g
    ang = np.asarray(positions, dtype=np.float64)[:, None] * base ** (-np.arange(hd // 2) * 2.0 / hd)
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    a, b = qk[..., :hd // 2], qk[..., hd // 2:]
    y = np.concatenate([a * c - b * s, b * c + a * s], -1)
    size = np.concatenate([np.abs(a) + np.abs(b)] * 2, -1)
    return y[:, :heads], y[:, heads:], x[:, heads + kv_heads:], size[:, :heads], size[:, heads:]


# --------------------------------------------------------------- tree attention --
def tree_attention(q, pool, table, ctx, cu, masks, scale, dtype):
    """(out, lse, bound on out, bound on lse), float64, of the valid rows; rows outside every request are NaN.
    q [rows, H, hd], pool [pages, 2, Hk, P, hd] float64, masks a boolean [rows, nodes] or None (earlier nodes)."""
    rows, H, hd = q.shape
    P, Hk = pool.shape[3], pool.shape[2]
    G = H // Hk
    out = np.full((rows, H, hd), np.nan)
    lse = np.full((rows, H), np.nan)
    tol, ltol = np.zeros((rows, H, hd)), np.zeros((rows, H))
    half = HALF_STEP[dtype]
    for r in range(len(ctx)):
        n = cu[r + 1] - cu[r]
        pos = np.arange(ctx[r] + n)
        pages = table[r][pos // P] if len(pos) else np.zeros(0, int)
        good = (pages >= 0) & (pages < pool.shape[0])
        for i in range(n):
            node = pos - ctx[r]
            if masks is None:
                see = node <= i
            else:
                see = (node < 0) | masks[cu[r] + i][np.clip(node, 0, None)]
            see = see & good
            kv = pool[pages[see], :, :, pos[see] % P]  # [keys, 2, Hk, hd]
            for h in range(H):
                k, v = kv[:, 0, h // G], kv[:, 1, h // G]
                if not len(k):
                    out[cu[r] + i, h], lse[cu[r] + i, h] = 0.0, -math.inf
                    continue
                x = q[cu[r] + i, h]
                s = scale * (k @ x)
                m = s.max()
                e = np.exp(s - m)
                p = e / e.sum()
                out[cu[r] + i, h] = p @ v
                lse[cu[r] + i, h] = m + math.log(e.sum())
                # scores: fp32 sums of hd products, the scale and the exponent's argument; sums of len(k) terms
                ds = ((hd + 4) * 2.0 ** -24 * scale * (np.abs(k) @ np.abs(x))).max() + 2.0 ** -22 * np.abs(s).max()
                rel = 2 * ds + len(k) * 2.0 ** -23 + 2.0 ** -19
                # each probability is rounded once to the type, and the result once
                # (denormal probabilities of fp16: off by at most half of 2^-24 of the largest)
                tiny = len(k) * 2.0 ** -25 if dtype == torch.float16 else 0.0
                tol[cu[r] + i, h] = ((half + rel) * (p @ np.abs(v)) + half * np.abs(p @ v)
                                     + tiny * np.abs(v).max() / e.sum() + 1e-7)
                ltol[cu[r] + i, h] = ds + len(k) * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -23 * abs(lse[cu[r] + i, h])
    return out, lse, tol, ltol
