"""The operators of serving with a tree of drafts, as measured work: cases, inputs, a plain form of each, the
framework's calls, and a 64-bit definition.

Four operators, in the order a serving step uses them: the batch plan (pages, slots, positions and tree masks from
request lengths), the per-head norm with rotation and cache append, attention of draft trees over the paged cache,
and the log probabilities of the head's logits.  A case is a dict with "op" and the sizes of one call.

The cache is one pool of pages, [n_pages, 2 (keys, values), kv heads, page tokens, head width].
"""
import math
import random

import torch

own = False  # True: run() makes the framework's calls; False: the plain form

DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"fp32": 4, "fp16": 2, "bf16": 2}


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one lane's logits at a draft position: the alternatives that open a tree's next level (latency)
        dict(name="logprobs one row", op="logprobs", rows=1, vocab=50257, dtype="fp32", top=8),
        # a decode step of 64 lanes with the alternatives of each token reported
        dict(name="logprobs 64 lanes", op="logprobs", rows=64, vocab=50257, dtype="fp32", top=5),
        # scoring of a long prompt with a large vocabulary in half width: the largest
        dict(name="logprobs scoring", op="logprobs", rows=1000, vocab=131072, dtype="bf16", top=20),
        # one token for each of 64 lanes: the plan of an ordinary decode step (latency)
        dict(name="plan decode", op="plan", requests=64, most=1, context=4000, page=64, tree=False),
        # draft trees of up to 64 nodes for 200 requests, short pages
        dict(name="plan trees", op="plan", requests=200, most=64, context=9000, page=16, tree=True),
        # 64 lanes' single tokens, shared key heads, both norms (latency)
        dict(name="norm-rope decode", op="norm_rope", rows=64, heads=32, kv_heads=8, hd=128, din="bf16", dcache="bf16",
             norm=True, page=64),
        # an odd number of rows of a narrow model, fp16 throughout, rotation alone
        dict(name="norm-rope narrow", op="norm_rope", rows=1021, heads=20, kv_heads=4, hd=64, din="fp16",
             dcache="fp16", norm=False, page=32),
        # the prompts of a batch from fp32 projections, every head with its own keys: the largest
        dict(name="norm-rope prompts", op="norm_rope", rows=8190, heads=16, kv_heads=16, hd=128, din="fp32",
             dcache="fp16", norm=True, page=64),
        # the first verification of a short prompt: one lane, seven nodes (latency)
        dict(name="tree one lane", op="tree", requests=1, nodes=7, context=100, heads=16, kv_heads=16, hd=64,
             dtype="fp16", page=64, ragged=False),
        # single tokens of 64 lanes, ragged contexts, shared key heads
        dict(name="tree single tokens", op="tree", requests=64, nodes=1, context=4000, heads=32, kv_heads=8, hd=128,
             dtype="bf16", page=16, ragged=True),
        # trees of 32 nodes for 16 lanes, shared key heads
        dict(name="tree 16 lanes", op="tree", requests=16, nodes=32, context=8190, heads=32, kv_heads=8, hd=128,
             dtype="bf16", page=64, ragged=True),
        # two lanes with long contexts, every head with its own keys: the largest
        dict(name="tree long contexts", op="tree", requests=2, nodes=48, context=60001, heads=16, kv_heads=16, hd=128,
             dtype="fp16", page=64, ragged=False),
    ]


def _spread(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng: random.Random):
    op = rng.choice(["logprobs", "plan", "norm_rope", "tree"])
    if op == "logprobs":
        dtype = rng.choice(["fp32", "bf16", "fp16"])
        vocab = _spread(rng, 500, 131072)
        most = min(4096, 131_000_000 // vocab // (SIZE[dtype] // 2))
        return dict(op=op, rows=_spread(rng, 1, most), vocab=vocab, dtype=dtype, top=rng.randint(1, 32))
    if op == "plan":
        tree = rng.random() < 0.5
        return dict(op=op, requests=_spread(rng, 1, 200), most=_spread(rng, 1, 64 if tree else 300),
                    context=_spread(rng, 10, 9000), page=rng.choice([16, 32, 64]), tree=tree)
    kv_heads, group = rng.choice([(1, 8), (2, 4), (4, 5), (8, 4), (8, 1), (16, 1)])
    hd = rng.choice([32, 64, 128])
    if op == "norm_rope":
        width = (kv_heads * group + 2 * kv_heads) * hd
        return dict(op=op, rows=_spread(rng, 1, min(8190, 50_000_000 // width)), heads=kv_heads * group,
                    kv_heads=kv_heads, hd=hd, din=rng.choice(["fp32", "bf16", "fp16"]),
                    dcache=rng.choice(["fp16", "bf16"]), norm=rng.random() < 0.5, page=rng.choice([16, 32, 64, 128]))
    requests = _spread(rng, 1, 64)
    nodes = _spread(rng, 1, 64)
    most = 60001 * 2 * 16 * 128 // (requests * kv_heads * hd)
    most = min(most, 60001 * 2 * 48 * 16 // (requests * nodes * kv_heads * group))
    return dict(op=op, requests=requests, nodes=nodes, context=_spread(rng, 1, max(2, min(32000, most // 2))),
                heads=kv_heads * group, kv_heads=kv_heads, hd=hd, dtype=rng.choice(["fp16", "bf16"]),
                page=rng.choice([16, 32, 64, 128]), ragged=rng.random() < 0.7)


# ----------------------------------------------------------------- inputs --
def _lengths(case):
    """Request lengths of a plan or attention case (the case alone sets them): (tokens in the cache, new tokens)."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    R = case["requests"]
    if case["op"] == "plan":
        old = [r.randint(0, case["context"]) for _ in range(R)]
        new = [r.randint(max(1, case["most"] // 2), case["most"]) for _ in range(R)]
    elif case["ragged"]:
        old = [r.randint(case["context"] // 8, case["context"]) for _ in range(R)]
        new = [r.randint((case["nodes"] + 1) // 2, case["nodes"]) for _ in range(R)]
    else:
        old, new = [case["context"]] * R, [case["nodes"]] * R
    return old, new


def _cu(counts):
    return [0] + list(torch.tensor(counts).cumsum(0).tolist())


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = random.Random(seed)
    dev = "cuda"

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).to(dtype)

    def ints(v, dtype=torch.int32):
        return torch.tensor(v, dtype=dtype, device=dev)

    def tree_parents(new, r):
        """Random draft trees, nodes in the order they were drafted: each one's parent (-1: hangs on the context)."""
        out = []
        for n in new:
            for j in range(n):
                out.append(-1 if j == 0 else r.randint(max(0, j // 2 - 2), j - 1))
        return out

    def mask_words(new, parents, words):
        """Each node's visible nodes (its ancestors and itself) as 32-bit words, as signed ints."""
        out, at = [], 0
        for n in new:
            bits = []
            for j in range(n):
                p = parents[at + j]
                bits.append((bits[p] if p >= 0 else 0) | 1 << j)
            for b in bits:
                for w in range(words):
                    v = b >> 32 * w & 0xFFFFFFFF
                    out.append(v - (1 << 32) if v >> 31 else v)
            at += n
        return out

    s = dict(case)
    if case["op"] == "logprobs":
        s["logits"] = (normal(case["rows"], case["vocab"]) * 3.0).to(DT[case["dtype"]])
        t = torch.randint(0, case["vocab"], (case["rows"],), generator=g, device=dev)
        # half of the targets are the most likely token, as in a scored text that the model knows
        best = s["logits"].float().argmax(1)
        s["targets"] = torch.where(torch.rand(case["rows"], generator=g, device=dev) < 0.5, best, t).int()
        return s
    page = case["page"]
    if case["op"] == "norm_rope":
        rows, H, Hk, hd = case["rows"], case["heads"], case["kv_heads"], case["hd"]
        n_pages = (rows + page - 1) // page + 3
        s["pool"] = normal(n_pages, 2, Hk, page, hd, dtype=DT[case["dcache"]])
        s["qkv"] = normal(rows, (H + 2 * Hk) * hd, dtype=DT[case["din"]])
        s["gq"], s["gk"] = (1 + 0.1 * normal(hd), 1 + 0.1 * normal(hd)) if case["norm"] else (None, None)
        s["slots"] = torch.randperm(n_pages * page, generator=g, device=dev)[:rows].contiguous()
        s["length"] = 16384
        s["positions"] = torch.randint(0, s["length"], (rows,), generator=g, device=dev).int()
        # the table of (cos, sin) that a program makes once: angles in 64 bits
        ang = torch.arange(s["length"], dtype=torch.float64, device=dev)[:, None] * \
            1e4 ** (-torch.arange(hd // 2, dtype=torch.float64, device=dev) * 2 / hd)
        s["rope"] = torch.stack([ang.cos(), ang.sin()], -1).float()
        s["q"] = torch.zeros(rows, H, hd, dtype=DT[case["dcache"]], device=dev)
        return s
    old, new = _lengths(case)
    R = case["requests"]
    s["cached"], s["fresh"] = ints(old), ints(new)
    s["cu"] = ints(_cu(new))
    s["total"] = sum(new)
    parents = tree_parents(new, r)
    max_pages = max((o + n + page - 1) // page for o, n in zip(old, new)) + 1
    n_pages = sum((o + n + page - 1) // page for o, n in zip(old, new)) + 8
    ids = torch.randperm(n_pages, generator=g, device=dev).int()
    if case["op"] == "plan":
        held = [-(-o // page) for o in old]
        table = torch.full((R, max_pages), -1, dtype=torch.int32, device=dev)
        col = torch.arange(max_pages, device=dev)
        table[col[None, :] < ints(held)[:, None]] = ids[:sum(held)]
        # with trees the pool has run low: the last requests that need a page are refused
        left = ids[sum(held):]
        s["table"], s["free"] = table, left[:len(left) * 9 // 10 if case["tree"] else len(left)].contiguous()
        s["free_head"] = ints([1])  # the first free page is gone already
        s["parents"] = ints(parents) if case["tree"] else None
        s["words"] = (case["most"] + 31) // 32 if case["tree"] else 0
        return s
    H, Hk, hd = case["heads"], case["kv_heads"], case["hd"]
    dt = DT[case["dtype"]]
    held = [(o + n + page - 1) // page for o, n in zip(old, new)]
    table = torch.full((R, max_pages), -1, dtype=torch.int32, device=dev)
    col = torch.arange(max_pages, device=dev)
    table[col[None, :] < ints(held)[:, None]] = ids[:sum(held)]
    s["table"] = table
    s["pool"] = torch.empty(n_pages, 2, Hk, page, hd, dtype=dt, device=dev).normal_(generator=g)
    s["q"] = normal(s["total"], H, hd, dtype=dt)
    words = (case["nodes"] + 31) // 32
    s["masks"] = ints(mask_words(new, parents, words)).view(s["total"], words)
    return s


# -------------------------------------------------------------- one pass --
def run(s):
    if own:
        import dynamic_depth_b200 as T
        if s["op"] == "logprobs":
            o = T.token_logprobs(s["logits"], s["targets"], n_top=s["top"])
            return dict(logprob=o.logprob, rank=o.rank, entropy=o.entropy, lse=o.lse, top_ids=o.top_ids,
                        top_logprobs=o.top_logprobs)
        if s["op"] == "plan":
            o = T.plan_batch(s["cached"], s["fresh"], s["table"], s["free"], s["free_head"], page_tokens=s["page"],
                             n_rows=s["total"], parents=s["parents"], mask_words=s["words"])
            d = dict(cu=o.cu, lens=o.lens, granted=o.granted, free_head=o.free_head, slots=o.slots,
                     positions=o.positions, table=s["table"])
            return dict(d, masks=o.masks) if s["words"] else d
        if s["op"] == "norm_rope":
            q = T.norm_rope_append(s["qkv"], s["heads"], s["pool"], s["slots"], s["positions"], s["rope"],
                                   q_gain=s["gq"], k_gain=s["gk"], eps=1e-6, q_out=s["q"])
            return dict(q=q, pool=s["pool"])
        out, lse = T.tree_attention(s["q"], s["pool"], s["table"], s["cached"], s["cu"], max_nodes=s["nodes"],
                                    masks=s["masks"], return_lse=True)
        return dict(out=out, lse=lse)
    return {"logprobs": _plain_logprobs, "plan": _plain_plan, "norm_rope": _plain_norm_rope,
            "tree": _plain_tree}[s["op"]](s)


# -------------------------------------------------------------- plain forms --
def _plain_logprobs(s):
    x, t = s["logits"].float(), s["targets"].long()[:, None]
    m = x.max(1, keepdim=True).values
    e = torch.exp(x - m)
    S = e.double().sum(1, keepdim=True)
    lnS = torch.log(S)
    xt = x.gather(1, t)
    entropy = lnS - ((x - m) * e).double().sum(1, keepdim=True) / S
    ids = torch.arange(x.shape[1], device=x.device)
    rank = ((x > xt) | ((x == xt) & (ids < t))).sum(1)
    best, at = torch.sort(x, dim=1, descending=True, stable=True)
    best, at = best[:, :s["top"]], at[:, :s["top"]]
    return dict(logprob=((xt - m).double() - lnS).float()[:, 0], rank=rank.int(), entropy=entropy.float()[:, 0],
                lse=(m.double() + lnS).float()[:, 0], top_ids=at.int(),
                top_logprobs=((best - m).double() - lnS).float())


def _twice(m):
    return ((m @ m) > 0).float()


def _plain_plan(s):
    c, f, P, R, n = s["cached"].long(), s["fresh"].long(), s["page"], s["requests"], s["total"]
    dev, table = c.device, s["table"]
    held, want = (c + P - 1) // P, (c + f + P - 1) // P
    need = want - held
    take = need.cumsum(0)
    head = s["free_head"].long()
    granted = ((need == 0) | (head + take <= s["free"].numel())) & (want <= table.shape[1])
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), f.cumsum(0)])
    # the new pages of each request, in order, from the front of the free list
    col = torch.arange(table.shape[1], device=dev)[None, :]
    src = head + (take - need)[:, None] + col - held[:, None]
    new_page = (col >= held[:, None]) & (col < want[:, None]) & granted[:, None]
    table.copy_(torch.where(new_page, s["free"][src.clamp(0, s["free"].numel() - 1)], table))
    req = torch.repeat_interleave(torch.arange(R, device=dev), f, output_size=n)
    j = torch.arange(n, device=dev) - cu[req]
    at = c[req] + j
    page = table[req, (at // P).clamp(max=table.shape[1] - 1)].long()
    slots = torch.where(granted[req] & (page >= 0), page * P + at % P, torch.full_like(at, -1))
    out = dict(cu=cu.int(), lens=torch.where(granted, c + f, c).int(), granted=granted.int(),
               free_head=(head + (need * granted).sum()).int(), slots=slots, table=table)
    if not s["words"]:
        return dict(out, positions=at.int())
    N = 32 * s["words"]
    par = s["parents"].long()
    reach = torch.eye(N, device=dev).repeat(R, 1, 1)
    reach[req, j, torch.where(par >= 0, par, j)] = 1.0
    reach = _twice(_twice(_twice(_twice(_twice(_twice(reach))))))  # paths of up to 64 steps
    rows = reach[req, j]
    bits = (rows.view(n, s["words"], 32).long() << torch.arange(32, device=dev)).sum(-1)
    masks = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).int()
    return dict(out, positions=(c[req] + rows.sum(1).long() - 1).int(), masks=masks)


def _plain_norm_rope(s):
    H, Hk, hd, rows = s["heads"], s["kv_heads"], s["hd"], s["rows"]
    x = s["qkv"].float().view(rows, H + 2 * Hk, hd)
    q, k, v = x[:, :H], x[:, H:H + Hk], x[:, H + Hk:]
    if s["gq"] is not None:
        q = q * torch.rsqrt((q * q).mean(-1, keepdim=True) + 1e-6) * s["gq"]
        k = k * torch.rsqrt((k * k).mean(-1, keepdim=True) + 1e-6) * s["gk"]
    cs = s["rope"][s["positions"].long()]
    c, n = cs[:, None, :, 0], cs[:, None, :, 1]

    def turn(y):
        a, b = y[..., :hd // 2], y[..., hd // 2:]
        return torch.cat([a * c - b * n, b * c + a * n], -1)
    page, off = s["slots"] // s["page"], s["slots"] % s["page"]
    s["pool"][page, 0, :, off] = turn(k).to(s["pool"].dtype)
    s["pool"][page, 1, :, off] = v.to(s["pool"].dtype)
    s["q"].copy_(turn(q).to(s["q"].dtype))
    return dict(q=s["q"], pool=s["pool"])


def _plain_tree(s):
    R, N, H, Hk, hd, P, n = s["requests"], s["nodes"], s["heads"], s["kv_heads"], s["hd"], s["page"], s["total"]
    dev, G = s["q"].device, s["heads"] // s["kv_heads"]
    pages = s["table"].clamp(min=0).long()
    T = pages.shape[1] * P
    kv = s["pool"][pages]  # [R, pages, 2, Hk, P, hd]
    k = kv[:, :, 0].permute(0, 2, 1, 3, 4).reshape(R, Hk, T, hd).float()
    v = kv[:, :, 1].permute(0, 2, 1, 3, 4).reshape(R, Hk, T, hd).float()
    f = s["fresh"].long()
    req = torch.repeat_interleave(torch.arange(R, device=dev), f, output_size=n)
    j = torch.arange(n, device=dev) - s["cu"].long()[req]
    q = torch.zeros(R, N, H, hd, device=dev)
    q[req, j] = s["q"].float()
    q = q.view(R, N, Hk, G, hd).permute(0, 2, 1, 3, 4).reshape(R, Hk, N * G, hd)
    bits = (s["masks"][:, :, None] >> torch.arange(32, device=dev)) & 1
    seen = torch.zeros(R, N, N, dtype=torch.bool, device=dev)
    seen[req, j] = bits.reshape(n, -1)[:, :N] > 0
    at = torch.arange(T, device=dev)[None, :] - s["cached"].long()[:, None]  # node index of each position
    node = torch.where(at >= 0, at, torch.zeros_like(at)).clamp(max=N - 1)
    ok = torch.gather(seen, 2, node[:, None, :].expand(R, N, T)) & (at >= 0)[:, None] & (at < f[:, None])[:, None]
    ok = (ok | (at < 0)[:, None]).repeat_interleave(G, 1)[:, None]  # [R, 1, N * G, T]
    sc = torch.matmul(q, k.transpose(-1, -2)) * hd ** -0.5
    sc = sc.masked_fill(~ok, -math.inf)
    m = sc.max(-1, keepdim=True).values
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = torch.exp(sc - m)
    z = e.sum(-1, keepdim=True)
    o = torch.matmul(e, v) / torch.where(z == 0, torch.ones_like(z), z)
    lse = (m + torch.log(z))[..., 0]
    o = o.view(R, Hk, N, G, hd).permute(0, 2, 1, 3, 4).reshape(R, N, H, hd)[req, j]
    lse = lse.view(R, Hk, N, G).permute(0, 2, 1, 3).reshape(R, N, H)[req, j]
    return dict(out=o.to(s["q"].dtype), lse=lse)


# ---------------------------------------------------------------- the work --
def work(case):
    if case["op"] == "logprobs":
        n, V = case["rows"], case["vocab"]
        return dict(bytes=n * V * SIZE[case["dtype"]] + n * (20 + 8 * case["top"]), flops=6 * n * V)
    if case["op"] == "norm_rope":
        width = (case["heads"] + 2 * case["kv_heads"]) * case["hd"]
        moved = case["rows"] * width * (SIZE[case["din"]] + 2) + case["rows"] * (12 + 4 * case["hd"])
        return dict(bytes=moved, flops=8 * case["rows"] * width)
    old, new = _lengths(case)
    if case["op"] == "plan":
        R, n = case["requests"], sum(new)
        pages = sum(-(-(o + f) // case["page"]) - -(-o // case["page"]) for o, f in zip(old, new))
        per = 12 + (4 + 4 * ((case["most"] + 31) // 32) if case["tree"] else 0)
        return dict(bytes=24 * R + 12 * pages + n * per, flops=4 * n)
    keys = sum(o + f for o, f in zip(old, new))
    pairs = sum(f * (o + f) for o, f in zip(old, new))
    moved = keys * 2 * case["kv_heads"] * case["hd"] * 2 + sum(new) * case["heads"] * (4 * case["hd"] + 4)
    return dict(bytes=moved, flops=4 * case["hd"] * case["heads"] * pairs)


# ------------------------------------------------------- the definitions --
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "logprobs":
        outs = []
        for x, t in zip(s["logits"].split(64), s["targets"].long().split(64)):
            lp = torch.log_softmax(x.double(), 1)
            p = lp.exp()
            top = lp.topk(case["top"], 1).values
            lse = torch.logsumexp(x.double(), 1)
            outs.append((lp.gather(1, t[:, None])[:, 0], -(p * lp).sum(1), lse, top))
        lp, ent, lse, top = (torch.cat(v) for v in zip(*outs))
        return dict(logprob=lp, rank=None, entropy=ent, lse=lse, top_ids=None, top_logprobs=top)
    if case["op"] == "plan":
        return None
    if case["op"] == "norm_rope":
        H, Hk, hd, P = case["heads"], case["kv_heads"], case["hd"], case["page"]
        x = s["qkv"].double().view(case["rows"], H + 2 * Hk, hd)
        if case["norm"]:
            g = torch.cat([s["gq"].double().expand(H, hd), s["gk"].double().expand(Hk, hd)])
            qk = x[:, :H + Hk]
            qk = qk / torch.sqrt(qk.pow(2).sum(-1, keepdim=True) / hd + 1e-6) * g
        else:
            qk = x[:, :H + Hk]
        freq = torch.pow(torch.tensor(1e4, dtype=torch.float64), -torch.arange(0, hd, 2, dtype=torch.float64) / hd)
        z = torch.polar(torch.ones(1, dtype=torch.float64, device="cuda"),
                        s["positions"].double()[:, None] * freq.cuda()[None, :])
        y = torch.view_as_real(torch.complex(qk[..., :hd // 2], qk[..., hd // 2:]) * z[:, None, :])
        y = torch.cat([y[..., 0], y[..., 1]], -1)
        flat = s["pool"].double().permute(0, 3, 1, 2, 4).reshape(-1, 2, Hk, hd)  # by slot
        flat[s["slots"], 0], flat[s["slots"], 1] = y[:, H:], x[:, H + Hk:]
        return dict(q=y[:, :H], pool=flat.view(-1, P, 2, Hk, hd).permute(0, 2, 3, 1, 4).contiguous())
    out, lse = [], []
    old, new = s["cached"].tolist(), s["fresh"].tolist()
    G, at = case["heads"] // case["kv_heads"], 0
    for r, (c, n) in enumerate(zip(old, new)):
        kv = torch.cat(list(s["pool"][s["table"][r, :(c + n + case["page"] - 1) // case["page"]].long()]), 2)
        k, v = kv[0, :, :c + n].double(), kv[1, :, :c + n].double()
        words = s["masks"][at:at + n].long() & 0xFFFFFFFF
        tree = torch.stack([(words[:, i // 32] >> (i % 32)) & 1 for i in range(n)], 1) == 0
        hidden = torch.cat([torch.zeros(n, c, dtype=torch.bool, device="cuda"), tree], 1)
        o_h, l_h = [], []
        for h in range(case["heads"]):
            w = s["q"][at:at + n, h].double() @ k[h // G].T / math.sqrt(case["hd"])
            w[hidden] = -math.inf
            l_h.append(torch.logsumexp(w, 1))
            o_h.append(torch.softmax(w, 1) @ v[h // G])
        out.append(torch.stack(o_h, 1))
        lse.append(torch.stack(l_h, 1))
        at += n
    return dict(out=torch.cat(out), lse=torch.cat(lse))
