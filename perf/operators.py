"""Serving operators for a batch of requests over one page pool: attention of
a batch that shares a long prefix, the pages of its cache (fork, reserve,
write, compact), and the verification of drafted tokens.

`run` computes an operator in its plain form with elementary torch
operations, or, when `own` is set, through the framework's calls. The cases'
sizes are the decode attention's of this repository (16 query heads on 2
key/value heads of 128, pages of 64 positions, contexts of 32768, 10
full-attention layers), with other head counts and sizes around them.

Cache state (all ops): pools 16-bit [n_phys][n_kv][64][D]; table int32
[n_slots][max_blocks]; lens int32 [n_slots]; refs int32 [n_phys], 0 = free.
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = 64
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


def device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def ceil_div(a, b):
    return -(-a // b)


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # two requests of one short system prompt: latency is what counts
        dict(name="attn-small", op="attn", slots=2, T=1, n_q=16, n_kv=2, D=128, prefix=4,
             suffix=50, type="bf16"),
        # a running server: single tokens of 48 requests under an 8K prompt
        dict(name="attn-decode", op="attn", slots=48, T=1, n_q=16, n_kv=2, D=128, prefix=128,
             suffix=777, type="bf16"),
        # no shared part, other heads: drafts of up to 3 tokens, long own contexts
        dict(name="attn-ragged", op="attn", slots=33, T=3, n_q=12, n_kv=4, D=64, prefix=0,
             suffix=5000, type="fp16"),
        # the largest: four drafted tokens of 256 requests under a 32K document
        dict(name="attn-long", op="attn", slots=256, T=4, n_q=16, n_kv=2, D=128, prefix=512,
             suffix=1500, type="bf16"),
        # one layer's step for a few requests: pages taken, rows written
        dict(name="step-small", op="step", slots=8, T=1, layers=1, n_kv=2, D=128, beams=1,
             shared=700, own=300, fresh=False, n_phys=256, short=False, type="bf16"),
        # samples just forked from their prompts take their first step: every
        # slot copies the partly filled page it shares, in all 10 layers
        dict(name="step-forked", op="step", slots=256, T=4, layers=10, n_kv=2, D=128, beams=16,
             shared=4000, own=0, fresh=True, n_phys=2500, short=False, type="bf16"),
        # beams of a few requests reordered
        dict(name="fork-small", op="fork", slots=16, beams=4, shared=2000, own=200, fresh=False,
             n_phys=512),
        # a full server after a verification: reorder, cut and free 1000 slots
        dict(name="fork-large", op="fork", slots=1000, beams=10, shared=16000, own=900,
             fresh=False, n_phys=60001),
        # a fragmented pool of K and V of two layers brought together
        dict(name="compact", op="compact", slots=301, layers=2, n_kv=2, D=128, beams=3,
             shared=700, own=600, fresh=False, n_phys=8192),
        # one request, three drafts, a 32000-token vocabulary
        dict(name="verify-small", op="verify", slots=1, T=3, V=32000, type="fp32", draft="sampled"),
        # a running server with a large vocabulary in bf16
        dict(name="verify-decode", op="verify", slots=64, T=5, V=131072, type="bf16",
             draft="sampled"),
        # many requests, an odd vocabulary, drafts looked up rather than sampled
        dict(name="verify-large", op="verify", slots=256, T=4, V=128001, type="fp32",
             draft="certain"),
    ]


def spread(rng, lo, hi):
    """A whole number in [lo, hi], even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "step", "step", "fork", "compact", "verify", "verify"])
    while True:
        if op == "attn":
            n_q, n_kv = rng.choice([(16, 2), (16, 2), (12, 4), (8, 8), (32, 4), (5, 1), (28, 4)])
            c = dict(op=op, slots=spread(rng, 1, 256), T=rng.choice([1, 1, 1, 2, 3, 4, 5, 8]),
                     n_q=n_q, n_kv=n_kv, D=rng.choice([64, 128, 128]),
                     prefix=rng.choice([0, spread(rng, 1, 512), spread(rng, 1, 512)]),
                     suffix=spread(rng, 1, 6000), type=rng.choice(["bf16", "bf16", "fp16"]))
            if c["T"] * n_q // n_kv > 64:
                continue
        elif op == "step":
            fresh = rng.random() < 0.4
            beams = rng.choice([1, 2, 5, 16])
            c = dict(op=op, slots=spread(rng, 1, 256), T=rng.choice([1, 1, 2, 3, 4, 7]),
                     layers=spread(rng, 1, 10), n_kv=rng.choice([1, 2, 4]),
                     D=rng.choice([64, 128]), beams=beams, shared=spread(rng, 1, 4000),
                     own=0 if fresh else spread(rng, 1, 500), fresh=fresh, n_phys=0,
                     short=rng.random() < 0.2, type=rng.choice(["bf16", "fp16"]))
            c["n_phys"] = pages_in_use(c) + 3 * c["slots"] + rng.randrange(1, 50)
            if c["n_phys"] * c["layers"] * c["n_kv"] * c["D"] > 2500 * 10 * 256:
                continue
        elif op == "fork":
            c = dict(op=op, slots=spread(rng, 1, 1000), beams=rng.choice([1, 2, 4, 10, 31]),
                     shared=spread(rng, 1, 16000), own=spread(rng, 1, 900), fresh=False, n_phys=0)
            c["n_phys"] = pages_in_use(c) + c["slots"] + rng.randrange(1, 5000)
            if c["n_phys"] > 60001:
                continue
        elif op == "compact":
            c = dict(op=op, slots=spread(rng, 1, 301), layers=rng.choice([1, 1, 2, 3]),
                     n_kv=rng.choice([1, 2, 4]), D=rng.choice([64, 128]),
                     beams=rng.choice([1, 3, 8]), shared=spread(rng, 1, 700),
                     own=spread(rng, 1, 600), fresh=False, n_phys=0)
            c["n_phys"] = int(pages_in_use(c) * rng.uniform(1.0, 3.0)) + c["slots"]
            if c["n_phys"] * c["layers"] * c["n_kv"] * c["D"] > 8192 * 2 * 256:
                continue
        else:
            c = dict(op=op, slots=spread(rng, 1, 256), T=rng.choice([1, 2, 3, 4, 5, 8]),
                     V=spread(rng, 100, 200000), type=rng.choice(["fp32", "fp32", "bf16", "fp16"]),
                     draft=rng.choice(["sampled", "sampled", "certain"]))
            if c["slots"] * (c["T"] + 1) * c["V"] * SIZE[c["type"]] > 256 * 5 * 128001 * 4:
                continue
        top = listed()[3]
        if work(c)["flops"] <= work(top)["flops"] and work(c)["bytes"] <= 1.4e9:
            return c


# ------------------------------------------------------------- cache state --
def own_lengths(c):
    """(the tokens of each slot past its group's shared ones, the groups' shared tokens)."""
    n = c["slots"]
    groups = ceil_div(n, c["beams"])
    shared = [max(1, c["shared"] - (37 * g) % max(1, c["shared"] // 2)) for g in range(groups)]
    tails = [0 if c["fresh"] else 1 + int(c["own"] * (i + 0.5) / n) for i in range(n)]
    return tails, shared


def pages_in_use(c):
    tails, shared = own_lengths(c)
    n = 0
    for g, s in enumerate(shared):
        n += ceil_div(s, BLOCK) if c["fresh"] else s // BLOCK
    for i, t in enumerate(tails):
        if not c["fresh"]:
            s = shared[i // c["beams"]]
            n += ceil_div(s + t, BLOCK) - s // BLOCK
    return n


def table_width(c, extra):
    tails, shared = own_lengths(c)
    return ceil_div(max(shared) + max(tails) + extra, BLOCK) + 1


def make_meta(c, seed, extra=0):
    """Table, lens and refs of slots in groups of `beams` that share their
    first pages, at random places of the pool (host arrays). The pool has to
    hold a page a slot more than pages_in_use: the tails' order differs."""
    rng = np.random.RandomState(seed % (1 << 31))
    tails, shared = own_lengths(c)
    tails = [tails[i] for i in rng.permutation(len(tails))]
    pages = rng.permutation(c["n_phys"]).astype(np.int32)
    width = table_width(c, extra)
    table = np.full((c["slots"], width), -1, np.int32)
    lens = np.zeros(c["slots"], np.int32)
    at = 0
    for g, s in enumerate(shared):
        whole = ceil_div(s, BLOCK) if c["fresh"] else s // BLOCK
        common = pages[at:at + whole]
        at += whole
        for i in range(g * c["beams"], min(c["slots"], (g + 1) * c["beams"])):
            n = s + tails[i]
            more = ceil_div(n, BLOCK) - whole
            lens[i] = n
            table[i, :whole] = common
            table[i, whole:whole + more] = pages[at:at + more]
            at += more
    refs = np.bincount(table[table >= 0], minlength=c["n_phys"]).astype(np.int32)
    return table, lens, refs


def gen_for(seed, dev):
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    return g


def normal(shape, dtype, g, dev):
    return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dtype)


def bits(shape, g, dev):
    return torch.randint(-30000, 30000, shape, generator=g, device=dev, dtype=torch.int16)


def on(dev, a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


# ---------------------------------------------------------------- prepare --
def attn_lengths(c):
    """Own positions and new tokens of each slot, the same for every seed: one
    slot in sixteen is idle, the others' lengths crowd toward the short ones."""
    n = c["slots"]
    out = []
    for i in range(n):
        new = 1 + (i * 7 + 3) % c["T"] if i % 3 else c["T"]
        idle = n >= 8 and i % 16 == 5
        tail = max(new, int(c["suffix"] * ((i + 0.5) / n) ** 1.5))
        out.append((0, 0) if idle else (tail, new))
    return out


def prepare_attn(c, seed):
    dev = device()
    g = gen_for(seed, dev)
    rng = np.random.RandomState(seed % (1 << 31))
    pairs = attn_lengths(c)
    pairs = [pairs[i] for i in rng.permutation(len(pairs))]
    P = c["prefix"]
    blocks = [ceil_div(t, BLOCK) for t, _ in pairs]
    n_phys = P + sum(blocks) + 3
    pages = rng.permutation(n_phys).astype(np.int32)
    table = np.full((c["slots"], P + max(blocks)), -1, np.int32)
    lens = np.zeros(c["slots"], np.int32)
    at = P
    for i, (t, new) in enumerate(pairs):
        if new == 0:
            continue
        lens[i] = P * BLOCK + t
        table[i, :P] = pages[:P]
        table[i, P:P + blocks[i]] = pages[at:at + blocks[i]]
        at += blocks[i]
    dt = TYPES[c["type"]]
    cache = (n_phys, c["n_kv"], BLOCK, c["D"])
    # queries a little longer than the keys, as trained heads have them: some
    # rows' softmax is flat, some rows' is not
    q = (normal((c["slots"], c["T"], c["n_q"], c["D"]), torch.float32, g, dev) *
         torch.linspace(0.5, 3.0, c["n_q"], device=dev)[None, None, :, None]).to(dt)
    st = dict(case=c, q=q, k=normal(cache, dt, g, dev), v=normal(cache, dt, g, dev),
              table=on(dev, table), lens=on(dev, lens),
              n_new=on(dev, np.array([p[1] for p in pairs], np.int32)),
              prefix=on(dev, pages[:P]) if P else None)
    if own:
        import bit_moe_expert_histogram_gb300 as m
        st["shape"] = m.make_attn_batch_shape(c["slots"], c["T"], c["n_q"], c["n_kv"], c["D"],
                                              table.shape[1], P, dtype=c["type"])
        st["ws"] = m.alloc_attn_batch_workspace(st["shape"], dev)
        st["o"] = torch.empty_like(q)
    return st


def prepare_pages(c, seed):
    dev = device()
    g = gen_for(seed, dev)
    rng = np.random.RandomState(seed % (1 << 31) ^ 0x5A5A)
    extra = c.get("T", 0) + BLOCK
    table, lens, refs = make_meta(c, seed, extra)
    st = dict(case=c)
    n = c["slots"]
    if c["op"] == "step":
        n_new = np.array([1 + (i * 5 + 1) % c["T"] for i in range(n)], np.int32)
        if n >= 8:
            n_new[rng.permutation(n)[:n // 8]] = 0  # idle slots
        st["n_new"] = on(dev, n_new)
        if c["short"]:  # a pool that runs out: pages held by nobody in the table
            free = np.nonzero(refs == 0)[0]
            refs[free[max(1, len(free) // 20):]] = 1
        # the projections' output, keys and values side by side
        st["kv_new"] = bits((c["layers"], n, c["T"], 2, c["n_kv"], c["D"]), g, dev)
    if c["op"] == "fork":
        parent = np.arange(n, dtype=np.int32)
        for i in range(n):
            if rng.rand() < 0.5:  # another beam of the same request
                lo = i // c["beams"] * c["beams"]
                parent[i] = rng.randint(lo, min(n, lo + c["beams"]))
            if rng.rand() < 0.05:  # done
                parent[i] = -1
        keep = np.where(rng.rand(n) < 0.6, lens[np.maximum(parent, 0)] - rng.randint(0, 5, n),
                        1 << 30)
        keep = np.maximum(keep, 0)
        st["parent"], st["keep"] = on(dev, parent), on(dev, keep.astype(np.int32))
    st["table"], st["lens"], st["refs"] = on(dev, table), on(dev, lens), on(dev, refs)
    if c["op"] != "fork":
        st["pool"] = bits((2 * c["layers"], c["n_phys"], c["n_kv"], BLOCK, c["D"]), g, dev)
    if own:
        import bit_moe_expert_histogram_gb300 as m
        st["shape"] = m.make_cache_shape(n, table.shape[1], c["n_phys"], c.get("n_kv", 1),
                                         c.get("D", 64))
        st["ws"] = m.alloc_cache_workspace(st["shape"], dev)
        st["meta"] = m.CacheMeta(st["table"], st["lens"], st["refs"])
        st["out"] = m.CacheMeta.empty(st["shape"], dev)
        if c["op"] != "fork":
            st["pools"] = m.pool_table(list(st["pool"]))
        if c["op"] == "step":
            st["granted"] = torch.empty_like(st["n_new"])
        if c["op"] == "compact":
            st["n_live"] = torch.empty(1, dtype=torch.int32, device=dev)
    return st


def prepare_verify(c, seed):
    dev = device()
    g = gen_for(seed, dev)
    B, T, V = c["slots"], c["T"], c["V"]
    dt = TYPES[c["type"]]
    p = torch.empty((B, T + 1, V), dtype=dt, device=dev)
    sampled = c["draft"] == "sampled"
    q = torch.empty((B, T, V), dtype=dt, device=dev) if sampled else None
    draft = torch.empty((B, T), dtype=torch.int32, device=dev)
    for b in range(B):  # a slot at a time keeps the scratch small
        logits = torch.randn((T + 1, V), generator=g, device=dev) * 3.0
        p[b] = torch.softmax(logits, -1).to(dt)
        if sampled:
            near = logits[:T] + torch.randn((T, V), generator=g, device=dev) * 0.7
            dq = torch.softmax(near, -1)
            q[b] = dq.to(dt)
            draft[b] = torch.multinomial(dq, 1, generator=g)[:, 0].to(torch.int32)
        else:  # looked up: often the likeliest token
            draft[b] = p[b, :T].float().argmax(-1).to(torch.int32)
    n_draft = torch.full((B,), T, dtype=torch.int32, device=dev)
    if B >= 4:  # some slots have fewer drafts, some none
        n_draft[::4] = torch.randint(0, T + 1, (ceil_div(B, 4),), generator=g, device=dev,
                                     dtype=torch.int32)
    u = torch.rand((B, T + 1), generator=g, device=dev)
    st = dict(case=c, p=p, q=q, draft=draft, n_draft=n_draft, u=u)
    if own:
        import bit_moe_expert_histogram_gb300 as m
        st["shape"] = m.make_verify_shape(B, T, V, dtype=c["type"])
        st["ws"] = m.alloc_verify_workspace(st["shape"], dev)
        st["tokens"] = torch.empty((B, T + 1), dtype=torch.int32, device=dev)
        st["n_acc"] = torch.empty(B, dtype=torch.int32, device=dev)
    return st


def prepare(case, seed):
    if case["op"] == "attn":
        return prepare_attn(case, seed)
    if case["op"] == "verify":
        return prepare_verify(case, seed)
    return prepare_pages(case, seed)


# -------------------------------------------------------------- plain forms --
def plain_attn(st):
    c = st["case"]
    B, T, n_q, n_kv, D = c["slots"], c["T"], c["n_q"], c["n_kv"], c["D"]
    G, P = n_q // n_kv, c["prefix"]
    dev = st["q"].device
    q = st["q"].float().view(B, T, n_kv, G, D) / math.sqrt(D)
    step = torch.arange(T, device=dev)
    pos = st["lens"][:, None] - st["n_new"][:, None] + step  # [B, T]
    pos = torch.where((step < st["n_new"][:, None]) & (pos >= 0), pos, -1)
    # every slot's own positions, gathered through the table
    own_blocks = st["table"][:, P:].clamp(min=0).long()
    W = own_blocks.shape[1] * BLOCK

    def rows(pool, blocks):  # [..., n] blocks -> [..., n_kv, n * BLOCK, D] in 32 bits
        x = pool[blocks].float().movedim(-3, -4)
        return x.reshape(*x.shape[:-3], -1, D)
    rq = q.permute(0, 2, 1, 3, 4).reshape(B, n_kv, T * G, D)
    at = P * BLOCK + torch.arange(W, device=dev)
    s = rq @ rows(st["k"], own_blocks).transpose(-1, -2)  # [B, n_kv, T G, W]
    ok = (at <= pos[:, :, None]).repeat_interleave(G, 1)[:, None]
    s = s.masked_fill(~ok, -math.inf)
    top = s.amax(-1, keepdim=True)
    if P:
        pq = rq.permute(1, 0, 2, 3).reshape(n_kv, B * T * G, D)
        sp = pq @ rows(st["k"], st["prefix"].long()).transpose(-1, -2)
        okp = torch.arange(P * BLOCK, device=dev) <= pos.repeat_interleave(G, 1).view(-1, 1)
        sp.masked_fill_(~okp, -math.inf)
        tp = sp.amax(-1, keepdim=True).view(n_kv, B, T * G, 1).transpose(0, 1)
        top = torch.maximum(top, tp)
    top = torch.where(top.isinf(), torch.zeros_like(top), top)
    e = torch.exp(s - top)
    den = e.sum(-1, keepdim=True)
    num = e @ rows(st["v"], own_blocks)
    if P:
        sp.sub_(top.transpose(0, 1).reshape(n_kv, B * T * G, 1)).exp_()
        den = den + sp.sum(-1, keepdim=True).view(n_kv, B, T * G, 1).transpose(0, 1)
        num = num + (sp @ rows(st["v"], st["prefix"].long())).view(n_kv, B, T * G, D).transpose(0, 1)
    o = torch.where(den > 0, num / den, torch.zeros_like(num))
    return o.view(B, n_kv, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, n_q, D).to(st["q"].dtype)


def plain_step(st):
    c = st["case"]
    table, lens, refs, n_new = st["table"], st["lens"].long(), st["refs"], st["n_new"].long()
    n, width = table.shape
    dev = table.device
    nb0, nb1 = (lens + BLOCK - 1) // BLOCK, (lens + n_new + BLOCK - 1) // BLOCK
    last = table.gather(1, (nb0 - 1).clamp(min=0)[:, None])[:, 0].long()
    shared = (lens % BLOCK > 0) & (n_new > 0) & (refs[last.clamp(min=0)] > 1)
    need = nb1 - nb0 + shared
    before = need.cumsum(0) - need
    free = torch.sort((refs != 0).int(), stable=True).indices  # free pages first, in order
    granted = (before + need <= (refs == 0).sum()) & (nb1 <= width)
    out_n = torch.where(granted, n_new, 0)
    out_len = lens + out_n
    shared = shared & granted
    nb1 = torch.where(granted, nb1, nb0)
    j = torch.arange(width, device=dev)
    copied = shared[:, None] & (j == nb0[:, None] - 1)
    fresh = (j >= nb0[:, None]) & (j < nb1[:, None])
    rank = before[:, None] + torch.where(copied, 0, shared[:, None] + j - nb0[:, None])
    pages = free[rank.clamp(0, refs.numel() - 1)].int()
    out = torch.where(copied | fresh, pages, torch.where(j < nb0[:, None], table, -1))
    out_refs = refs.clone()
    one = torch.ones_like(out)
    out_refs.index_put_((pages.long(),), torch.where(copied | fresh, one, 0), accumulate=True)
    out_refs.index_put_((last.clamp(min=0),), torch.where(shared, -1, 0).int(), accumulate=True)
    # copy-on-write: the filled rows of the shared page, in every pool
    pool = st["pool"]
    src = last[shared]
    dst = free[before[shared]]
    old, new = pool[:, src], pool[:, dst]
    filled = torch.arange(BLOCK, device=dev) < (lens[shared] % BLOCK)[:, None]
    pool[:, dst] = torch.where(filled[None, :, None, :, None], old, new)
    # the new rows
    t = torch.arange(c["T"], device=dev)
    slot, tok = (t < out_n[:, None]).nonzero(as_tuple=True)
    pos = lens[slot] + tok
    page = out[slot, pos // BLOCK].long()
    rows = st["kv_new"][:, slot, tok]  # [layers, m, 2, n_kv, D]
    pool.view(c["layers"], 2, *pool.shape[1:]).permute(0, 2, 4, 1, 3, 5)[:, page, pos % BLOCK] = rows
    return {"table": out, "lens": out_len.int(), "refs": out_refs, "granted": out_n.int(),
            "pool": pool}


def plain_fork(st):
    table, lens, refs = st["table"], st["lens"], st["refs"]
    n, width = table.shape
    parent = st["parent"].long()
    live = (parent >= 0) & (parent < n)
    src = parent.clamp(0, n - 1)
    out_len = torch.where(live, torch.minimum(lens[src], st["keep"]), 0)
    j = torch.arange(width, device=table.device)
    held = j < ((lens + BLOCK - 1) // BLOCK)[:, None]
    holds = j < ((out_len + BLOCK - 1) // BLOCK)[:, None]
    out = torch.where(holds, table[src], -1)
    out_refs = refs.clone()
    one = torch.ones_like(out)
    out_refs.index_put_((out.clamp(min=0).long(),), torch.where(holds, one, 0), accumulate=True)
    out_refs.index_put_((table.clamp(min=0).long(),), torch.where(held, -one, 0), accumulate=True)
    return {"table": out, "lens": out_len, "refs": out_refs}


def plain_compact(st):
    table, lens, refs, pool = st["table"], st["lens"], st["refs"], st["pool"]
    idx = torch.arange(refs.numel(), device=refs.device)
    live = refs > 0
    n_live = live.sum()
    src = (live & (idx >= n_live)).nonzero()[:, 0]
    dst = (~live & (idx < n_live)).nonzero()[:, 0]
    move = idx.clone()
    move[src] = dst
    pool[:, dst] = pool[:, src]
    held = torch.arange(table.shape[1], device=refs.device) < ((lens + BLOCK - 1) // BLOCK)[:, None]
    out = torch.where(held, move[table.clamp(min=0).long()].int(), -1)
    out_refs = refs.clone()
    out_refs[dst] = refs[src]
    out_refs = torch.where(idx < n_live, out_refs, 0)
    return {"table": out, "lens": lens.clone(), "refs": out_refs, "n_live": n_live.int().view(1),
            "pool": pool}


def plain_verify(st):
    p, q, draft, u = st["p"], st["q"], st["draft"].long(), st["u"].double()
    B, T1, V = p.shape
    T = T1 - 1
    step = torch.arange(T, device=p.device)
    px = p[:, :T].gather(2, draft[:, :, None])[:, :, 0].double()
    qx = q.gather(2, draft[:, :, None])[:, :, 0].double() if q is not None else torch.ones_like(px)
    ok = (u[:, :T] * qx < px) & (step < st["n_draft"][:, None])
    n_acc = ok.long().cumprod(1).sum(1)
    b = torch.arange(B, device=p.device)
    rejected = n_acc < st["n_draft"]
    row = p[b, n_acc].double()
    at = n_acc.clamp(max=T - 1)
    if q is not None:
        w = row - q[b, at].double()
    else:
        w = row.scatter(1, draft[b, at][:, None], 0.0)
    w = torch.where((w > 0) & (w < math.inf), w, 0.0)
    w = torch.where((rejected & (w.sum(1) > 0))[:, None], w, torch.where((row > 0) & (row < math.inf), row, 0.0))
    cum = w.cumsum(1)
    token = (cum <= (u[:, T] * cum[:, -1])[:, None]).sum(1)
    lastw = V - 1 - (w.flip(1) > 0).int().argmax(1)
    token = torch.where(cum[:, -1] > 0, torch.minimum(token, lastw), -1)
    grid = torch.arange(T1, device=p.device)
    kept = torch.nn.functional.pad(draft, (0, 1), value=-1)
    tokens = torch.where(grid < n_acc[:, None], kept, torch.where(grid == n_acc[:, None], token[:, None], -1))
    return {"tokens": tokens.int(), "n_acc": n_acc.int()}


PLAIN = dict(attn=plain_attn, step=plain_step, fork=plain_fork, compact=plain_compact,
             verify=plain_verify)


# --------------------------------------------------------------- own forms --
def own_attn(m, st):
    m.moe_attn_batch(st["shape"], st["q"], st["k"], st["v"], st["table"], st["lens"], st["o"],
                     st["ws"], n_new=st["n_new"], prefix=st["prefix"])
    return st["o"]


def own_step(m, st):
    m.moe_cache_reserve(st["shape"], st["meta"], st["n_new"], st["out"], st["granted"],
                        st["pools"], st["ws"])
    pool, kv = st["pool"], st["kv_new"]
    for layer in range(st["case"]["layers"]):  # as the layers of a step call it
        m.moe_cache_write(st["shape"], st["out"], st["granted"], kv[layer, :, :, 0],
                          kv[layer, :, :, 1], pool[2 * layer], pool[2 * layer + 1], st["ws"])
    out = st["out"]
    return {"table": out.table, "lens": out.lens, "refs": out.refs, "granted": st["granted"],
            "pool": pool}


def own_fork(m, st):
    out = st["out"]
    m.moe_cache_fork(st["shape"], st["meta"], st["parent"], out, st["ws"], keep=st["keep"])
    return {"table": out.table, "lens": out.lens, "refs": out.refs}


def own_compact(m, st):
    out = st["out"]
    m.moe_cache_compact(st["shape"], st["meta"], out, st["n_live"], st["pools"], st["ws"])
    return {"table": out.table, "lens": out.lens, "refs": out.refs, "n_live": st["n_live"],
            "pool": st["pool"]}


def own_verify(m, st):
    m.moe_verify_drafts(st["shape"], st["p"], st["q"], st["draft"], st["n_draft"], st["u"],
                        st["tokens"], st["n_acc"], st["ws"])
    return {"tokens": st["tokens"], "n_acc": st["n_acc"]}


OWN = dict(attn=own_attn, step=own_step, fork=own_fork, compact=own_compact, verify=own_verify)


def run(state):
    op = state["case"]["op"]
    if own:
        import bit_moe_expert_histogram_gb300 as m
        return OWN[op](m, state)
    return PLAIN[op](state)


# ------------------------------------------------------------------- work --
def work(case):
    c = case
    if c["op"] == "attn":
        e, P = SIZE[c["type"]], c["prefix"] * BLOCK
        pairs = attn_lengths(c)
        row = 2 * c["n_kv"] * c["D"] * e  # one position's key and value
        qo = 2 * sum(new for _, new in pairs) * c["n_q"] * c["D"] * e
        table = 4 * sum(ceil_div(t, BLOCK) for t, _ in pairs) + 4 * c["prefix"]
        seen = sum(new * (P + t) for t, new in pairs)
        return {"bytes": row * (P + sum(t for t, _ in pairs)) + qo + table,
                "flops": 4 * c["D"] * c["n_q"] * seen}
    if c["op"] == "verify":
        rows = 2 if c["draft"] == "sampled" else 1
        n = c["slots"]
        return {"bytes": n * rows * c["V"] * SIZE[c["type"]] + n * c["T"] * 16,
                "flops": n * c["V"] * (rows + 1)}
    tails, shared = own_lengths(c)
    n = c["slots"]
    lens = [shared[i // c["beams"]] + tails[i] for i in range(n)]
    used = sum(ceil_div(x, BLOCK) for x in lens)
    width = table_width(c, c.get("T", 0) + BLOCK)
    meta = 4 * (used + n * width + 2 * n + 2 * c["n_phys"])
    flops = used + c["n_phys"]  # whole-number work: one addition an entry
    if c["op"] == "fork":
        return {"bytes": meta + 8 * n, "flops": flops}
    row = c["n_kv"] * c["D"] * 2
    pools = 2 * c["layers"]
    if c["op"] == "step":
        new = [1 + (i * 5 + 1) % c["T"] for i in range(n)]
        copied = sum(x % BLOCK for x in lens) if c["fresh"] and c["beams"] > 1 else 0
        return {"bytes": meta + 2 * row * pools * (copied + sum(new)), "flops": flops}
    live = min(pages_in_use(c), c["n_phys"])
    moves = int(live * (1 - live / c["n_phys"]))  # what random places leave past the live count
    return {"bytes": meta + 2 * moves * pools * row * BLOCK, "flops": flops}


# ------------------------------------------------------------------ exact --
def exact_attn(c, seed):
    st = prepare_attn(c, seed)
    B, T, n_q, n_kv, D = c["slots"], c["T"], c["n_q"], c["n_kv"], c["D"]
    lens, n_new = st["lens"].tolist(), st["n_new"].tolist()
    o = torch.zeros((B, T, n_q, D), dtype=torch.float64, device=st["q"].device)
    P = c["prefix"]
    for b in range(B):
        n, L = n_new[b], lens[b]
        if n == 0 or L == 0:
            continue
        blocks = st["table"][b, :ceil_div(L, BLOCK)].long()
        for h in range(n_kv):
            k = st["k"][blocks, h].double().reshape(-1, D)[:L]
            v = st["v"][blocks, h].double().reshape(-1, D)[:L]
            heads = range(h * (n_q // n_kv), (h + 1) * (n_q // n_kv))
            x = st["q"][b, :n, heads.start:heads.stop].double()  # [n, G, D]
            s = torch.einsum("tgd,ld->tgl", x, k) * D ** -0.5
            for t in range(n):
                s[t, :, L - n + t + 1:] = -math.inf
            o[b, :n, heads.start:heads.stop] = torch.softmax(s, -1) @ v
    return o


def exact_pages(c, seed):
    """The state after the operation, one slot and one page after the other."""
    dev = device()
    st = prepare_pages(c, seed)
    table, lens = st["table"].cpu().numpy(), st["lens"].cpu().numpy()
    refs = st["refs"].cpu().numpy()
    n, width = table.shape
    out, out_len, out_refs = np.full_like(table, -1), lens.copy(), refs.copy()
    nb = lambda x: ceil_div(int(x), BLOCK)  # noqa: E731
    if c["op"] == "fork":
        parent, keep = st["parent"].cpu().numpy(), st["keep"].cpu().numpy()
        for i in range(n):
            out_refs -= np.bincount(table[i, :nb(lens[i])], minlength=len(refs)).astype(np.int32)
            a = parent[i]
            out_len[i] = min(lens[a], keep[i]) if 0 <= a < n else 0
            if out_len[i]:
                row = table[a, :nb(out_len[i])]
                out[i, :len(row)] = row
                out_refs += np.bincount(row, minlength=len(refs)).astype(np.int32)
        return {"table": on(dev, out), "lens": on(dev, out_len), "refs": on(dev, out_refs)}
    if c["op"] == "step":
        n_new, granted = st["n_new"].cpu().numpy(), np.zeros(n, np.int32)
        free = [int(x) for x in np.nonzero(refs == 0)[0]]
        asked = 0
        for i in range(n):
            b0, b1 = nb(lens[i]), nb(lens[i] + n_new[i])
            out[i, :b0] = table[i, :b0]
            cow = n_new[i] > 0 and lens[i] % BLOCK > 0 and refs[table[i, b0 - 1]] > 1
            first, asked = asked, asked + b1 - b0 + int(cow)
            if asked > len(free) or b1 > width:
                continue
            granted[i], out_len[i] = n_new[i], lens[i] + n_new[i]
            taken = free[first:asked]
            if cow:
                out_refs[table[i, b0 - 1]] -= 1
                out[i, b0 - 1] = taken[0]
                taken_new = taken[1:]
            else:
                taken_new = taken
            out[i, b0:b1] = taken_new
            out_refs[taken] += 1
        return {"table": on(dev, out), "lens": on(dev, out_len), "refs": on(dev, out_refs),
                "granted": on(dev, granted), "pool": None}
    live = [i for i in range(len(refs)) if refs[i] > 0]
    L = len(live)
    to = dict(zip([i for i in live if i >= L], [i for i in range(L) if refs[i] == 0]))
    out_refs[:] = 0
    for i in live:
        out_refs[to.get(i, i)] = refs[i]
    for i in range(n):
        for j in range(nb(lens[i])):
            out[i, j] = to.get(int(table[i, j]), int(table[i, j]))
    return {"table": on(dev, out), "lens": on(dev, out_len), "refs": on(dev, out_refs),
            "n_live": torch.tensor([L], dtype=torch.int32, device=dev), "pool": None}


def exact_verify(c, seed):
    st = prepare_verify(c, seed)
    B, T, V = c["slots"], c["T"], c["V"]
    draft, n_draft = st["draft"].tolist(), st["n_draft"].tolist()
    u = st["u"].double().tolist()
    tokens, acc = np.full((B, T + 1), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        i = 0
        while i < n_draft[b]:
            x = draft[b][i]
            bar = u[b][i] * (float(st["q"][b, i, x]) if st["q"] is not None else 1.0)
            if not bar < float(st["p"][b, i, x]):
                break
            tokens[b, i] = x
            i += 1
        acc[b] = i
        w = st["p"][b, i].double().cpu().numpy()
        if i < n_draft[b]:
            d = np.zeros(V) if st["q"] is None else st["q"][b, i].double().cpu().numpy()
            if st["q"] is None:
                d[draft[b][i]] = w[draft[b][i]]
            rest = np.maximum(w - d, 0.0)
            w = rest if rest.sum() > 0 else w
        cum = np.cumsum(w)
        tokens[b, i] = int(np.searchsorted(cum, u[b][T] * cum[-1], side="right"))
    dev = device()
    return {"tokens": on(dev, tokens), "n_acc": on(dev, acc)}


def exact(case, seed):
    if case["op"] == "attn":
        return exact_attn(case, seed)
    if case["op"] == "verify":
        return exact_verify(case, seed)
    return exact_pages(case, seed)


if __name__ == "__main__":
    for name in range(20):
        print(draw(random.Random(name)))
