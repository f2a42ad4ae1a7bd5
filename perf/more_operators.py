"""Serving operators over a key/value cache held in 4 bits, and the log
probabilities of what is answered: rows quantised as they are written and read
back, decode attention of a batch over the 4-bit pages, log probabilities of
given tokens with entropy and top alternatives.

`run` computes an operator in its plain form with elementary torch
operations, or, when `own` is set, through the framework's calls. Sizes are
the decode attention's and the verification's of this repository (16 query
heads on 2 key/value heads of 128, pages of 64 positions, 10 full-attention
layers, vocabularies of 32000 to 131072), with others around them.

A position's row of one head: D / 2 bytes of codes, four bf16 scales, four bf16
biases, one of each for every D / 4 consecutive elements, which stand for
scale * code + bias. Pools are 16-bit [n_phys][n_kv][64][D / 4 + 8].
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = 64
GROUPS = 4
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


def device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def ceil_div(a, b):
    return -(-a // b)


def units(D):
    """16-bit units of a row."""
    return D // 4 + 2 * GROUPS


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # two short requests, one token each: latency is what counts
        dict(name="attn4-small", op="attn", slots=2, T=1, n_q=16, n_kv=2, D=128, base=256, own=50,
             type="bf16"),
        # a running server: single tokens of 48 requests of 8K and more
        dict(name="attn4-decode", op="attn", slots=48, T=1, n_q=16, n_kv=2, D=128, base=8192,
             own=777, type="bf16"),
        # other heads and sizes: drafts of up to 3 tokens, contexts of all lengths
        dict(name="attn4-ragged", op="attn", slots=33, T=3, n_q=12, n_kv=4, D=64, base=0, own=5000,
             type="fp16"),
        # a few very long documents
        dict(name="attn4-long", op="attn", slots=8, T=1, n_q=16, n_kv=2, D=128, base=100000,
             own=31000, type="bf16"),
        # the largest: up to four drafted tokens of 256 requests
        dict(name="attn4-drafts", op="attn", slots=256, T=4, n_q=16, n_kv=2, D=128, base=200,
             own=16000, type="bf16"),
        # a step's new rows of 48 requests into all 10 layers' pages, and what
        # those pages now stand for
        dict(name="write-step", op="write", slots=48, T=4, layers=10, n_kv=2, D=128, base=4000,
             own=300, type="bf16"),
        # prompts of 16 requests into one layer; their own attention then runs
        # over the same rounded numbers that later steps will read
        dict(name="write-prompt", op="write", slots=16, T=8192, layers=1, n_kv=2, D=128, base=0,
             own=0, type="bf16"),
        # the tails of a few slots read back in 32 bits
        dict(name="read-small", op="read", slots=3, T=70, n_kv=4, D=64, base=90, own=500,
             type="fp32"),
        # whole contexts read back for kernels that take 16-bit rows
        dict(name="read-long", op="read", slots=16, T=9000, n_kv=2, D=128, base=3000, own=6000,
             type="bf16"),
        # one request's token, a 32000-token vocabulary
        dict(name="logp-small", op="logp", rows=1, V=32000, pad=0, k=5, masked=0.0, type="fp32"),
        # a running server: a token each with twenty alternatives, logits cut
        # out of a padded vocabulary, a grammar that forbids half of it
        dict(name="logp-decode", op="logp", rows=64, V=131072, pad=512, k=20, masked=0.5,
             type="bf16"),
        # the tokens of a whole prompt, an odd vocabulary
        dict(name="logp-prompt", op="logp", rows=2048, V=128001, pad=0, k=1, masked=0.0,
             type="bf16"),
    ]


def spread(rng, lo, hi):
    """A whole number in [lo, hi], even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "write", "read", "logp", "logp"])
    top = {c["name"]: work(c) for c in listed()}
    most = {"attn": "attn4-drafts", "write": "write-prompt", "read": "read-long",
            "logp": "logp-prompt"}[op]
    while True:
        if op == "attn":
            n_q, n_kv = rng.choice([(16, 2), (16, 2), (12, 4), (8, 8), (32, 4), (5, 1), (28, 4)])
            c = dict(op=op, slots=spread(rng, 1, 256), T=rng.choice([1, 1, 1, 2, 3, 4, 5, 8]),
                     n_q=n_q, n_kv=n_kv, D=rng.choice([64, 128, 128]),
                     base=rng.choice([0, spread(rng, 1, 100000)]), own=spread(rng, 1, 31000),
                     type=rng.choice(["bf16", "bf16", "fp16"]))
            if c["T"] * n_q // n_kv > 64:
                continue
        elif op == "write":
            c = dict(op=op, slots=spread(rng, 1, 256), T=spread(rng, 1, 8192),
                     layers=rng.choice([1, 1, 2, 10]), n_kv=rng.choice([1, 2, 4, 8]),
                     D=rng.choice([64, 128, 128]), base=rng.choice([0, spread(rng, 1, 4000)]),
                     own=spread(rng, 1, 300), type=rng.choice(["bf16", "fp16"]))
        elif op == "read":
            c = dict(op=op, slots=spread(rng, 1, 256), T=spread(rng, 1, 9000),
                     n_kv=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128, 128]),
                     base=spread(rng, 1, 3000), own=spread(rng, 1, 6000),
                     type=rng.choice(["bf16", "fp16", "fp32"]))
        else:
            V = spread(rng, 100, 200000)
            c = dict(op=op, rows=spread(rng, 1, 2048), V=V, pad=rng.choice([0, 0, 64, 7]),
                     k=rng.choice([0, 1, 5, 20, 32]),
                     masked=rng.choice([0.0, 0.5, 0.97]) if V > 5000 else 0.0,
                     type=rng.choice(["fp32", "bf16", "bf16", "fp16"]))
        w = work(c)
        if w["flops"] <= top[most]["flops"] and w["bytes"] <= top[most]["bytes"]:
            return c


def lengths(c):
    """Positions and new tokens of each slot, the same for every seed: of eight
    slots and more one in sixteen is idle, lengths crowd toward the short ones."""
    n = c["slots"]
    out = []
    for i in range(n):
        new = 1 + (i * 7919 + 3) % c["T"] if i % 3 else c["T"]
        idle = n >= 8 and i % 16 == 5
        more = int(c["own"] * ((i + 0.5) / n) ** 1.5)
        if c["op"] == "read":  # what is read ends at the slot's end at the latest
            size = max(1, c["base"] + more)
            out.append((size, 0 if idle else min(new, size)))
        elif c["op"] == "write":
            out.append((c["base"] + more + new, new))
        else:
            out.append((0, 0) if idle else (max(new, c["base"] + more), new))
    return out


# --------------------------------------------------------------- the rows --
def round_bf16(x):
    """float64 >= 0 to the nearest bf16, ties to even (values stay float64)."""
    e = torch.frexp(x).exponent
    unit = torch.ldexp(torch.ones_like(x), (e - 8).clamp(min=-133))
    return torch.round(x / unit) * unit


def floor_bf16(x):
    """float32 to the largest bf16 that is not above it."""
    up = x.view(torch.int32)
    cut = torch.where(x < 0, (up + 0xFFFF) & -0x10000, up & -0x10000)
    return cut.view(torch.float32)


def quantise(x):
    """[..., D] values: codes uint8 [..., D], scales and biases bf16 [..., 4]."""
    g = x.float().view(*x.shape[:-1], GROUPS, x.shape[-1] // GROUPS)
    b = floor_bf16(g.amin(-1).contiguous()).double()
    s = round_bf16((g.amax(-1).double() - b) / 15.0)
    step = torch.where(s > 0, s, torch.ones_like(s))[..., None]
    q = torch.floor((g.double() - b[..., None]) / step + 0.5).clamp(max=15)
    q = torch.where(s[..., None] > 0, q, torch.zeros_like(q))
    return q.to(torch.uint8).view(x.shape), s.bfloat16(), b.bfloat16()


def pack(q, s, b):
    """Rows of 16-bit units [..., units(D)]. A byte holds two elements, the
    first in its low half; with D = 64 the bytes of the two groups of a half
    row alternate."""
    D = q.shape[-1]
    by = q[..., 0::2] | (q[..., 1::2] << 4)
    if D == 64:
        by = by.view(*q.shape[:-1], 2, 2, 8).transpose(-1, -2).reshape(*q.shape[:-1], 32)
    codes = by.contiguous().view(torch.int16)
    return torch.cat([codes, s.view(torch.int16), b.view(torch.int16)], -1)


def unpack(rows, D):
    """What rows of a pool stand for, float32 [..., D]."""
    by = rows[..., :D // 4].contiguous().view(torch.uint8)
    if D == 64:
        by = by.view(*rows.shape[:-1], 2, 8, 2).transpose(-1, -2).reshape(*rows.shape[:-1], 32)
    q = torch.stack([by & 15, by >> 4], -1).float().view(*rows.shape[:-1], GROUPS, D // GROUPS)
    par = rows[..., D // 4:].contiguous().view(torch.bfloat16).float()
    return (q * par[..., :GROUPS, None] + par[..., GROUPS:, None]).view(*rows.shape[:-1], D)


# ---------------------------------------------------------------- prepare --
def gen_for(seed, dev):
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    return g


def on(dev, a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def like_keys(shape, g, dev, keys):
    """Rows as trained heads have them: keys with a few strong channels, values
    even; both with rows of different size."""
    x = torch.randn(shape, generator=g, device=dev)
    x *= torch.exp(0.4 * torch.randn((*shape[:-1], 1), generator=g, device=dev))
    if keys:
        strong = torch.rand(shape[-1], generator=g, device=dev) < 0.05
        x = x * torch.where(strong, 4.0, 1.0) + torch.where(strong, 3.0, 0.0)
    return x


def filled_pool(c, n_phys, g, dev, keys):
    """A pool of quantised rows, made some pages at a time."""
    pool = torch.empty((n_phys, c["n_kv"], BLOCK, units(c["D"])), dtype=torch.int16, device=dev)
    step = max(1, (1 << 25) // (c["n_kv"] * BLOCK * c["D"]))
    for i in range(0, n_phys, step):
        part = pool[i:i + step]
        part.copy_(pack(*quantise(like_keys((*part.shape[:3], c["D"]), g, dev, keys).bfloat16())))
    return pool


def slots_state(c, seed, dev):
    """table, lens, n_new of slots whose pages lie at random places."""
    rng = np.random.RandomState(seed % (1 << 31))
    pairs = lengths(c)
    pairs = [pairs[i] for i in rng.permutation(len(pairs))]
    blocks = [ceil_div(n, BLOCK) for n, _ in pairs]
    n_phys = sum(blocks) + 3
    pages = rng.permutation(n_phys).astype(np.int32)
    table = np.full((c["slots"], max(blocks) + 1), -1, np.int32)
    at = 0
    for i, nb in enumerate(blocks):
        table[i, :nb] = pages[at:at + nb]
        at += nb
    lens = np.array([p[0] for p in pairs], np.int32)
    new = np.array([p[1] for p in pairs], np.int32)
    return on(dev, table), on(dev, lens), on(dev, new), n_phys


def prepare_attn(c, seed):
    dev = device()
    g = gen_for(seed, dev)
    table, lens, n_new, n_phys = slots_state(c, seed, dev)
    dt = TYPES[c["type"]]
    q = torch.randn((c["slots"], c["T"], c["n_q"], c["D"]), generator=g, device=dev)
    q = (q * torch.linspace(0.4, 1.6, c["n_q"], device=dev)[:, None]).to(dt)
    st = dict(case=c, q=q, k=filled_pool(c, n_phys, g, dev, True),
              v=filled_pool(c, n_phys, g, dev, False), table=table, lens=lens, n_new=n_new)
    if own:
        import bit_moe_expert_histogram_gb300 as m
        st["shape"] = m.make_attn_batch_shape(c["slots"], c["T"], c["n_q"], c["n_kv"], c["D"],
                                              table.shape[1], dtype=c["type"])
        st["ws"] = m.alloc_attn_batch_q4_workspace(st["shape"], dev)
        st["o"] = torch.empty_like(q)
    return st


def prepare_rows(c, seed):
    dev = device()
    g = gen_for(seed, dev)
    table, lens, n_new, n_phys = slots_state(c, seed, dev)
    dt = TYPES[c["type"]]
    layers = c.get("layers", 1)
    st = dict(case=c, table=table, lens=lens, n_new=n_new)
    tokens = (c["slots"], c["T"], c["n_kv"], c["D"])
    if c["op"] == "write":
        # the projections' output, keys and values side by side; pages that
        # hold anything
        kv = torch.empty((layers, c["slots"], c["T"], 2, c["n_kv"], c["D"]), dtype=dt, device=dev)
        for i in range(layers):
            for j in range(2):
                kv[i, :, :, j] = like_keys(tokens, g, dev, j == 0).to(dt)
        st["kv_new"] = kv
        st["pool"] = torch.randint(-30000, 30000, (2 * layers, n_phys, c["n_kv"], BLOCK,
                                                   units(c["D"])), generator=g, device=dev,
                                   dtype=torch.int16)
    else:
        st["pool"] = torch.stack([filled_pool(c, n_phys, g, dev, j == 0) for j in range(2)])
    st["first"] = (lens - n_new).to(torch.int32)
    st["k_out"] = torch.zeros((layers, *tokens), dtype=dt, device=dev)
    st["v_out"] = torch.zeros((layers, *tokens), dtype=dt, device=dev)
    if own:
        import bit_moe_expert_histogram_gb300 as m
        st["shape"] = m.make_cache_shape(c["slots"], table.shape[1], n_phys, c["n_kv"], c["D"])
        st["ws"] = m.alloc_cache_workspace(st["shape"], dev)
        st["meta"] = m.CacheMeta(table, lens, torch.ones(n_phys, dtype=torch.int32, device=dev))
    return st


def prepare_logp(c, seed):
    dev = device()
    g = gen_for(seed, dev)
    n, V = c["rows"], c["V"]
    dt = TYPES[c["type"]]
    full = torch.zeros((n, V + c["pad"]), dtype=dt, device=dev)
    tokens = torch.empty(n, dtype=torch.int32, device=dev)
    step = max(1, (1 << 26) // V)
    for i in range(0, n, step):  # some rows at a time keep the scratch small
        x = torch.randn((min(step, n - i), V), generator=g, device=dev) * 3.0
        if c["masked"] > 0:
            hide = torch.rand(V, generator=g, device=dev) < c["masked"]
            x = x.masked_fill(hide, -math.inf)
        full[i:i + step, :V] = x.to(dt)
        # a sampled token: the largest of the logits with Gumbel noise
        u = torch.rand(x.shape, generator=g, device=dev).clamp(min=1e-30)
        x -= torch.log(-torch.log(u).clamp(min=1e-30))
        tokens[i:i + step] = x.argmax(-1).to(torch.int32)
    if n >= 8:
        tokens[5::16] = -1  # rows of padding: no token asked for
    st = dict(case=c, logits=full[:, :V], tokens=tokens)
    if own:
        import bit_moe_expert_histogram_gb300 as m
        st["shape"] = m.make_logprobs_shape(n, V, c["k"], dtype=c["type"])
        st["ws"] = m.alloc_logprobs_workspace(st["shape"], dev)
        f32 = lambda *s: torch.empty(s, dtype=torch.float32, device=dev)  # noqa: E731
        st["logp"], st["entropy"] = f32(n), f32(n)
        st["top_ids"] = torch.empty((n, c["k"]), dtype=torch.int32, device=dev)
        st["top_logp"] = f32(n, c["k"])
    return st


PREPARE = dict(attn=prepare_attn, write=prepare_rows, read=prepare_rows, logp=prepare_logp)


def prepare(case, seed):
    return PREPARE[case["op"]](case, seed)


# -------------------------------------------------------------- plain forms --
def plain_attn(st):
    c = st["case"]
    T, n_q, n_kv, D = c["T"], c["n_q"], c["n_kv"], c["D"]
    G = n_q // n_kv
    dev = st["q"].device
    W = st["table"].shape[1] * BLOCK
    o = torch.empty_like(st["q"])
    at = torch.arange(W, device=dev)
    tok = torch.arange(T, device=dev)
    some = max(1, (1 << 29) // (W * n_kv * D))  # slots at a time, what 2 GB hold
    for i in range(0, c["slots"], some):
        q, table = st["q"][i:i + some].float(), st["table"][i:i + some].clamp(min=0).long()
        lens, new = st["lens"][i:i + some, None], st["n_new"][i:i + some, None]
        B = q.shape[0]
        pos = torch.where((tok < new) & (lens - new + tok >= 0), lens - new + tok, -1)  # [B, T]

        def rows(pool):
            return unpack(pool[table], D).transpose(1, 2).reshape(B, n_kv, W, D)
        q = q.view(B, T, n_kv, G, D).transpose(1, 2).reshape(B, n_kv, T * G, D) / math.sqrt(D)
        s = q @ rows(st["k"]).transpose(-1, -2)
        ok = (at <= pos[:, :, None]).repeat_interleave(G, 1)[:, None]
        s.masked_fill_(~ok, -math.inf)
        top = s.amax(-1, keepdim=True)
        s.sub_(torch.where(top.isinf(), torch.zeros_like(top), top)).exp_()
        den = s.sum(-1, keepdim=True)
        # what lies past a slot's end weighs 0 and may be anything
        v = rows(st["v"]).masked_fill_((at >= lens)[:, None, :, None], 0.0)
        num = s @ v
        r = torch.where(den > 0, num / den, torch.zeros_like(num))
        o[i:i + some] = r.view(B, n_kv, T, G, D).transpose(1, 2).reshape(B, T, n_q, D).to(o.dtype)
    return o


def places(st):
    """(slot, token, page, row in the page) of the tokens to write or read."""
    n_new = st["n_new"].long()
    tok = torch.arange(st["case"]["T"], device=n_new.device)
    slot, tok = (tok < n_new[:, None]).nonzero(as_tuple=True)
    pos = st["first"].long()[slot] + tok
    return slot, tok, st["table"][slot, pos // BLOCK].long(), pos % BLOCK


def plain_write(st):
    slot, tok, page, row = places(st)
    for i in range(st["case"]["layers"]):
        for j in range(2):
            new = st["kv_new"][i, slot, tok, j]  # [m, n_kv, D]
            st["pool"][2 * i + j].transpose(1, 2)[page, row] = pack(*quantise(new))
    return plain_read(st)


def plain_read(st):
    slot, tok, page, row = places(st)
    D = st["case"]["D"]
    for i in range(st["k_out"].shape[0]):
        for j, out in enumerate((st["k_out"], st["v_out"])):
            held = st["pool"][2 * i + j].transpose(1, 2)[page, row]
            out[i, slot, tok] = unpack(held, D).to(out.dtype)
    return {"k": st["k_out"], "v": st["v_out"]}


def plain_logp(st):
    c = st["case"]
    x = st["logits"].float()
    m = x.amax(-1, keepdim=True)
    d = x - m
    e = torch.exp(d)
    z = e.sum(-1)
    a = torch.where(e > 0, e * d, torch.zeros_like(d)).sum(-1)
    lse = torch.log(z)
    tok = st["tokens"].long()
    got = d.gather(1, tok.clamp(min=0)[:, None])[:, 0] - lse
    out = {"logp": torch.where(tok >= 0, got, torch.zeros_like(got)), "entropy": lse - a / z}
    if c["k"] > 0:
        v, i = torch.sort(d, dim=-1, descending=True, stable=True)
        v, i = v[:, :c["k"]], i[:, :c["k"]]
        out["top_ids"] = torch.where(v == -math.inf, -1, i).to(torch.int32)
        out["top_logp"] = v - lse[:, None]
    return out


PLAIN = dict(attn=plain_attn, write=plain_write, read=plain_read, logp=plain_logp)


# --------------------------------------------------------------- own forms --
def own_attn(m, st):
    m.moe_attn_batch_q4(st["shape"], st["q"], st["k"], st["v"], st["table"], st["lens"], st["o"],
                        st["ws"], n_new=st["n_new"])
    return st["o"]


def own_write(m, st):
    pool, kv = st["pool"], st["kv_new"]
    for i in range(st["case"]["layers"]):  # as the layers of a step call it
        m.moe_cache_write_q4(st["shape"], st["meta"], st["n_new"], kv[i, :, :, 0], kv[i, :, :, 1],
                             pool[2 * i], pool[2 * i + 1], st["ws"])
        m.moe_cache_read_q4(st["shape"], st["meta"], st["first"], st["n_new"], pool[2 * i],
                            pool[2 * i + 1], st["k_out"][i], st["v_out"][i], st["ws"])
    return {"k": st["k_out"], "v": st["v_out"]}


def own_read(m, st):
    m.moe_cache_read_q4(st["shape"], st["meta"], st["first"], st["n_new"], st["pool"][0],
                        st["pool"][1], st["k_out"][0], st["v_out"][0], st["ws"])
    return {"k": st["k_out"], "v": st["v_out"]}


def own_logp(m, st):
    k = st["case"]["k"]
    m.moe_token_logprobs(st["shape"], st["logits"], st["tokens"], st["logp"], st["ws"],
                         entropy=st["entropy"], top_ids=st["top_ids"] if k else None,
                         top_logp=st["top_logp"] if k else None)
    out = {"logp": st["logp"], "entropy": st["entropy"]}
    if k > 0:
        out["top_ids"], out["top_logp"] = st["top_ids"], st["top_logp"]
    return out


OWN = dict(attn=own_attn, write=own_write, read=own_read, logp=own_logp)


def run(state):
    op = state["case"]["op"]
    if own:
        import bit_moe_expert_histogram_gb300 as m
        return OWN[op](m, state)
    return PLAIN[op](state)


# ------------------------------------------------------------------- work --
def work(case):
    c = case
    if c["op"] == "logp":
        n, size = c["rows"], c["rows"] * c["V"]
        return {"bytes": size * SIZE[c["type"]] + n * (12 + 8 * c["k"]), "flops": 5 * size}
    row = 2 * units(c["D"])
    pairs = lengths(c)
    new = sum(n for _, n in pairs)
    table = 4 * sum(ceil_div(n, BLOCK) for n, _ in pairs) + 8 * c["slots"]
    if c["op"] == "attn":
        qo = 2 * new * c["n_q"] * c["D"] * 2
        held = sum(n for n, _ in pairs)
        return {"bytes": 2 * c["n_kv"] * row * held + qo + table,
                "flops": 4 * c["D"] * c["n_q"] * sum(a * b for a, b in pairs)}
    values = 2 * c.get("layers", 1) * new * c["n_kv"]
    dense = c["D"] * SIZE[c["type"]]
    times = 2 if c["op"] == "write" else 1  # rows in, values out; values out
    return {"bytes": values * (times * dense + row) + table, "flops": values * c["D"] * 4 * times}


# ------------------------------------------------------------------ exact --
def exact_row_values(rows, D):
    """float64 values of one pool's rows [..., units], element by element place."""
    raw = rows.long() & 0xFFFF
    e = torch.arange(D, device=rows.device)
    if D == 128:
        unit, nib = e // 4, e % 4
    else:  # 4 elements of a unit: two of each group of its half
        half, r = e // 32, e % 32
        unit, nib = half * 8 + (r % 16) // 2, 2 * (r // 16) + r % 2
    code = (raw[..., unit] >> (4 * nib)) & 15

    def bf16(u):
        return (u << 16).to(torch.int32).view(torch.float32).double()
    g = e // (D // 4)
    scale = bf16(raw[..., D // 4:D // 4 + 4])[..., g]
    return code.double() * scale + bf16(raw[..., D // 4 + 4:])[..., g]


def exact_attn(c, seed):
    st = prepare_attn(c, seed)
    n_q, n_kv, D = c["n_q"], c["n_kv"], c["D"]
    G = n_q // n_kv
    lens, n_new = st["lens"].tolist(), st["n_new"].tolist()
    o = torch.zeros(st["q"].shape, dtype=torch.float64, device=st["q"].device)
    for b, (L, n) in enumerate(zip(lens, n_new)):
        if n == 0:
            continue
        blocks = st["table"][b, :ceil_div(L, BLOCK)].long()
        for h in range(n_kv):
            k = exact_row_values(st["k"][blocks, h], D).reshape(-1, D)[:L]
            v = exact_row_values(st["v"][blocks, h], D).reshape(-1, D)[:L]
            x = st["q"][b, :n, h * G:(h + 1) * G].double()
            s = torch.einsum("tgd,ld->tgl", x, k) * D ** -0.5
            for t in range(n):
                s[t, :, L - n + t + 1:] = -math.inf
            o[b, :n, h * G:(h + 1) * G] = torch.softmax(s, -1) @ v
    return o


def exact_quantised(x):
    """What a row [.., D] stands for once written, by counting borders."""
    D = x.shape[-1]
    x = x.double().unflatten(-1, (4, D // 4))
    lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
    b = lo.float().bfloat16()  # nearest, then one down where that is above
    bits = b.view(torch.int16).int()
    down = torch.where(b == 0, torch.full_like(bits, -32767), torch.where(bits < 0, bits + 1, bits - 1))
    b = torch.where(b.double() > lo, down.to(torch.int16).view(torch.bfloat16), b).double()
    want = (hi - b) / 15.0
    near = want.float().bfloat16().view(torch.int16).int()  # one of the three around it
    best = None
    for step in (-1, 0, 1):
        bits = (near + step).clamp(min=0).to(torch.int16)
        val = bits.view(torch.bfloat16).double()
        off = (val - want).abs()
        if best is None:
            best, s, even = off, val, bits % 2 == 0
            continue
        take = (off < best) | ((off == best) & ~even & (bits % 2 == 0))
        best, s = torch.where(take, off, best), torch.where(take, val, s)
        even = torch.where(take, bits % 2 == 0, even)
    code = torch.zeros_like(x)
    for j in range(1, 16):
        code += ((x - b) >= (j - 0.5) * s) & (s > 0)
    return (code * s + b).flatten(-2)


def exact_rows(c, seed):
    st = prepare_rows(c, seed)
    D = c["D"]
    k = torch.zeros(st["k_out"].shape, dtype=torch.float64, device=st["k_out"].device)
    v = torch.zeros_like(k)
    table = st["table"].cpu()
    for b, (first, n) in enumerate(zip(st["first"].tolist(), st["n_new"].tolist())):
        for i in range(k.shape[0]):
            for j, out in enumerate((k, v)):
                if c["op"] == "write":
                    out[i, b, :n] = exact_quantised(st["kv_new"][i, b, :n, j])
                    continue
                pages = table[b, first // BLOCK:ceil_div(first + n, BLOCK)].long().to(k.device)
                if n == 0:
                    continue
                rows = st["pool"][j][pages].transpose(1, 2).flatten(0, 1)
                out[i, b, :n] = exact_row_values(rows[first % BLOCK:][:n], D)
    return {"k": k, "v": v}


def exact_logp(c, seed):
    st = prepare_logp(c, seed)
    n, V, k = c["rows"], c["V"], c["k"]
    dev = st["tokens"].device
    f64 = lambda *s: torch.zeros(s, dtype=torch.float64, device=dev)  # noqa: E731
    out = {"logp": f64(n), "entropy": f64(n)}
    if k > 0:
        out["top_ids"] = torch.full((n, k), -1, dtype=torch.int32, device=dev)
        out["top_logp"] = f64(n, k)
    step = max(1, (1 << 26) // V)
    for i in range(0, n, step):
        x = torch.log_softmax(st["logits"][i:i + step].double(), -1)
        r = torch.arange(x.shape[0], device=dev)
        tok = st["tokens"][i:i + step].long()
        out["logp"][i:i + step] = torch.where(tok >= 0, x[r, tok.clamp(min=0)], 0.0)
        p = torch.exp(x)
        out["entropy"][i:i + step] = -torch.where(p > 0, p * x, torch.zeros_like(x)).sum(-1)
        for j in range(k):  # the largest that is left, the first of its kind
            at = x.argmax(-1)
            best = x[r, at]
            out["top_ids"][i:i + step, j] = torch.where(best == -math.inf, -1, at).to(torch.int32)
            out["top_logp"][i:i + step, j] = best
            x[r, at] = -math.inf
    return out


def exact(case, seed):
    return dict(attn=exact_attn, write=exact_rows, read=exact_rows,
                logp=exact_logp)[case["op"]](case, seed)


if __name__ == "__main__":
    for number in range(20):
        print(draw(random.Random(number)))
