"""Plain references of the 4-bit cache and of token log probabilities, in 64
bits: rows quantised by counting borders, packed nibble by nibble, attention
and log probabilities from their formulas."""
import numpy as np

BLOCK = 64


def units(D):
    return D // 4 + 8


def bf16_of(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32)


def bf16_bits(x):
    """float32 numbers that are bf16 numbers -> their bits."""
    return (np.ascontiguousarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint16)


def bf16_grid(x, how):
    """float64 -> the bf16 number that `how` (np.floor, np.rint) picks."""
    x = np.asarray(x, np.float64)
    _, e = np.frexp(x)
    step = np.ldexp(1.0, np.maximum(e - 8, -133))
    return how(x / step) * step


def quantise(x):
    """[..., D] float64 -> codes uint8 [..., D], s, b float64 [..., 4]."""
    D = x.shape[-1]
    g = np.asarray(x, np.float64).reshape(*x.shape[:-1], 4, D // 4)
    b = bf16_grid(g.min(-1), np.floor)
    s = bf16_grid((g.max(-1) - b) / 15.0, np.rint)
    code = np.zeros(g.shape, np.uint8)
    for j in range(1, 16):
        code += ((g - b[..., None]) >= (j - 0.5) * s[..., None]) & (s[..., None] > 0)
    return code.reshape(x.shape), s, b


def place(D):
    """Element e's code: (16-bit unit, shift in it)."""
    where = []
    for e in range(D):
        if D == 128:
            where.append((e // 4, 4 * (e % 4)))
        else:
            half, group, i = e // 32, e % 32 // 16, e % 16
            where.append((8 * half + i // 2, 8 * group + 4 * (i % 2)))
    return np.array(where)


def pack(code, s, b):
    D = code.shape[-1]
    out = np.zeros((*code.shape[:-1], units(D)), np.uint16)
    for e, (u, sh) in enumerate(place(D)):
        out[..., u] |= code[..., e].astype(np.uint16) << np.uint16(sh)
    out[..., D // 4:D // 4 + 4] = bf16_bits(s)
    out[..., D // 4 + 4:] = bf16_bits(b)
    return out.view(np.int16)


def parts(rows, D):
    """codes float64 [..., D], s and b of every element [..., D]."""
    raw = np.ascontiguousarray(rows).view(np.uint16)
    p = place(D)
    code = (raw[..., p[:, 0]] >> p[:, 1].astype(np.uint16) & 15).astype(np.float64)
    g = np.arange(D) // (D // 4)
    with np.errstate(invalid="ignore"):  # pages that were never written hold anything
        s = bf16_of(raw[..., D // 4:D // 4 + 4]).astype(np.float64)[..., g]
        b = bf16_of(raw[..., D // 4 + 4:]).astype(np.float64)[..., g]
    return code, s, b


def values(rows, D):
    code, s, b = parts(rows, D)
    return code * s + b


def attention(q, k, v, table, lens, n_new):
    """(o, bound per output but for o's own rounding): q float64
    [B][T][n_q][D], pools int16 [n_phys][n_kv][64][units]. Positions on pages
    that are none are left out. The bound counts the roundings that the
    call's documentation allows, e = 2^-11 being half a step of fp16:
    - weights p (1 + d), |d| <= e, the same in numerator and denominator:
      sum p (1 + d) v / sum p (1 + d) - o = sum p d (v - o) / sum p (1 + d), at
      most (1 + 2 e) e sum p |v - o|;
    - their products with the scales, e of sum p s c, a second time;
    - below 2^-14 fp16 is off by half its least number, 2^-25: scales and biases
      under the group's power of two 2^g, 2^-25 2^g each; products and weights,
      of which there are n beside a sum of 2^8 or more, n 2^-33 2^g and n 2^-33
      |v - o|. 2^g is at most twice the largest of 16 s and |b|, and so |v| is at
      most 2^g, |v - o| twice that;
    - the scores' fp32 sums (up to 136 terms, 2^-23 each) in the exponent, twice
      for numerator and denominator; fp32 sums over the positions, sixteen a step
      and some ten steps more for joining."""
    B, T, n_q, D = q.shape
    n_phys, n_kv = k.shape[:2]
    G = n_q // n_kv
    o, tol = np.zeros(q.shape), np.zeros(q.shape)
    for s in range(B):
        L, n = int(lens[s]), int(n_new[s])
        if n == 0 or L == 0:
            continue
        pages = table[s, :-(-L // BLOCK)]
        ok = (pages >= 0) & (pages < n_phys)
        there = np.repeat(ok, BLOCK)[:L]
        for h in range(n_kv):
            rows = [np.concatenate([p[x, h] if y else np.zeros((BLOCK, p.shape[-1]), np.int16)
                                    for x, y in zip(pages, ok)])[:L] for p in (k, v)]
            kc, ks, kb = parts(rows[0], D)
            vc, vs, vb = parts(rows[1], D)
            for t in range(n):
                see = there & (np.arange(L) <= L - n + t)
                if not see.any():
                    continue
                x = q[s, t, h * G:(h + 1) * G]
                sc = x @ (kc * ks + kb)[see].T / np.sqrt(D)
                mag = np.abs(x) @ (kc * np.abs(ks) + np.abs(kb))[see].T / np.sqrt(D)
                p = np.exp(sc - sc.max(-1, keepdims=True))
                p /= p.sum(-1, keepdims=True)
                val = (vc * vs + vb)[see]
                o[s, t, h * G:(h + 1) * G] = p @ val
                off = np.stack([p[i] @ np.abs(val - o[s, t, h * G + i]) for i in range(G)])
                big = np.maximum(16 * vs, np.abs(vb))[:L][there].max(0)
                w = p @ (vc * vs)[see]
                a = w + p @ np.abs(vb)[see]
                far = 2 * 136 * 2.0**-23 * mag.max(-1, keepdims=True) + (see.sum() / 16 + 32) * 2.0**-23
                least = 2 * big * (2 * 2.0**-25 + 3 * see.sum() * 2.0**-33)
                tol[s, t, h * G:(h + 1) * G] = 2.0**-11 * (1 + 2.0**-9) * (w + off) + least + far * a
    return o, tol


def logprobs(x, tokens, k):
    """x float64 [n][V]: logp, entropy, top ids, top logp."""
    n, V = x.shape
    m = x.max(-1, keepdims=True)
    d = x - m
    lp = d - np.log(np.exp(d).sum(-1, keepdims=True))
    p = np.exp(lp)
    ent = -(p * np.where(p > 0, lp, 0.0)).sum(-1)
    got = np.array([lp[i, t] if t >= 0 else 0.0 for i, t in enumerate(tokens)])
    ids, top = np.full((n, k), -1, np.int64), np.full((n, k), -np.inf)
    for i in range(n):
        order = np.lexsort((np.arange(V), -x[i]))[:k]
        order = order[x[i, order] > -np.inf]
        ids[i, :len(order)], top[i, :len(order)] = order, lp[i, order]
    return got, ent, ids, top
