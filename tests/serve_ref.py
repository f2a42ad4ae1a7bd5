"""Plain references of the batch serving calls, one slot, page and token after
the other: the cache's pages in whole numbers, attention and verification in
64 bits."""
import numpy as np

BLOCK = 64


def nb(n):
    return -(-int(n) // BLOCK)


def make_state(rng, n_slots, max_blocks, n_phys, fill=0.6, share=0.5):
    """A consistent state: slots with random lengths; some start with pages of
    an earlier slot (its partly filled last page among them)."""
    table = np.full((n_slots, max_blocks), -1, np.int32)
    lens = np.zeros(n_slots, np.int32)
    free = list(rng.permutation(n_phys))
    budget = int(n_phys * fill)
    for s in range(n_slots):
        row = []
        if s and rng.random() < share:
            a = int(rng.integers(s))
            keep = int(rng.integers(lens[a] + 1))
            row = list(table[a, :nb(keep)])
            lens[s] = keep
        if not row or lens[s] % BLOCK == 0:  # a tail of its own past whole shared pages
            more = int(rng.integers(0, max(1, max_blocks - len(row)) + 1))
            more = min(more, max_blocks - len(row), budget, len(free))
            if more:
                row += [free.pop() for _ in range(more)]
                budget -= more
                lens[s] = len(row) * BLOCK - int(rng.integers(0, BLOCK))
        table[s, :len(row)] = row
    refs = np.bincount(table[table >= 0], minlength=n_phys).astype(np.int32)
    return table, lens, refs


def fork(table, lens, refs, parent, keep):
    n, width = table.shape
    t, ln, rf = np.full_like(table, -1), np.zeros_like(lens), refs.copy()
    for s in range(n):
        for p in table[s, :nb(lens[s])]:
            rf[p] -= 1
    for s in range(n):
        a = parent[s]
        if 0 <= a < n:
            ln[s] = lens[a] if keep is None else min(lens[a], max(0, keep[s]))
            t[s, :nb(ln[s])] = table[a, :nb(ln[s])]
            for p in t[s, :nb(ln[s])]:
                rf[p] += 1
    return t, ln, rf


def reserve(table, lens, refs, n_new, pools):
    """(table, lens, refs, granted); pools [n][n_phys][n_kv][64][D] in place."""
    n, width = table.shape
    t, ln, rf = table.copy(), lens.copy(), refs.copy()
    granted = np.zeros(n, np.int32)
    free = [int(p) for p in np.nonzero(refs == 0)[0]]
    asked = 0
    for s in range(n):
        b0, b1 = nb(lens[s]), nb(int(lens[s]) + max(0, int(n_new[s])))
        t[s, b0:] = -1
        cow = n_new[s] > 0 and lens[s] % BLOCK and refs[table[s, b0 - 1]] > 1
        first, asked = asked, asked + b1 - b0 + bool(cow)
        if n_new[s] <= 0 or asked > len(free) or b1 > width:
            continue
        take = free[first:asked]
        granted[s] = n_new[s]
        ln[s] += n_new[s]
        rf[take] += 1
        if cow:
            old = table[s, b0 - 1]
            rf[old] -= 1
            rows = lens[s] % BLOCK
            pools[:, take[0], :, :rows] = pools[:, old, :, :rows]
            t[s, b0 - 1] = take[0]
            take = take[1:]
        t[s, b0:b1] = take
    return t, ln, rf, granted


def write(table, lens, n_new, new, pool):
    """new [n_slots][T][n_kv][D] into pool, in place."""
    for s in range(table.shape[0]):
        for i in range(n_new[s]):
            pos = lens[s] - n_new[s] + i
            pool[table[s, pos // BLOCK], :, pos % BLOCK] = new[s, i]


def compact(table, lens, refs, pools):
    live = np.nonzero(refs)[0]
    L = len(live)
    src, dst = live[live >= L], np.nonzero(refs[:L] == 0)[0]
    to = np.arange(len(refs), dtype=np.int32)
    to[src] = dst
    pools[:, dst] = pools[:, src]
    rf = np.zeros_like(refs)
    rf[to[live]] = refs[live]
    t = np.full_like(table, -1)
    for s in range(table.shape[0]):
        t[s, :nb(lens[s])] = to[table[s, :nb(lens[s])]]
    return t, lens.copy(), rf, L


def verify(p, q, draft, n_draft, u):
    """p [B][T+1][V], q [B][T][V] or None, in float64 (exact values of the
    inputs); (tokens, n_acc)."""
    B, T1, V = p.shape
    tokens, acc = np.full((B, T1), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        i = 0
        while i < n_draft[b]:
            x = draft[b, i]
            if not (0 <= x < V) or not u[b, i] * (1.0 if q is None else q[b, i, x]) < p[b, i, x]:
                break
            tokens[b, i] = x
            i += 1
        acc[b] = i
        clean = lambda w: np.where((w > 0) & np.isfinite(w), w, 0.0)  # noqa: E731
        w = clean(p[b, i])
        if i < n_draft[b]:
            sub = np.zeros(V)
            if q is not None:
                sub = q[b, i]
            elif 0 <= draft[b, i] < V:
                sub[draft[b, i]] = p[b, i, draft[b, i]]
            rest = clean(p[b, i] - sub)
            if rest.sum() > 0:
                w = rest
        cum = np.cumsum(w)
        if cum[-1] > 0:
            past = np.nonzero(cum > u[b, T1 - 1] * cum[-1])[0]
            tokens[b, i] = past[0] if len(past) else np.nonzero(w)[0][-1]
    return tokens, acc
