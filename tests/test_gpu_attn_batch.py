"""GPU parity of the batch's decode attention (moe_attn_batch) with a plain
evaluation in 64 bits.

Tolerance, from the roundings: the output is rounded once (half a step of the
type, h = eps / 2, relative) and so is each softmax weight before it
multiplies V, while the sum of the weights takes the rounded ones. An element
o = sum w_j v_j is therefore off by at most h |o| + h sum w_j |v_j| (1 + h)
plus h |o| from the normaliser, and fp32 sums, the exponential and the scores
(|x| <= 40 in log2 units, error 40 x 2^-22) add less than 2^-15 of
sum w_j |v_j|. The tests bound every element by
2 h |o| + h A + 2^-14 A with A = sum w_j |v_j|."""
import numpy as np
import pytest
import torch

import bit_moe_expert_histogram_gb300 as m

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    m.load()


class Case:
    """Slots with given (len, n_new) over random pages, the first `prefix`
    blocks shared; rows of pages past a slot's end hold NaN."""

    def __init__(self, seed, pairs, T, n_q, n_kv, D, prefix=0, dtype="bf16", scale=2.0, extra=0):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.dims = (len(pairs), T, n_q, n_kv, D, prefix, dtype)
        dt = TYPES[dtype]
        B = len(pairs)
        need = [max(0, -(-n // 64) - prefix) for n, _ in pairs]
        n_phys = prefix + sum(need) + 2
        pages = rng.permutation(n_phys).astype(np.int32)
        width = prefix + max(need + [1]) + extra
        table = np.full((B, width), -1, np.int32)
        self.k = torch.full((n_phys, n_kv, 64, D), float("nan"), dtype=dt)
        self.v = self.k.clone()
        rnd = lambda *s: torch.randn(s, generator=g).to(dt)  # noqa: E731
        for p in pages[:prefix]:
            self.k[p], self.v[p] = rnd(n_kv, 64, D), rnd(n_kv, 64, D)
        at = prefix
        for s, (n, _) in enumerate(pairs):
            for j in range(need[s]):
                p = pages[at]
                at += 1
                table[s, prefix + j] = p
                rows = min(64, n - (prefix + j) * 64)
                self.k[p, :, :rows], self.v[p, :, :rows] = rnd(n_kv, rows, D), rnd(n_kv, rows, D)
        self.q = (torch.randn((B, T, n_q, D), generator=g) * scale).to(dt)
        self.table, self.prefix = table, pages[:prefix]
        self.lens = np.array([n for n, _ in pairs], np.int32)
        self.n_new = np.array([t for _, t in pairs], np.int32)

    def run(self, n_new=True, q=None, table=None, prefix=None, status=0, lens=None):
        B, T, n_q, n_kv, D, P, dtype = self.dims
        up = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV)  # noqa: E731
        table = self.table if table is None else table
        prefix = self.prefix if prefix is None else prefix
        shape = m.make_attn_batch_shape(B, T, n_q, n_kv, D, table.shape[1], P, dtype)
        ws = m.alloc_attn_batch_workspace(shape, DEV)
        o = torch.full((B, T, n_q, D), 7.0, dtype=TYPES[dtype], device=DEV)
        outs = []
        for _ in range(2):  # the second call finds the counters as the first left them
            m.moe_attn_batch(shape, self.q.to(DEV) if q is None else q, self.k.to(DEV),
                             self.v.to(DEV), up(table), up(self.lens if lens is None else lens), o,
                             ws, n_new=up(self.n_new) if n_new else None,
                             prefix=up(prefix) if P else None)
            assert m.moe_query_device_status(ws) == status
            outs.append(o.cpu().view(torch.int16))
        assert torch.equal(*outs)  # the same bits each time
        return o.cpu().double().numpy()

    def want(self, skip=()):
        """(o, A): the result and the sums of w_j |v_j|; skip: pages left out."""
        B, T, n_q, n_kv, D, P, _ = self.dims
        k, v, q = self.k.double().numpy(), self.v.double().numpy(), self.q.double().numpy()
        o, A = np.zeros((B, T, n_q, D)), np.zeros((B, T, n_q, D))
        G = n_q // n_kv
        for s in range(B):
            L, n = int(self.lens[s]), int(self.n_new[s])
            blocks = [self.prefix[j] if j < P else self.table[s, j] for j in range(-(-L // 64))]
            for h in range(n_kv):
                kk = np.concatenate([k[p, h] for p in blocks] or [np.zeros((0, D))])[:L]
                vv = np.concatenate([v[p, h] for p in blocks] or [np.zeros((0, D))])[:L]
                gone = np.repeat([p in skip for p in blocks], 64)[:L].astype(bool)
                kk, vv = np.where(gone[:, None], 0, kk), np.where(gone[:, None], 0, vv)
                for t in range(n):
                    pos = L - n + t
                    if pos < 0:
                        continue
                    x = q[s, t, h * G:(h + 1) * G] @ kk[:pos + 1].T / np.sqrt(D)
                    x = np.where(gone[:pos + 1], -np.inf, x)
                    if not np.isfinite(x).any():
                        continue
                    w = np.exp(x - x.max(-1, keepdims=True))
                    w /= w.sum(-1, keepdims=True)
                    o[s, t, h * G:(h + 1) * G] = w @ vv[:pos + 1]
                    A[s, t, h * G:(h + 1) * G] = w @ np.abs(vv[:pos + 1])
        return o, A

    def check(self, skip=(), **kw):
        got = self.run(**kw)
        o, A = self.want(skip)
        h = torch.finfo(TYPES[self.dims[-1]]).eps / 2
        assert np.isfinite(got).all()
        off = np.abs(got - o) - (2 * h * np.abs(o) + h * A + 2.0 ** -14 * A)
        assert off.max() <= 0, "over by %.3g at %s" % (off.max(),
                                                       np.unravel_index(off.argmax(), off.shape))
        return got


LENGTHS = [1, 2, 63, 64, 65, 128, 200, 777]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n_q,n_kv,D", [(16, 2, 128), (8, 8, 64), (12, 4, 64), (5, 1, 128),
                                        (64, 1, 128), (32, 1, 64)])
def test_single_tokens(n_q, n_kv, D, dtype):
    Case(n_q + D, [(n, 1) for n in LENGTHS], 1, n_q, n_kv, D, dtype=dtype).check()


@pytest.mark.parametrize("T,n_q,n_kv,D", [(2, 16, 2, 128), (4, 16, 2, 64), (8, 16, 2, 128),
                                          (3, 12, 4, 64), (64, 2, 2, 64), (7, 9, 1, 128)])
def test_drafts_of_uneven_number(T, n_q, n_kv, D):
    """Fewer new tokens than T, a slot's first tokens of all, idle slots; new
    tokens on both sides of a page's end."""
    pairs = [(100, T), (64 + T // 2, T), (T, T), (300, 1), (0, 0), (65, min(2, T)), (129, 0)]
    Case(T, pairs, T, n_q, n_kv, D).check()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("prefix", [1, 2, 3, 9])
@pytest.mark.parametrize("T,n_q,n_kv,D", [(1, 16, 2, 128), (3, 12, 4, 64), (4, 16, 2, 128)])
def test_shared_prefix(T, n_q, n_kv, D, prefix, dtype):
    """Slots that end past the prefix, with it, inside it, before it."""
    P = prefix * 64
    pairs = [(P + 5, T), (P + 200, T), (P + 64, 1), (P, T), (P - 10, T), (T, T), (0, 0), (P + 1, 1)]
    Case(prefix * 10 + T, pairs, T, n_q, n_kv, D, prefix=prefix, dtype=dtype).check()


@pytest.mark.parametrize("B,T,n_q,n_kv,D,prefix", [(300, 1, 16, 2, 128, 5), (40, 5, 16, 2, 128, 40),
                                                   (130, 2, 8, 8, 64, 17), (2, 1, 16, 2, 128, 150),
                                                   (1, 1, 4, 1, 128, 64), (33, 1, 16, 2, 64, 33)])
def test_many_slots_on_a_prefix(B, T, n_q, n_kv, D, prefix):
    rng = np.random.default_rng(B)
    pairs = [(prefix * 64 + int(rng.integers(T, 400)), int(rng.integers(1, T + 1))) for _ in range(B)]
    Case(B + 1, pairs, T, n_q, n_kv, D, prefix=prefix).check()


@pytest.mark.parametrize("B,T,n_q,n_kv,D,prefix,extra,new", [
    (130, 4, 32, 4, 128, 4, 200, "few"), (130, 4, 32, 4, 128, 4, 0, "some"),
    (64, 8, 8, 8, 64, 20, 0, "one"), (64, 8, 8, 8, 64, 20, 40, "none"),
    (300, 4, 16, 2, 64, 30, 3, "all"), (90, 1, 8, 8, 128, 17, 0, "some")])
def test_shared_part_beside_the_own_lines(B, T, n_q, n_kv, D, prefix, extra, new):
    """The SMs are divided by what there is of both: few and many tokens,
    short and long own lines, tables wider than any length, nothing at all."""
    rng = np.random.default_rng(B + extra)
    n_new = {"few": rng.integers(0, T + 1, B) * (rng.random(B) < 0.1),
             "some": rng.integers(0, T + 1, B), "one": (np.arange(B) == 41) * T,
             "none": np.zeros(B), "all": np.full(B, T)}[new].astype(int)
    own = rng.integers(1, 100, B)
    own[B // 2] = 2000  # one slot goes on long after the others
    own[3] = -100  # and one ends inside the prefix
    Case(B, [(prefix * 64 + int(a), int(t)) for a, t in zip(own, n_new)], T, n_q, n_kv, D,
         prefix=prefix, extra=extra).check()


def test_long_and_short_slots_together():
    pairs = [(9000, 1), (3, 1), (0, 0), (64 * 90, 1), (1, 1), (4097, 1)]
    Case(17, pairs, 1, 16, 2, 128).check()


def test_n_new_left_out_and_more_than_the_length():
    """n_new None means T; a slot with fewer positions than new tokens has
    rows before its first position: they are 0."""
    c = Case(5, [(70, 3), (2, 3), (0, 3), (3, 3)], 3, 16, 2, 128)
    got = c.check(n_new=False)
    assert not got[1, 0].any() and not got[2].any() and got[1, 1].any()


def test_sharp_and_flat_rows():
    """Scores far apart (one position takes everything, in the first page or
    the last) and all alike (the mean of the values)."""
    c = Case(9, [(500, 1), (64 * 4 + 70, 1)], 1, 16, 2, 128, prefix=4, scale=0.0)
    got = c.check()
    assert np.isfinite(got).all()
    c = Case(10, [(500, 1), (64 * 4 + 70, 1)], 1, 16, 2, 128, prefix=4, scale=3.0)
    big = c.k[c.prefix[1], 0, 3].double()
    c.q[0, 0, 0] = (big * 2).to(c.q.dtype)
    last = c.k[c.table[1, 5], 1, 5].double()
    c.q[1, 0, 15] = (last * 2).to(c.q.dtype)
    c.check()


def test_large_scores_do_not_overflow():
    for dtype in ("bf16", "fp16"):
        c = Case(11, [(400, 2), (64 * 3 + 9, 1)], 2, 16, 2, 128, prefix=3, dtype=dtype, scale=1.0)
        c.q[:] = (c.q.double() * 20).to(c.q.dtype)
        got = c.run()
        assert np.isfinite(got).all()


def test_growing_scores_rescale_what_is_there():
    """Every block's scores lie above the last one's, so the running maximum
    moves with every block, in the shared part and the own one."""
    c = Case(12, [(64 * 12 + 300, 1)] * 3, 1, 16, 2, 128, prefix=12, scale=0.2)
    ramp = torch.arange(17) * 2.0
    for j in range(12):
        c.k[c.prefix[j], :, :, 0] = ramp[j]
    for s in range(3):
        for j in range(12, 17):
            p = c.table[s, j]
            c.k[p, :, :, 0] = torch.where(torch.isnan(c.k[p, :, :, 0]), c.k[p, :, :, 0], ramp[j].to(c.k.dtype))
    c.q[..., 0] = 12.0
    c.check()


def test_joint_projection_slices():
    c = Case(13, [(100, 3), (65, 2), (700, 3)], 3, 16, 2, 128)
    B, T, n_q, n_kv, D, _, _ = c.dims
    qkv = torch.randn((B, T, n_q + 2 * n_kv, D)).to(c.q.dtype)
    qkv[:, :, :n_q] = c.q
    c.check(q=qkv.to(DEV)[:, :, :n_q])


def test_absent_rows_are_zero_whatever_lies_there():
    """Queries of tokens that are not there hold NaN; a slot whose values are
    infinite gives infinities to its own row only, and zeros to absent ones."""
    for prefix in (0, 40):
        P = 64 * prefix
        c = Case(20 + prefix, [(P + 100, 1), (P + 70, 2), (0, 0), (P + 5, 3)] * 8, 3, 16, 2, 128,
                 prefix=prefix)
        for s in range(32):
            c.q[s, c.n_new[s]:] = float("nan")
        got = c.check()
        page = c.table[0, prefix]
        c.v[page, 0, 3, 5] = float("inf")
        again = c.run()
        assert np.isposinf(again[0, 0, :8, 5]).all()
        again[0, 0, :8, 5] = got[0, 0, :8, 5]
        np.testing.assert_array_equal(again, got)


def test_pages_past_32_bits_of_elements():
    """A pool of 150000 pages of 2 heads: 2.5e9 elements, the pages used at its
    end, in a per-slot call and in one with a shared part."""
    n_phys, n_kv, D = 150000, 2, 128
    for prefix in (0, 60):
        c = Case(31, [(64 * prefix + 200, 1)] * 12, 1, 16, n_kv, D, prefix=prefix)
        small = c.k.shape[0]
        big = torch.zeros((n_phys, n_kv, 64, D), dtype=c.k.dtype, device=DEV)
        bigv = torch.zeros_like(big)
        big[n_phys - small:] = c.k.to(DEV)
        bigv[n_phys - small:] = c.v.to(DEV)
        off = n_phys - small
        up = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV)  # noqa: E731
        shape = m.make_attn_batch_shape(12, 1, 16, n_kv, D, c.table.shape[1], prefix)
        ws = m.alloc_attn_batch_workspace(shape, DEV)
        o = torch.empty((12, 1, 16, D), dtype=c.k.dtype, device=DEV)
        m.moe_attn_batch(shape, c.q.to(DEV), big, bigv, up(np.where(c.table < 0, -1, c.table + off)),
                         up(c.lens), o, ws, prefix=up(c.prefix + off) if prefix else None)
        assert m.moe_query_device_status(ws) == 0
        np.testing.assert_array_equal(o.cpu().double().numpy(), c.run())
        del big, bigv


def test_two_streams_with_their_own_workspaces():
    cases = [Case(41, [(64 * 30 + 90, 2)] * 40, 2, 16, 2, 128, prefix=30),
             Case(42, [(700, 1)] * 30, 1, 8, 8, 64)]
    want = [c.run() for c in cases]
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV)  # noqa: E731
    work = []
    for c in cases:
        B, T, n_q, n_kv, D, P, dtype = c.dims
        shape = m.make_attn_batch_shape(B, T, n_q, n_kv, D, c.table.shape[1], P, dtype)
        work.append((shape, c.q.to(DEV), c.k.to(DEV), c.v.to(DEV), up(c.table), up(c.lens),
                     torch.empty_like(c.q, device=DEV), m.alloc_attn_batch_workspace(shape, DEV),
                     up(c.n_new), up(c.prefix) if P else None, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for shape, q, k, v, tab, ln, o, ws, nn, pre, st in work:
            with torch.cuda.stream(st):
                m.moe_attn_batch(shape, q, k, v, tab, ln, o, ws, n_new=nn, prefix=pre)
    torch.cuda.synchronize()
    for w, x in zip(want, work):
        np.testing.assert_array_equal(x[6].cpu().double().numpy(), w)


def test_bad_pages_are_recorded_and_left_out():
    c = Case(14, [(64 * 3 + 250, 1), (64 * 3 + 10, 1)], 1, 16, 2, 128, prefix=3)
    t = c.table.copy()
    bad = t[0, 4]
    t[0, 4] = c.k.shape[0]
    c.check(skip=(bad,), table=t, status=m.MOE_ERR_BAD_INPUT)
    pre = c.prefix.copy()
    bad = pre[1]
    pre[1] = -3
    c.check(skip=(bad,), prefix=pre, status=m.MOE_ERR_BAD_INPUT)
    # nothing but bad pages: the row sees nothing
    c = Case(15, [(64, 1)], 1, 16, 2, 128)
    t = np.full_like(c.table, 1 << 30)
    got = c.run(table=t, status=m.MOE_ERR_BAD_INPUT)
    assert not got.any()


def test_bad_lengths_are_brought_into_range():
    c = Case(16, [(128, 1), (128, 1), (128, 1)], 1, 16, 2, 128)
    good = c.run()
    got = c.run(lens=[128, -1, 129], status=m.MOE_ERR_BAD_INPUT)
    np.testing.assert_array_equal(got[0], good[0])
    assert not got[1].any()
    np.testing.assert_array_equal(got[2], good[2])  # 129 past a row of two pages counts as 128


def test_in_a_graph_on_a_side_stream():
    c = Case(18, [(64 * 5 + 100, 1)] * 20, 1, 16, 2, 128, prefix=5)
    B, T, n_q, n_kv, D, P, dtype = c.dims
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    shape = m.make_attn_batch_shape(B, T, n_q, n_kv, D, c.table.shape[1], P, dtype)
    ws = m.alloc_attn_batch_workspace(shape, DEV)
    q, k, v, tab, ln = c.q.to(DEV), c.k.to(DEV), c.v.to(DEV), up(c.table), up(c.lens)
    pre, o = up(c.prefix), torch.empty_like(c.q, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        m.moe_attn_batch(shape, q, k, v, tab, ln, o, ws, prefix=pre)
    first = c.run()
    for step in range(3):  # the graph reads the lengths of the time
        g.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(o.cpu().double().numpy(), first)
    ln.fill_(64 * 5)
    g.replay()
    torch.cuda.synchronize()
    c.lens[:] = 64 * 5
    np.testing.assert_array_equal(o.cpu().double().numpy(), c.run())


def test_binding_refuses_wrong_tensors():
    c = Case(19, [(100, 1), (65, 1)], 1, 16, 2, 128)
    shape = m.make_attn_batch_shape(2, 1, 16, 2, 128, c.table.shape[1], 0, "bf16")
    ws = m.alloc_attn_batch_workspace(shape, DEV)
    q, k = c.q.to(DEV), c.k.to(DEV)
    tab = torch.from_numpy(c.table).to(DEV)
    ln = torch.from_numpy(c.lens).to(DEV)
    o = torch.empty_like(q)
    for bad in (dict(q=q[:1]), dict(q=q.half()), dict(k=k[:, :1]), dict(tab=tab[:, :1]),
                dict(ln=ln.long()), dict(o=o.transpose(1, 2)), dict(v=k.float()),
                dict(pre=torch.zeros(3, dtype=torch.int32, device=DEV))):
        a = {**dict(q=q, k=k, v=k, tab=tab, ln=ln, o=o, pre=None), **bad}
        with pytest.raises(ValueError):
            m.moe_attn_batch(shape, a["q"], a["k"], a["v"], a["tab"], a["ln"], a["o"], ws,
                             prefix=a["pre"])
