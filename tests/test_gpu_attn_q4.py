"""Attention over 4-bit pages against 64 bits. The bound counts the roundings
that the call's documentation allows (tests/q4_ref.py derives it) and the
output's own, half a step."""
import numpy as np
import pytest
import torch

import bit_moe_expert_histogram_gb300 as m
import q4_ref as ref

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


def ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV)


class Case:
    """Slots (length, new tokens) over pools whose rows past a slot's end hold
    anything, scales that are NaN or infinite among it."""

    def __init__(self, seed, slots, T, n_q, n_kv, D, dtype="bf16", k_std=1.0, v_std=1.0, v_spread=0.5):
        rng = self.rng = np.random.default_rng(seed)
        B = len(slots)
        self.dims = (B, T, n_q, n_kv, D)
        self.dtype = dtype
        self.lens = np.array([s[0] for s in slots], np.int32)
        self.new = np.array([s[1] for s in slots], np.int32)
        nb = -(-np.clip(self.lens, 0, None) // 64)
        n_phys = int(nb.sum()) + 2
        self.table = np.full((B, max(1, int(nb.max()))), -1, np.int32)
        pages = rng.permutation(n_phys)
        self.q = torch.from_numpy(rng.normal(size=(B, T, n_q, D))).to(TYPES[dtype])
        shape = (n_phys, n_kv, 64, ref.units(D))
        self.k, self.v = [rng.integers(-32768, 32768, shape, dtype=np.int16) for _ in range(2)]
        at = 0
        for s in range(B):
            self.table[s, :nb[s]] = pages[at:at + nb[s]]
            at += nb[s]
            for j in range(nb[s]):
                n = min(64, self.lens[s] - 64 * j)
                for pool, std in ((self.k, k_std), (self.v, v_std)):
                    x = rng.normal(size=(n_kv, n, D)) * std * np.exp(v_spread * rng.normal(size=(n_kv, n, 1)))
                    pool[self.table[s, j], :, :n] = ref.pack(*ref.quantise(x.astype(np.float32)))

    def shape(self):
        B, T, n_q, n_kv, D = self.dims
        return m.make_attn_batch_shape(B, T, n_q, n_kv, D, self.table.shape[1], dtype=self.dtype)

    def call(self, ws=None, q=None):
        shape = self.shape()
        if ws is None:
            ws = m.alloc_attn_batch_q4_workspace(shape, DEV)
        self.ws = ws
        q = self.q.to(DEV) if q is None else q
        o = torch.full(self.q.shape, 7.0, dtype=self.q.dtype, device=DEV)
        m.moe_attn_batch_q4(shape, q, torch.from_numpy(self.k).to(DEV), torch.from_numpy(self.v).to(DEV),
                            ints(self.table), ints(self.lens), o, ws, n_new=ints(self.new))
        return o

    def check(self, status=0, o=None, lens=None, new=None):
        if o is None:
            o = self.call()
            assert m.moe_query_device_status(self.ws) == status
        got = o.cpu().double().numpy()
        want, tol = ref.attention(self.q.double().numpy(), self.k, self.v, self.table,
                                  self.lens if lens is None else lens, self.new if new is None else new)
        half = torch.finfo(self.q.dtype).eps / 2
        floor = 0.0 if self.dtype == "bf16" else 2.0**-25  # fp16's smallest numbers
        bad = ~(np.abs(got - want) <= tol + half * (np.abs(want) + tol) + floor)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], tol[bad][:4])
        return got


def some(rng, n, most, T):
    return [(int(x), int(min(x, rng.integers(0, T + 1)))) for x in rng.integers(0, most, n)]


CASES = {
    "one position": ([(1, 1)], 1, 8, 1, 128, "bf16"),
    "unit borders": ([(n, 1) for n in (1, 31, 32, 33, 63, 64, 65, 96, 97, 127, 128, 129)], 1, 16, 2, 128, "bf16"),
    "fp16, D = 64": ([(n, 1) for n in (1, 16, 31, 32, 33, 64, 100, 700)], 1, 8, 4, 64, "fp16"),
    "no new tokens, empty slots": ([(0, 0), (70, 0), (0, 1), (5, 1), (0, 0)], 1, 16, 2, 128, "bf16"),
    "more new than held": ([(1, 3), (2, 2), (0, 3), (33, 3)], 3, 6, 2, 64, "bf16"),
    "drafts": ([(300, 4), (65, 2), (4, 4), (130, 1), (64, 3)], 4, 16, 2, 128, "bf16"),
    "nine rows": ([(200, 3), (31, 1)], 3, 3, 1, 128, "fp16"),
    "seventeen rows": ([(200, 17), (90, 5)], 17, 2, 2, 64, "bf16"),
    "64 rows": ([(333, 8), (40, 8), (64, 7)], 8, 16, 2, 128, "bf16"),
    "64 tokens of one head": ([(100, 64), (64, 64), (20, 33)], 64, 1, 1, 64, "fp16"),
    "a head each": ([(150, 1), (77, 1)], 1, 8, 8, 128, "bf16"),
    "five heads on one": ([(500, 1), (1, 1)], 1, 5, 1, 128, "bf16"),
    "28 on 4, two tokens": ([(260, 2), (129, 2), (3, 1)], 2, 28, 4, 64, "fp16"),
    "one long slot": ([(20000, 1)], 1, 16, 2, 128, "bf16"),
    "long beside short": ([(9000, 2), (1, 1), (40, 2), (3000, 1), (64, 2)], 2, 8, 2, 64, "bf16"),
    "many short slots": (some(np.random.default_rng(1), 400, 200, 1), 1, 8, 2, 64, "bf16"),
    "many slots": (some(np.random.default_rng(2), 160, 600, 2), 2, 16, 2, 128, "fp16"),
}


@pytest.mark.parametrize("name", list(CASES))
def test_against_64_bits(name):
    slots, T, n_q, n_kv, D, dtype = CASES[name]
    c = Case(len(name), slots, T, n_q, n_kv, D, dtype, k_std=0.3)
    got = c.check()
    for s, (L, n) in enumerate(slots):  # what sees nothing is 0
        assert not got[s, n:].any()
        assert not got[s, :max(0, n - L)].any()


@pytest.mark.parametrize("D,dtype", [(128, "bf16"), (64, "fp16")])
@pytest.mark.parametrize("k_std,v_std,v_spread", [(3.0, 1.0, 0.5), (0.0, 1.0, 0.0), (1.0, 1e-4, 2.0), (1.0, 5.0, 2.0),
                                                  (0.01, 0.0, 0.0)])
def test_sizes_of_keys_and_values(D, dtype, k_std, v_std, v_spread):
    """Sharp and flat softmax, values small, large and of very different size
    from position to position, constant groups."""
    Case(11, [(700, 2), (64, 1), (129, 2)], 2, 8, 2, D, dtype, k_std, v_std, v_spread).check()


def test_values_far_from_1():
    """bf16 values of 1e-20 and of 1e20, and one strong position among weak ones."""
    for std in (1e-20, 1e20):
        Case(12, [(300, 1), (33, 1)], 1, 8, 1, 128, "bf16", 0.5, std).check()
    c = Case(13, [(400, 1)], 1, 8, 1, 128, "bf16", 0.5)
    x = c.rng.normal(size=(1, 128)) * 1e6
    for pos in (0, 399):
        c.v[c.table[0, pos // 64], :, pos % 64] = ref.pack(*ref.quantise(x.astype(np.float32)))
    c.check()


def test_queries_of_every_size():
    c = Case(14, [(200, 1)] * 6, 1, 8, 2, 128, "bf16")
    scale = np.array([0.0, 1e-30, 1e-6, 1.0, 4.0, 1e3])
    c.k = c.k.copy()
    c.q = (c.q.double() * torch.from_numpy(scale)[:, None, None, None]).to(torch.bfloat16)
    # the last slot's scores are so far apart that one position has all
    c.check()
    mixed = Case(15, [(200, 1)], 1, 8, 2, 64, "fp16")
    mixed.q[..., ::7] *= 2.0**-12  # elements far below the row's largest
    mixed.check()


def test_pages_that_are_none_are_left_out():
    c = Case(16, [(300, 2), (200, 1), (64, 1)], 2, 16, 2, 128)
    c.table[0, 1], c.table[1, 0], c.table[2, 0] = -1, c.k.shape[0], 1 << 30
    got = c.check(status=m.MOE_ERR_BAD_INPUT)
    assert not got[2].any()  # nothing left to see


def test_lengths_and_counts_out_of_range():
    c = Case(17, [(320, 2), (200, 1), (64, 1), (100, 2)], 2, 16, 2, 128)  # slot 0 fills its pages
    new = c.new.copy()
    c.lens = np.array([320, -5, 64, 100], np.int32)
    c.new = np.array([3, 1, -1, 2], np.int32)
    o = c.call()
    assert m.moe_query_device_status(c.ws) == m.MOE_ERR_BAD_INPUT
    c.check(o=o, lens=[320, 0, 64, 100], new=[2, 1, 0, 2])
    c.lens = np.array([320, 10**6, 64, 100], np.int32)
    c.new = new
    c.table[1] = c.table[0]
    o = c.call()
    assert m.moe_query_device_status(c.ws) == m.MOE_ERR_BAD_INPUT
    c.check(o=o, lens=[320, 320, 64, 100])


def test_queries_out_of_a_joint_projection():
    c = Case(18, [(90, 3), (40, 1)], 3, 8, 2, 64, "bf16", 0.3)
    joint = torch.full((2, 3, 12, 64), float("nan"), dtype=torch.bfloat16, device=DEV)
    joint[:, :, 2:10] = c.q.to(DEV)
    o = c.call(q=joint[:, :, 2:10])
    c.check(o=o)
    # rows without a token may hold anything
    joint[1, 1:] = float("nan")
    assert torch.equal(c.call(q=joint[:, :, 2:10]), o)


def test_one_workspace_for_a_batch_that_changes():
    rng = np.random.default_rng(19)
    cases = [Case(20 + i, *a) for i, a in enumerate((
        ([(5000, 1), (300, 1)], 1, 16, 2, 128), (some(rng, 200, 150, 1), 1, 8, 4, 64),
        ([(700, 4)] * 20, 4, 16, 2, 128), ([(3, 1)], 1, 5, 1, 64, "fp16"), (some(rng, 60, 900, 3), 3, 12, 4, 64)))]
    alone = [c.call() for c in cases]
    ws = torch.empty(max(m.load().moe_attn_batch_q4_workspace_bytes(c.shape()) for c in cases),
                     dtype=torch.uint8, device=DEV)
    m.moe_workspace_init(ws)
    for i in (0, 1, 0, 2, 3, 2, 4, 1, 4, 0, 3):
        assert torch.equal(cases[i].call(ws=ws), alone[i]), i
    assert m.moe_query_device_status(ws) == 0


def test_two_streams_with_a_workspace_each():
    a = Case(30, [(4000, 1), (900, 1)], 1, 16, 2, 128)
    b = Case(31, [(2500, 2)] * 3, 2, 8, 2, 64, "fp16")
    want = a.call(), b.call()
    up = lambda c: (c.shape(), c.q.to(DEV), torch.from_numpy(c.k).to(DEV), torch.from_numpy(c.v).to(DEV),  # noqa: E731
                    ints(c.table), ints(c.lens), torch.empty(c.q.shape, dtype=c.q.dtype, device=DEV),
                    m.alloc_attn_batch_q4_workspace(c.shape(), DEV), ints(c.new))
    calls = up(a), up(b)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        for (shape, q, k, v, table, lens, o, ws, new), s in zip(calls, streams):
            m.moe_attn_batch_q4(shape, q, k, v, table, lens, o, ws, n_new=new, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(calls[0][6], want[0]) and torch.equal(calls[1][6], want[1])


def test_a_captured_call_takes_new_lengths():
    c = Case(32, [(500, 2), (300, 1), (64, 2)], 2, 8, 2, 128, "bf16", 0.3)
    shape, ws = c.shape(), m.alloc_attn_batch_q4_workspace(c.shape(), DEV)
    q, k, v = c.q.to(DEV), torch.from_numpy(c.k).to(DEV), torch.from_numpy(c.v).to(DEV)
    table, lens, new = ints(c.table), ints(c.lens), ints(c.new)
    o = torch.empty_like(q)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            m.moe_attn_batch_q4(shape, q, k, v, table, lens, o, ws, n_new=new)
            m.moe_attn_batch_q4(shape, q, k, v, table, lens, o, ws, n_new=new)
    for now, n in (([500, 300, 64], [2, 1, 2]), ([10, 299, 1], [1, 2, 1]), ([450, 0, 33], [2, 0, 0])):
        lens.copy_(ints(now))
        new.copy_(ints(n))
        graph.replay()
        torch.cuda.synchronize()
        c.check(o=o, lens=now, new=n)


def test_pools_past_32_bits_of_bytes():
    c = Case(33, [(200, 1), (70, 1)], 1, 8, 2, 128, "bf16", 0.3)
    n_phys = 450000  # 4.6 GB a pool
    shape = m.make_cache_shape(2, c.table.shape[1], n_phys, 2, 128)
    k, v = m.alloc_q4_pool(shape, DEV), m.alloc_q4_pool(shape, DEV)
    far = np.where(c.table >= 0, n_phys - 1 - 5 * c.table, -1).astype(np.int32)
    for s, j in np.argwhere(c.table >= 0):
        k[int(far[s, j])] = torch.from_numpy(c.k[c.table[s, j]]).to(DEV)
        v[int(far[s, j])] = torch.from_numpy(c.v[c.table[s, j]]).to(DEV)
    o, ws = torch.empty_like(c.q, device=DEV), m.alloc_attn_batch_q4_workspace(c.shape(), DEV)
    m.moe_attn_batch_q4(c.shape(), c.q.to(DEV), k, v, ints(far), ints(c.lens), o, ws, n_new=ints(c.new))
    c.check(o=o)


def test_the_same_bits_every_time():
    c = Case(34, some(np.random.default_rng(3), 90, 2000, 2), 2, 16, 2, 128)
    first = c.call()
    for _ in range(5):
        assert torch.equal(c.call(ws=c.ws), first)


def test_as_the_16_bit_attention_over_the_same_numbers():
    """Rows written and read back give moe_attn_batch the numbers that
    moe_attn_batch_q4 sees (bf16 once more): both agree within the 16-bit
    rows' roundings, 2^-9 of keys, values, weights and outputs."""
    B, T, n_q, n_kv, D = 3, 2, 16, 2, 128
    lens = [260, 64, 131]
    shape = m.make_cache_shape(B, 6, 20, n_kv, D)
    page, ws = m.q4_page_shape(shape), m.alloc_cache_workspace(shape, DEV)
    k4, v4 = m.alloc_q4_pool(shape, DEV), m.alloc_q4_pool(shape, DEV)
    k16, v16 = [torch.zeros((20, n_kv, 64, D), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    a, b = m.CacheMeta.empty(shape, DEV), m.CacheMeta.empty(shape, DEV)
    g = torch.Generator().manual_seed(5)
    x, y = [torch.randn((B, 260, n_kv, D), generator=g).to(torch.bfloat16).to(DEV) for _ in range(2)]
    granted = ints([0] * B)
    m.moe_cache_reserve(page, a, ints(lens), b, granted, m.pool_table([k4, v4]), ws)
    m.moe_cache_write_q4(shape, b, granted, x, y, k4, v4, ws)
    m.moe_cache_read_q4(shape, b, None, granted, k4, v4, x, y, ws)
    m.moe_cache_write(shape, b, granted, x, y, k16, v16, ws)
    assert m.moe_query_device_status(ws) == 0
    q = (torch.randn((B, T, n_q, D), generator=g) * 0.5).to(torch.bfloat16).to(DEV)
    s = m.make_attn_batch_shape(B, T, n_q, n_kv, D, 6)
    o4, o16 = torch.empty_like(q), torch.empty_like(q)
    m.moe_attn_batch_q4(s, q, k4, v4, b.table, b.lens, o4, m.alloc_attn_batch_q4_workspace(s, DEV))
    m.moe_attn_batch(s, q, k16, v16, b.table, b.lens, o16, m.alloc_attn_batch_workspace(s, DEV))
    # |v| up to some 4: weights' and values' roundings 2 x 2^-9 of it, two
    # outputs' of |o| < 2; keys' 2^-9 of scores' magnitudes sum |q k| / sqrt(D)
    # < 8, which move weights by as much: 4 (2 + 8) 2^-9 + 4 2^-9 < 0.09
    assert (o4.float() - o16.float()).abs().max() < 0.09
    assert (o4.float() - o16.float()).abs().mean() < 0.004


def wide(c):
    """Tables so wide that tiles have sixteen rows: more blocks than are ever read."""
    B, T, n_q, n_kv, D = c.dims
    tiles = -(-T * n_q // n_kv // 16)
    warps = 8 * torch.cuda.get_device_properties(0).multi_processor_count
    blocks = warps * (48 if D == 128 else 4) // (B * n_kv * tiles) + 1
    table = np.full((B, max(blocks, c.table.shape[1])), 1 << 20, np.int32)
    table[:, :c.table.shape[1]] = c.table
    c.table = table
    return c


@pytest.mark.parametrize("name", [n for n, (_, T, n_q, n_kv, *_) in CASES.items() if T * n_q // n_kv > 8])
def test_tiles_of_sixteen_rows(name):
    slots, T, n_q, n_kv, D, dtype = CASES[name]
    got = wide(Case(len(name), slots, T, n_q, n_kv, D, dtype, k_std=0.3)).check()
    for s, (L, n) in enumerate(slots):  # what sees nothing is 0
        assert not got[s, n:].any()
        assert not got[s, :max(0, n - L)].any()


@pytest.mark.parametrize("D,dtype", [(128, "bf16"), (64, "fp16"), (128, "fp16")])
@pytest.mark.parametrize("k_std,v_std,v_spread", [(3.0, 1.0, 0.5), (1.0, 1e-4, 2.0), (1.0, 5.0, 2.0)])
def test_sizes_in_tiles_of_sixteen(D, dtype, k_std, v_std, v_spread):
    wide(Case(35, [(700, 4), (64, 1), (129, 3)], 4, 8, 2, D, dtype, k_std, v_std, v_spread)).check()


def test_sixteen_rows_over_many_units():
    """Shares of several pairs, first pieces before other pairs among them."""
    rng = np.random.default_rng(36)
    c = wide(Case(37, some(rng, 150, 1500, 4), 4, 16, 2, 128, "bf16", 0.5))
    first = c.call()
    c.check(o=first)
    for _ in range(3):
        assert torch.equal(c.call(ws=c.ws), first)
    c = wide(Case(38, some(rng, 90, 1500, 3), 3, 12, 4, 64, "fp16", 0.5))
    c.check()


@pytest.mark.parametrize("T", [1, 4])
def test_slots_that_share_pages(T):
    """Forked slots: one table's pages in several, cut at different lengths."""
    c = Case(39, [(700, T)] * 6, T, 16, 2, 128, "bf16", 0.5)
    c.table[1:] = c.table[0]
    c.lens = np.array([700, 640, 641, 64, 699, 5], np.int32)
    for s in range(6):  # pages past a slot's end are another's
        c.new[s] = min(T, c.lens[s])
    c.check()


def test_a_page_that_is_none_in_tiles_of_sixteen():
    c = wide(Case(40, [(300, 2), (200, 1), (64, 1)], 2, 16, 2, 128))
    c.table[0, 1], c.table[1, 0], c.table[2, 0] = -1, c.k.shape[0], 1 << 30
    got = c.check(status=m.MOE_ERR_BAD_INPUT)
    assert not got[2].any()
