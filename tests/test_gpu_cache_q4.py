"""Rows of a 4-bit cache on the GPU: written rows are the reference's bit for
bit (the decisions are exact by definition), what is read back is each code's
number rounded once, pages move as 16-bit pools do."""
import numpy as np
import pytest
import torch

import bit_moe_expert_histogram_gb300 as m
import q4_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    m.load()


def ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV)


class State:
    """Slots with pages at random places and pools that hold anything."""

    def __init__(self, seed, lens, n_kv, D, spare=3, width=None):
        self.rng = np.random.default_rng(seed)
        self.lens = np.array(lens, np.int32)
        nb = -(-np.maximum(self.lens, 0) // 64)
        n_phys = int(nb.sum()) + spare
        self.table = np.full((len(lens), width or int(nb.max()) + 1), -1, np.int32)
        pages = self.rng.permutation(n_phys)
        at = 0
        for i, n in enumerate(nb):
            self.table[i, :n] = pages[at:at + n]
            at += n
        self.shape = m.make_cache_shape(len(lens), self.table.shape[1], n_phys, n_kv, D)
        self.ws = m.alloc_cache_workspace(self.shape, DEV)
        shape = (n_phys, n_kv, 64, ref.units(D))
        self.k0, self.v0 = [self.rng.integers(-32768, 32768, shape, dtype=np.int16) for _ in range(2)]
        self.k, self.v = torch.from_numpy(self.k0).to(DEV), torch.from_numpy(self.v0).to(DEV)

    def meta(self):
        return m.CacheMeta(ints(self.table), ints(self.lens),
                           torch.ones(self.shape.n_phys, dtype=torch.int32, device=DEV))

    def written(self, pool, x, first, n):
        """`pool` with rows x float64 [B][T][n_kv][D] at first[s] + t."""
        out = pool.copy()
        rows = ref.pack(*ref.quantise(x))
        for s in range(len(n)):
            for t in range(n[s]):
                pos = first[s] + t
                out[self.table[s, pos // 64], :, pos % 64] = rows[s, t]
        return out


def rows(rng, shape, dtype):
    x = rng.normal(size=shape) * np.exp(rng.normal(size=shape[:-1] + (1,)))
    return torch.from_numpy(x).to(TYPES[dtype])


CASES = [([1], 1, 1, 128, "bf16"), ([64, 65, 63, 1], 1, 2, 128, "bf16"), ([200, 7, 130], 7, 3, 64, "fp16"),
         ([300, 129, 0, 64, 500], 130, 2, 128, "fp16"), ([70] * 40, 3, 1, 64, "bf16"),
         ([1000, 333], 333, 8, 128, "bf16")]


@pytest.mark.parametrize("lens,T,n_kv,D,dtype", CASES)
def test_written_rows_are_the_formulas(lens, T, n_kv, D, dtype):
    st = State(sum(lens), lens, n_kv, D)
    B = len(lens)
    n = np.array([min(x, T if i % 3 != 2 else T // 2) for i, x in enumerate(lens)], np.int32)
    kv = rows(st.rng, (B, T, 2 * n_kv, D), dtype)  # keys and values side by side
    x = kv.to(DEV)
    m.moe_cache_write_q4(st.shape, st.meta(), ints(n), x[:, :, :n_kv], x[:, :, n_kv:], st.k, st.v, st.ws)
    assert m.moe_query_device_status(st.ws) == 0
    kd = kv.double().numpy()
    first = st.lens - n
    for pool, old, part in ((st.k, st.k0, kd[:, :, :n_kv]), (st.v, st.v0, kd[:, :, n_kv:])):
        np.testing.assert_array_equal(pool.cpu().numpy(), st.written(old, part, first, n))


def test_every_slot_writes_t_without_counts():
    st = State(9, [5, 70], 2, 128)
    k, v = rows(st.rng, (2, 5, 2, 128), "bf16"), rows(st.rng, (2, 5, 2, 128), "bf16")
    m.moe_cache_write_q4(st.shape, st.meta(), None, k.to(DEV), v.to(DEV), st.k, st.v, st.ws)
    np.testing.assert_array_equal(st.v.cpu().numpy(),
                                  st.written(st.v0, v.double().numpy(), st.lens - 5, [5, 5]))


def special_rows(D, dtype):
    """Groups where a rounding could change a code, a scale or a bias."""
    q = D // 4
    rng = np.random.default_rng(D)
    tiny, big = (2.0**-133, 2.0**126) if dtype == "bf16" else (2.0**-24, 32752.0)
    g = [np.zeros(q), -np.zeros(q), np.full(q, 3.140625), np.full(q, -1.0 - 2.0**-10), np.full(q, tiny),
         np.arange(q) % 16 * 0.5,                       # every x on a code
         (np.arange(q) % 31) * 0.5,                     # every second x on a border (step 1)
         np.where(np.arange(q) % 2, 16.0, 241 / 256), np.where(np.arange(q) % 2, 16.0, 211 / 256),
         tiny * (np.arange(q) % 16), tiny * (np.arange(q) % 7), -tiny * (np.arange(q) % 3),
         np.where(np.arange(q) % 5, -big, big), np.where(np.arange(q) % 5, tiny, big),
         np.where(np.arange(q) % 3, -tiny, -big), 100.0 + np.arange(q) / 16, -100.0 - np.arange(q) / 16,
         np.linspace(-7.5, 7.5, q), np.linspace(0, 1, q) ** 4, big * rng.uniform(-1, 1, q),
         # borders approached from both sides, at many steps
         *[(np.arange(q) % 15 + 0.5) * s * (1 + rng.integers(-2, 3, q) * 2.0**-8) for s in (1.0, 1.3125, 0.0703125)],
         *[rng.uniform(1, 2) * np.exp2(rng.integers(-10, 10)) * rng.normal(size=q) for _ in range(400)]]
    while len(g) % 4:
        g.append(np.zeros(q))
    x = torch.from_numpy(np.stack(g).reshape(len(g) // 4, D)).to(TYPES[dtype])
    return x


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_borders_and_extremes(D, dtype):
    x = special_rows(D, dtype)
    n = x.shape[0]
    st = State(1, [n], 1, D)
    x = x.view(1, n, 1, D)
    m.moe_cache_write_q4(st.shape, st.meta(), None, x.to(DEV), x.flip(-1).contiguous().to(DEV), st.k, st.v, st.ws)
    for pool, old, y in ((st.k, st.k0, x), (st.v, st.v0, x.flip(-1))):
        np.testing.assert_array_equal(pool.cpu().numpy(), st.written(old, y.double().numpy(), [0], [n]))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_many_random_rows_bit_for_bit(dtype):
    """A million elements: some dozens come within fp32's error of a border."""
    st = State(2, [4096], 2, 128)
    k = torch.randn((1, 4096, 2, 128), generator=torch.Generator().manual_seed(3)).to(TYPES[dtype])
    m.moe_cache_write_q4(st.shape, st.meta(), None, k.to(DEV), (k * 7).to(DEV), st.k, st.v, st.ws)
    np.testing.assert_array_equal(st.k.cpu().numpy(), st.written(st.k0, k.double().numpy(), [0], [4096]))
    np.testing.assert_array_equal(st.v.cpu().numpy(), st.written(st.v0, (k * 7).double().numpy(), [0], [4096]))


@pytest.mark.parametrize("D", [64, 128])
def test_a_group_that_is_not_finite_leaves_the_others(D):
    st = State(3, [3], 1, D)
    x = rows(st.rng, (1, 3, 1, D), "bf16")
    want = st.written(st.k0, x.double().numpy(), [0], [3])
    x[0, 0, 0, 5], x[0, 1, 0, D // 4], x[0, 2, 0, D - 1] = float("nan"), float("inf"), float("-inf")
    m.moe_cache_write_q4(st.shape, st.meta(), None, x.to(DEV), x.to(DEV), st.k, st.v, st.ws)
    out = [torch.zeros((1, 3, 1, D), device=DEV) for _ in range(2)]
    m.moe_cache_read_q4(st.shape, st.meta(), None, None, st.k, st.v, *out, st.ws)
    assert m.moe_query_device_status(st.ws) == 0
    got = out[0].cpu().double().numpy().reshape(3, 4, D // 4)
    for t in range(3):
        good = ref.values(want[st.table[0, 0], 0, t], D).reshape(4, D // 4)
        hit = (0, 1, 3)[t]
        for g in range(4):
            if g == hit:
                assert not np.isfinite(got[t, g]).any()
            else:
                np.testing.assert_array_equal(got[t, g], good[g].astype(np.float32))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("lens,T,n_kv,D", [([1], 1, 1, 128), ([130, 64, 0, 5], 66, 3, 64), ([700, 80], 200, 2, 128)])
def test_rows_are_read_back(dtype, lens, T, n_kv, D):
    st = State(T, lens, n_kv, D)
    x = st.rng.normal(size=(st.shape.n_phys, n_kv, 64, D)) * 3
    st.k.copy_(torch.from_numpy(ref.pack(*ref.quantise(x))))
    st.v.copy_(torch.from_numpy(ref.pack(*ref.quantise(-x / 5))))
    B = len(lens)
    n = np.minimum(st.lens, [T - i for i in range(B)]).astype(np.int32)
    first = np.array([st.rng.integers(0, L - a + 1) for L, a in zip(lens, n)], np.int32)
    dt = TYPES[dtype]
    both = torch.full((B, T, 2 * n_kv, D), 7.0, dtype=dt, device=DEV)  # side by side
    m.moe_cache_read_q4(st.shape, st.meta(), ints(first), ints(n), st.k, st.v, both[:, :, :n_kv],
                        both[:, :, n_kv:], st.ws)
    assert m.moe_query_device_status(st.ws) == 0
    for pool, got in ((st.k, both[:, :, :n_kv]), (st.v, both[:, :, n_kv:])):
        want = torch.full((B, T, n_kv, D), 7.0, dtype=torch.float64)
        val = ref.values(pool.cpu().numpy(), D)
        for s in range(B):
            for t in range(n[s]):
                pos = first[s] + t
                want[s, t] = torch.from_numpy(val[st.table[s, pos // 64], :, pos % 64])
        # an fp32 number rounded again may lie half a step of fp32 off a tie
        tol = torch.finfo(dt).eps / 2 * (1 + 2.0**-12)
        err = (got.cpu().double() - want).abs()
        assert (err <= tol * want.abs() + 2.0**-25).all()


def test_reading_without_ranges_starts_at_the_front():
    st = State(4, [64, 100], 1, 128)
    x = rows(st.rng, (2, 64, 1, 128), "bf16")
    m.moe_cache_write_q4(st.shape, m.CacheMeta(ints(st.table), ints([64, 64]), st.meta().refs), None,
                         x.to(DEV), x.to(DEV), st.k, st.v, st.ws)
    out = [torch.zeros((2, 64, 1, 128), device=DEV) for _ in range(2)]
    m.moe_cache_read_q4(st.shape, st.meta(), None, None, st.k, st.v, *out, st.ws)
    q, s, b = ref.quantise(x.double().numpy())
    want = q * np.repeat(s, 32, -1) + np.repeat(b, 32, -1)
    np.testing.assert_array_equal(out[1].cpu().numpy(), want.astype(np.float32))


def test_bad_counts_lengths_and_pages_leave_their_slot_out():
    lens = [100, 100, 100, 100, 100]
    st = State(5, lens, 2, 64)
    k = rows(st.rng, (5, 70, 2, 64), "fp16")
    bad = State(5, lens, 2, 64)
    bad.table[4, 1] = st.shape.n_phys
    n = np.array([71, -1, 70, 70, 70], np.int32)
    meta = m.CacheMeta(ints(bad.table), ints([100, 100, 69, 100, 100]), st.meta().refs)
    m.moe_cache_write_q4(st.shape, meta, ints(n), k.to(DEV), k.to(DEV), st.k, st.v, st.ws)
    assert m.moe_query_device_status(st.ws) == m.MOE_ERR_BAD_INPUT
    want = st.written(st.k0, k.double().numpy(), [0, 0, 0, 30, 0], [0, 0, 0, 70, 0])
    # slot 4: positions 30 .. 63 lie on its first page
    want = st.written(want, np.repeat(k[4:].double().numpy(), 5, 0), [0, 0, 0, 0, 30], [0, 0, 0, 0, 34])
    np.testing.assert_array_equal(st.k.cpu().numpy(), want)
    for first, count, length in ((31, 70, 100), (-1, 5, 100), (0, 71, 100), (0, -1, 100), (0, 5, -3),
                                 (0, 5, 10**6), (2**31 - 1, 5, 100), (0, 5, -2**31)):
        out = [torch.full((5, 70, 2, 64), 9.0, device=DEV) for _ in range(2)]
        meta = m.CacheMeta(ints(st.table), ints([100, length, 100, 100, 100]), st.meta().refs)
        m.moe_cache_read_q4(st.shape, meta, ints([0, first, 0, 0, 0]), ints([3, count, 0, 0, 0]), st.k, st.v,
                            *out, st.ws)
        assert m.moe_query_device_status(st.ws) == m.MOE_ERR_BAD_INPUT
        assert (out[0][1:] == 9).all() and (out[0][0, :3] != 9).any() and (out[0][0, 3:] == 9).all()


def test_page_calls_move_4_bit_pools():
    """Fork, reserve with copy-on-write and compact, then read: the same numbers."""
    shape = m.make_cache_shape(3, 6, 24, 2, 128)
    page = m.q4_page_shape(shape)
    ws = m.alloc_cache_workspace(shape, DEV)
    k, v = m.alloc_q4_pool(shape, DEV), m.alloc_q4_pool(shape, DEV)
    pools = m.pool_table([k, v])
    a, b = m.CacheMeta.empty(shape, DEV), m.CacheMeta.empty(shape, DEV)
    granted = ints([0, 0, 0])
    rng = np.random.default_rng(6)
    x = rows(rng, (3, 150, 2, 128), "bf16")
    m.moe_cache_reserve(page, a, ints([150, 0, 0]), b, granted, pools, ws)
    m.moe_cache_write_q4(shape, b, granted, x.to(DEV), x.to(DEV), k, v, ws)
    m.moe_cache_fork(page, b, ints([0, 0, 0]), a, ws)
    m.moe_cache_reserve(page, a, ints([3, 5, 0]), b, granted, pools, ws)
    y = rows(rng, (3, 5, 2, 128), "bf16")
    m.moe_cache_write_q4(shape, b, granted, y.to(DEV), y.to(DEV), k, v, ws)
    n_live = ints([0])
    m.moe_cache_compact(page, b, a, n_live, pools, ws)
    out = [torch.zeros((3, 155, 2, 128), device=DEV) for _ in range(2)]
    m.moe_cache_read_q4(shape, a, None, ints([153, 155, 150]), k, v, *out, ws)
    assert m.moe_query_device_status(ws) == 0
    for s, more in enumerate((3, 5, 0)):
        whole = np.concatenate([x[0].double().numpy(), y[s, :more].double().numpy()])
        q, sc, bi = ref.quantise(whole)
        want = q * np.repeat(sc, 32, -1) + np.repeat(bi, 32, -1)
        np.testing.assert_array_equal(out[1][s, :150 + more].cpu().numpy(), want.astype(np.float32))


def test_pages_past_32_bits_of_bytes():
    n_phys = 450000  # 4.6 GB
    shape = m.make_cache_shape(2, 2, n_phys, 2, 128)
    k = m.alloc_q4_pool(shape, DEV)
    v = m.alloc_q4_pool(shape, DEV)
    ws = m.alloc_cache_workspace(shape, DEV)
    meta = m.CacheMeta(ints([[n_phys - 1, 0], [n_phys - 3, n_phys - 2]]), ints([100, 128]),
                       torch.ones(n_phys, dtype=torch.int32, device=DEV))
    rng = np.random.default_rng(7)
    x = rows(rng, (2, 100, 2, 128), "bf16")
    m.moe_cache_write_q4(shape, meta, None, x.to(DEV), (-x).to(DEV), k, v, ws)
    out = [torch.zeros((2, 100, 2, 128), device=DEV) for _ in range(2)]
    m.moe_cache_read_q4(shape, meta, ints([0, 28]), None, k, v, *out, ws)
    assert m.moe_query_device_status(ws) == 0
    for got, y in zip(out, (x, -x)):
        q, s, b = ref.quantise(y.double().numpy())
        np.testing.assert_array_equal(got.cpu().numpy(),
                                      (q * np.repeat(s, 32, -1) + np.repeat(b, 32, -1)).astype(np.float32))


def test_captured_calls_take_new_numbers():
    st = State(8, [90, 64], 2, 128)
    meta = st.meta()
    x = rows(st.rng, (2, 4, 2, 128), "bf16").to(DEV)
    out = [torch.zeros((2, 4, 2, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    n, first = ints([4, 2]), ints([86, 62])
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            m.moe_cache_write_q4(st.shape, meta, n, x, x, st.k, st.v, st.ws)
            m.moe_cache_read_q4(st.shape, meta, first, n, st.k, st.v, *out, st.ws)
    for seed in range(3):
        x.copy_(rows(np.random.default_rng(seed), (2, 4, 2, 128), "bf16"))
        n.copy_(ints([seed + 1, 4 - seed]))
        first.copy_(meta.lens - n)
        out[0].fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        q, s, b = ref.quantise(x.cpu().double().numpy())
        want = torch.from_numpy(q * np.repeat(s, 32, -1) + np.repeat(b, 32, -1))
        for i, c in enumerate((seed + 1, 4 - seed)):
            err = (out[0][i, :c].cpu().double() - want[i, :c]).abs()
            assert (err <= 2.0**-8 * want[i, :c].abs() + 2.0**-25).all()
            assert (out[0][i, c:] == 5).all()


@pytest.mark.parametrize("D,dtype,lens,T", [(128, "bf16", [500, 449, 385, 384, 5], 500),
                                            (64, "fp16", [1000, 769, 768, 130], 1000)])
def test_slots_of_very_different_length(D, dtype, lens, T):
    """A CTA goes on along its slot where there are too few for one a stretch
    (40 slots of 8 heads have six each)."""
    lens = lens + [1] * (40 - len(lens))
    st = State(D, lens, 8, D)
    n = st.lens.copy()
    k, v = rows(st.rng, (40, T, 8, D), dtype), rows(st.rng, (40, T, 8, D), dtype)
    m.moe_cache_write_q4(st.shape, st.meta(), ints(n), k.to(DEV), v.to(DEV), st.k, st.v, st.ws)
    assert m.moe_query_device_status(st.ws) == 0
    for pool, old, x in ((st.k, st.k0, k), (st.v, st.v0, v)):
        np.testing.assert_array_equal(pool.cpu().numpy(), st.written(old, x.double().numpy(), 0 * n, n))
    out = [torch.full((40, T, 8, D), 7.0, device=DEV) for _ in range(2)]
    m.moe_cache_read_q4(st.shape, st.meta(), None, ints(n), st.k, st.v, *out, st.ws)
    assert m.moe_query_device_status(st.ws) == 0
    for x, got in zip((k, v), out):
        for s in range(40):
            want = ref.values(ref.pack(*ref.quantise(x[s, :n[s]].double().numpy())), D)
            np.testing.assert_array_equal(got[s, :n[s]].cpu().numpy(), want.astype(np.float32))
            assert (got[s, n[s]:] == 7.0).all()
