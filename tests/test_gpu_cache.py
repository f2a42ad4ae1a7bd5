"""GPU parity of the cache's page operations (moe_cache_fork, _reserve,
_write, _compact, _copy_pages) with the plain references: whole numbers and
copied bits, all equal."""
import numpy as np
import pytest
import torch

import bit_moe_expert_histogram_gb300 as m
import serve_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    m.load()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


class Cache:
    """One state on both sides."""

    def __init__(self, seed, n_slots, max_blocks, n_phys, n_kv=2, D=64, pools=2, **kw):
        self.rng = np.random.default_rng(seed)
        self.host = ref.make_state(self.rng, n_slots, max_blocks, n_phys, **kw)
        self.shape = m.make_cache_shape(n_slots, max_blocks, n_phys, n_kv, D)
        self.ws = m.alloc_cache_workspace(self.shape, DEV)
        self.pools = self.rng.integers(-30000, 30000, (pools, n_phys, n_kv, 64, D)).astype(np.int16)
        self.upload()

    def upload(self):
        self.meta = m.CacheMeta(*[dev(a) for a in self.host])
        self.out = m.CacheMeta.empty(self.shape, DEV)
        for t in (self.out.table, self.out.lens, self.out.refs):
            t.fill_(-7)  # every entry has to be written
        self.dpools = dev(self.pools)
        self.table = m.pool_table(list(self.dpools))

    def check(self, want, status=0):
        assert m.moe_query_device_status(self.ws) == status
        for name, a in zip(("table", "lens", "refs"), want):
            np.testing.assert_array_equal(getattr(self.out, name).cpu().numpy(), a, err_msg=name)
        np.testing.assert_array_equal(self.dpools.cpu().numpy(), self.pools)
        # the old state is as it was
        for t, a in zip((self.meta.table, self.meta.lens, self.meta.refs), self.host):
            np.testing.assert_array_equal(t.cpu().numpy(), a)


@pytest.mark.parametrize("n_slots,max_blocks,n_phys", [(1, 1, 1), (3, 5, 20), (40, 17, 300),
                                                       (257, 130, 5000), (4096, 3, 2049)])
def test_fork(n_slots, max_blocks, n_phys):
    c = Cache(n_slots, n_slots, max_blocks, n_phys, pools=1, D=8)
    for keep in (None, c.rng.integers(-2, max_blocks * 64 + 5, n_slots).astype(np.int32)):
        parent = c.rng.integers(-1, n_slots, n_slots).astype(np.int32)
        parent[::3] = np.arange(n_slots)[::3]
        m.moe_cache_fork(c.shape, c.meta, dev(parent), c.out, c.ws,
                         keep=None if keep is None else dev(keep))
        c.check(ref.fork(*c.host, parent, keep))


def test_fork_bad_parent_length_and_entry():
    c = Cache(5, 6, 8, 60, pools=1, D=8, share=0.0)
    table, lens, refs = c.host
    lens[:] = 200
    table[:, :4] = np.arange(24).reshape(6, 4)
    table[:, 4:] = -1
    refs[:] = np.bincount(table[table >= 0], minlength=60)
    c.upload()
    parent = np.array([0, 1, 2, 3, 4, 6], np.int32)  # slot 6 does not exist
    m.moe_cache_fork(c.shape, c.meta, dev(parent), c.out, c.ws)
    c.check(ref.fork(table, lens, refs, parent, None), m.MOE_ERR_BAD_INPUT)
    # an entry outside the pool is left out, on both sides of a move
    table[1, 2] = 60
    c.upload()
    parent = np.array([1, 0, 2, 3, 4, 5], np.int32)
    m.moe_cache_fork(c.shape, c.meta, dev(parent), c.out, c.ws)
    t = table.copy()
    t[[0, 1]] = table[[1, 0]]
    t[0, 2] = -1
    rf = refs.copy()
    rf[2] = 2       # slot 0's third page is now slot 1's too: its entry in row 0 went
    want_refs = np.bincount(t[t >= 0], minlength=60).astype(np.int32)
    want_refs[6] = 1  # slot 1 held page 6 where the bad entry is: the count was never given back
    c.check((t, lens, want_refs), m.MOE_ERR_BAD_INPUT)
    # a length past the row counts as the row's whole width
    table[1, 2] = 6
    lens[3] = 8 * 64 + 1
    table[3] = np.arange(40, 48)
    refs[:] = np.bincount(table[table >= 0], minlength=60)
    c.upload()
    parent = np.arange(6, dtype=np.int32)
    m.moe_cache_fork(c.shape, c.meta, dev(parent), c.out, c.ws)
    n = lens.copy()
    n[3] = 512
    c.check((table, n, refs), m.MOE_ERR_BAD_INPUT)


@pytest.mark.parametrize("n_slots,max_blocks,n_phys,most,fill", [
    (1, 2, 4, 70, 0.3), (5, 9, 40, 130, 0.5), (64, 12, 700, 5, 0.5), (300, 20, 4100, 200, 0.7),
    (1500, 4, 9000, 65, 0.3), (33, 10, 120, 300, 0.6)])
def test_reserve(n_slots, max_blocks, n_phys, most, fill):
    c = Cache(n_phys, n_slots, max_blocks, n_phys, D=16, fill=fill)
    n_new = c.rng.integers(0, most + 1, n_slots).astype(np.int32)
    n_new[::4] = 0
    granted = torch.full((n_slots,), -7, dtype=torch.int32, device=DEV)
    m.moe_cache_reserve(c.shape, c.meta, dev(n_new), c.out, granted, c.table, c.ws)
    *want, g = ref.reserve(*c.host, n_new, c.pools)
    c.check(want)
    np.testing.assert_array_equal(granted.cpu().numpy(), g)


def test_reserve_of_forks_copies_the_shared_page():
    """Every slot just forked from slot 0: all of them copy its partly filled
    page, in every pool; it is free afterwards."""
    n, width = 9, 4
    c = Cache(3, n, width, 50, n_kv=3, D=128, pools=5, share=0.0)
    table, lens, refs = c.host
    table[:], lens[:] = -1, 100
    table[:, :2] = (17, 30)
    refs[:] = 0
    refs[[17, 30]] = n
    c.upload()
    n_new = np.array([1, 28, 29, 64, 92, 93, 1, 0, 157], np.int32)  # 157: past the row
    granted = torch.empty(n, dtype=torch.int32, device=DEV)
    m.moe_cache_reserve(c.shape, c.meta, dev(n_new), c.out, granted, c.table, c.ws)
    *want, g = ref.reserve(*c.host, n_new, c.pools)
    assert g.tolist() == [1, 28, 29, 64, 92, 93, 1, 0, 0]
    c.check(want)


def test_reserve_bad_length_entry_and_request():
    c = Cache(8, 4, 3, 30, share=0.0)
    table, lens, refs = c.host
    table[:] = -1
    lens[:] = [10, 10, -5, 10]
    table[[0, 1, 3], 0] = [4, 31, 9]  # slot 1's page does not exist
    refs[:] = 0
    refs[[4, 9]] = 1
    c.upload()
    n_new = np.array([60, 60, 3, -1], np.int32)
    granted = torch.empty(4, dtype=torch.int32, device=DEV)
    m.moe_cache_reserve(c.shape, c.meta, dev(n_new), c.out, granted, c.table, c.ws)
    t, n, rf = table.copy(), np.array([70, 10, 3, 10], np.int32), refs.copy()
    t[0, 1], t[2, 0] = 0, 1
    rf[[0, 1]] = 1
    c.check((t, n, rf), m.MOE_ERR_BAD_INPUT)
    assert granted.tolist() == [60, 0, 3, 0]


@pytest.mark.parametrize("n_slots,T,n_kv,D", [(1, 1, 1, 64), (7, 5, 2, 128), (50, 1, 4, 64),
                                              (3, 200, 2, 8), (2, 3, 3, 200)])
@pytest.mark.parametrize("joint", [False, True])
def test_write(n_slots, T, n_kv, D, joint):
    c = Cache(T + D, n_slots, 6, n_slots * 6 + 3, n_kv=n_kv, D=D, fill=1.0, share=0.0)
    table, lens, refs = c.host
    n_new = np.minimum(c.rng.integers(0, T + 1, n_slots), lens).astype(np.int32)
    new = c.rng.integers(-30000, 30000, (n_slots, T, 2 if joint else 1, n_kv, D)).astype(np.int16)
    v = c.rng.integers(-30000, 30000, (n_slots, T, n_kv, D)).astype(np.int16)
    dn, dv = dev(new), dev(v)
    k_new, v_new = (dn[:, :, 0], dn[:, :, 1]) if joint else (dn[:, :, 0], dv)
    m.moe_cache_write(c.shape, c.meta, dev(n_new), k_new, v_new, c.dpools[0], c.dpools[1], c.ws)
    ref.write(table, lens, n_new, new[:, :, 0], c.pools[0])
    ref.write(table, lens, n_new, new[:, :, 1] if joint else v, c.pools[1])
    assert m.moe_query_device_status(c.ws) == 0
    np.testing.assert_array_equal(c.dpools.cpu().numpy(), c.pools)


def test_write_bad_values_write_nothing():
    c = Cache(4, 5, 2, 20, share=0.0)
    table, lens, refs = c.host
    table[:] = np.arange(10).reshape(5, 2)
    lens[:] = [3, 129, 70, -1, 1]
    table[2, 1] = 20
    c.upload()
    new = dev(np.ones((5, 2, 2, 64), np.int16))
    n_new = np.array([3, 2, 2, 1, 2], np.int32)  # more than T; too long; no such page; < 0; < n_new
    m.moe_cache_write(c.shape, c.meta, dev(n_new), new, new, c.dpools[0], c.dpools[1], c.ws)
    assert m.moe_query_device_status(c.ws) == m.MOE_ERR_BAD_INPUT
    np.testing.assert_array_equal(c.dpools.cpu().numpy(), c.pools)


@pytest.mark.parametrize("n_slots,max_blocks,n_phys,fill", [
    (1, 1, 1, 1.0), (2, 3, 7, 0.5), (30, 10, 1024, 0.2), (60, 30, 1025, 0.9), (50, 50, 2048, 0.5),
    (80, 40, 3001, 0.6), (16, 64, 1024, 1.0)])
def test_compact(n_slots, max_blocks, n_phys, fill):
    c = Cache(n_phys, n_slots, max_blocks, n_phys, n_kv=1, D=16, pools=3, fill=fill, share=0.2)
    n_live = torch.empty(1, dtype=torch.int32, device=DEV)
    m.moe_cache_compact(c.shape, c.meta, c.out, n_live, c.table, c.ws)
    *want, L = ref.compact(*c.host, c.pools)
    c.check(want)
    assert n_live.item() == L


@pytest.mark.parametrize("live", [0, 1, 1024, 2048])
def test_compact_edges(live):
    """Nothing held; one page at the end; a pool whose held pages end on a
    border of the ranks' chunks; a full pool."""
    c = Cache(live, 1, 2048, 2048, n_kv=1, D=8, pools=1, share=0.0)
    table, lens, refs = c.host
    table[:], lens[:], refs[:] = -1, 0, 0
    pages = np.arange(2048 - live, 2048)
    table[0, :live], lens[0] = pages, live * 64
    refs[pages] = 1
    c.upload()
    n_live = torch.empty(1, dtype=torch.int32, device=DEV)
    m.moe_cache_compact(c.shape, c.meta, c.out, n_live, c.table, c.ws)
    *want, L = ref.compact(*c.host, c.pools)
    c.check(want)
    assert n_live.item() == L == live


def test_compact_entry_of_a_free_page():
    c = Cache(2, 2, 2, 8, n_kv=1, D=8, pools=1, share=0.0)
    table, lens, refs = c.host
    table[:] = [[7, 6], [5, -1]]  # page 5 is not counted, page 6 is
    lens[:] = [128, 64]
    refs[:] = 0
    refs[[6, 7]] = 1
    c.upload()
    n_live = torch.empty(1, dtype=torch.int32, device=DEV)
    m.moe_cache_compact(c.shape, c.meta, c.out, n_live, c.table, c.ws)
    c.pools[:, [0, 1]] = c.pools[:, [6, 7]]
    rf = np.zeros_like(refs)
    rf[:2] = 1
    c.check((np.array([[1, 0], [-1, -1]], np.int32), lens, rf), m.MOE_ERR_BAD_INPUT)


def test_copy_pages_out_and_in():
    c = Cache(6, 2, 2, 40, n_kv=3, D=24, pools=4)
    other = c.rng.integers(-9, 9, (4, 17, 3, 64, 24)).astype(np.int16)
    do = dev(other)
    src, dst = np.array([39, 0, 7, 8], np.int32), np.array([16, 3, 0, 1], np.int32)
    m.moe_cache_copy_pages(c.shape, dev(src), dev(dst), c.table, m.pool_table(list(do)), c.ws)
    other[:, dst] = c.pools[:, src]
    np.testing.assert_array_equal(do.cpu().numpy(), other)
    assert m.moe_query_device_status(c.ws) == 0
    # pairs out of range on either side are left out
    src, dst = np.array([40, 5, -1, 2], np.int32), np.array([1, 17, 2, 5], np.int32)
    m.moe_cache_copy_pages(c.shape, dev(src), dev(dst), c.table, m.pool_table(list(do)), c.ws)
    other[:, 5] = c.pools[:, 2]
    np.testing.assert_array_equal(do.cpu().numpy(), other)
    assert m.moe_query_device_status(c.ws) == m.MOE_ERR_BAD_INPUT


def test_pages_past_32_bits_of_elements():
    """Pools of 150000 pages of 2 heads of 128: 2.5e9 elements. Copy-on-write
    and write at their end, then everything brought to the front."""
    n_phys, n_kv, D = 150000, 2, 128
    shape = m.make_cache_shape(3, 2, n_phys, n_kv, D)
    ws = m.alloc_cache_workspace(shape, DEV)
    pools = [torch.zeros((n_phys, n_kv, 64, D), dtype=torch.int16, device=DEV) for _ in range(2)]
    table = np.full((3, 2), -1, np.int32)
    table[:, 0] = (n_phys - 1, n_phys - 1, n_phys - 7)
    lens = np.array([10, 10, 64], np.int32)
    refs = np.ones(n_phys, np.int32)  # all pinned but a few at the end
    refs[n_phys - 1], refs[[n_phys - 3, n_phys - 2, n_phys - 9]] = 2, 0
    g = torch.Generator(device=DEV).manual_seed(0)
    for p in pools:
        p[n_phys - 10:] = torch.randint(-99, 99, (10, n_kv, 64, D), generator=g, device=DEV,
                                        dtype=torch.int16)
    before = [p[n_phys - 10:].clone() for p in pools]
    meta = m.CacheMeta(dev(table), dev(lens), dev(refs))
    out, granted = m.CacheMeta.empty(shape, DEV), torch.empty(3, dtype=torch.int32, device=DEV)
    ptable = m.pool_table(pools)
    m.moe_cache_reserve(shape, meta, dev(np.array([2, 2, 2], np.int32)), out, granted, ptable, ws)
    new = torch.randint(100, 200, (3, 2, n_kv, D), generator=g, device=DEV, dtype=torch.int16)
    m.moe_cache_write(shape, out, granted, new, new, pools[0], pools[1], ws)
    assert m.moe_query_device_status(ws) == 0 and granted.tolist() == [2, 2, 2]
    assert out.table.tolist() == [[n_phys - 9, -1], [n_phys - 3, -1], [n_phys - 7, n_phys - 2]]
    for p, b in zip(pools, before):
        for s, page in ((0, 1), (1, 7)):
            torch.testing.assert_close(p[n_phys - 10 + page, :, :10], b[9, :, :10], rtol=0, atol=0)
            torch.testing.assert_close(p[n_phys - 10 + page, :, 10:12], new[s].transpose(0, 1),
                                       rtol=0, atol=0)
        torch.testing.assert_close(p[n_phys - 2, :, :2], new[2].transpose(0, 1), rtol=0, atol=0)
    # free everything but the slots' pages, and compact
    out.refs.zero_()
    out.refs[out.table[out.table >= 0].long()] = 1
    want = [p[out.table[2, 1].long()].clone() for p in pools]
    n_live = torch.empty(1, dtype=torch.int32, device=DEV)
    m.moe_cache_compact(shape, out, meta, n_live, ptable, ws)
    assert m.moe_query_device_status(ws) == 0 and n_live.item() == 4
    assert meta.table.tolist() == [[0, -1], [2, -1], [1, 3]]
    for p, w in zip(pools, want):
        torch.testing.assert_close(p[3], w, rtol=0, atol=0)


def test_step_in_a_graph_on_a_side_stream():
    """Reserve and write captured once and replayed over a state that moves
    on: the graph's calls read what the buffers hold at the time."""
    c = Cache(11, 12, 8, 120, D=64, share=0.0, fill=0.3)
    n_new = np.full(12, 3, np.int32)
    granted = torch.empty(12, dtype=torch.int32, device=DEV)
    dn = dev(n_new)
    new = dev(c.rng.integers(-99, 99, (12, 3, 2, 64)).astype(np.int16))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        m.moe_cache_reserve(c.shape, c.meta, dn, c.out, granted, c.table, c.ws)
        m.moe_cache_write(c.shape, c.out, granted, new, new, c.dpools[0], c.dpools[1], c.ws)
        for a, b in ((c.meta.table, c.out.table), (c.meta.lens, c.out.lens),
                     (c.meta.refs, c.out.refs)):
            a.copy_(b)
    for _ in range(30):
        g.replay()
        t, n, r, gr = ref.reserve(*c.host, n_new, c.pools)
        ref.write(t, n, gr, new.cpu().numpy(), c.pools[0])
        ref.write(t, n, gr, new.cpu().numpy(), c.pools[1])
        c.host = (t, n, r)
    torch.cuda.synchronize()
    c.check(c.host)


def test_binding_refuses_wrong_tensors():
    c = Cache(1, 3, 2, 9)
    with pytest.raises(ValueError):
        m.moe_cache_fork(c.shape, c.meta, torch.zeros(2, dtype=torch.int32, device=DEV), c.out, c.ws)
    with pytest.raises(ValueError):
        m.moe_cache_fork(c.shape, c.meta, torch.zeros(3, dtype=torch.int64, device=DEV), c.out, c.ws)
    k = torch.zeros((3, 2, 2, 64), dtype=torch.int16, device=DEV)
    with pytest.raises(ValueError):  # the heads of a token lie apart
        m.moe_cache_write(c.shape, c.meta, None, k.transpose(1, 2).contiguous().transpose(1, 2), k,
                          c.dpools[0], c.dpools[1], c.ws)
    with pytest.raises(ValueError):  # pools of another page count
        m.moe_cache_write(c.shape, c.meta, None, k, k, c.dpools[0][:4], c.dpools[1][:4], c.ws)
    with pytest.raises(m.MoeError):
        m.moe_cache_fork(c.shape, c.meta, torch.zeros(3, dtype=torch.int32, device=DEV), c.meta,
                         c.ws)
