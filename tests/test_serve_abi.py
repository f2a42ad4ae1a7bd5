"""Host checks of the batch serving calls: every refusal is returned before
anything is enqueued (no GPU needed), and the references that the GPU tests
use agree with hand-worked states."""
import ctypes as C

import numpy as np
import pytest

import bit_moe_expert_histogram_gb300 as m
import serve_ref as ref

P = C.c_void_p(0x10000)
ODD = C.c_void_p(0x10002)


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return m.load()


def meta(a=0x1000, b=0x2000, c=0x3000):
    return m.CacheMetaPtrs(a, b, c)


def test_cache_shapes(lib):
    ok = dict(n_slots=8, max_blocks=16, n_phys=100, n_kv=2, D=128, block=64)
    assert lib.moe_cache_workspace_bytes(C.byref(m.CacheShape(**ok))) > 0
    for bad in (dict(n_slots=0), dict(n_slots=4097), dict(max_blocks=0), dict(max_blocks=2**18 + 1),
                dict(n_phys=0), dict(n_phys=2**20 + 1), dict(n_kv=0), dict(n_kv=65), dict(D=4),
                dict(D=100), dict(D=520), dict(block=32)):
        s = m.CacheShape(**{**ok, **bad})
        assert lib.moe_cache_workspace_bytes(C.byref(s)) == 0, bad
        i, o = meta(), meta(0x4000, 0x5000, 0x6000)
        assert lib.moe_cache_fork(C.byref(s), C.byref(i), P, None, C.byref(o), P, 1 << 30,
                                  None) == m.MOE_ERR_UNSUPPORTED_SHAPE
    assert lib.moe_cache_workspace_bytes(None) == 0


def test_cache_argument_errors(lib):
    s = m.CacheShape(8, 16, 100, 2, 128, 64)
    need = lib.moe_cache_workspace_bytes(C.byref(s))
    i, o = meta(), meta(0x4000, 0x5000, 0x6000)
    pools = (C.c_void_p * 2)(0x10000, 0x20000)
    pp = C.cast(pools, C.c_void_p)

    def fork(i=i, o=o, parent=P, keep=None, ws=P, n=need):
        return lib.moe_cache_fork(C.byref(s), C.byref(i), parent, keep, C.byref(o), ws, n, None)
    assert fork(parent=None) == m.MOE_ERR_INVALID_ARG
    assert fork(keep=ODD) == m.MOE_ERR_INVALID_ARG
    assert fork(ws=None) == m.MOE_ERR_INVALID_ARG
    assert fork(ws=C.c_void_p(0x10080)) == m.MOE_ERR_INVALID_ARG  # not 256-byte aligned
    assert fork(n=need - 1) == m.MOE_ERR_WORKSPACE
    assert fork(i=meta(0)) == m.MOE_ERR_INVALID_ARG
    for shared in (meta(0x1000, 0x5000, 0x6000), meta(0x4000, 0x2000, 0x6000),
                   meta(0x4000, 0x5000, 0x3000)):  # the states may not share an array
        assert fork(o=shared) == m.MOE_ERR_INVALID_ARG

    def reserve(n_new=P, granted=P, pools=pp, k=2, ws=P, n=need):
        return lib.moe_cache_reserve(C.byref(s), C.byref(i), n_new, C.byref(o), granted, pools, k,
                                     ws, n, None)
    assert reserve(n_new=None) == m.MOE_ERR_INVALID_ARG
    assert reserve(granted=None) == m.MOE_ERR_INVALID_ARG
    assert reserve(pools=None) == m.MOE_ERR_INVALID_ARG
    assert reserve(k=129) == m.MOE_ERR_INVALID_ARG
    assert reserve(k=-1) == m.MOE_ERR_INVALID_ARG
    assert reserve(pools=C.cast((C.c_void_p * 2)(0x10000, 0x20008), C.c_void_p)) == \
        m.MOE_ERR_INVALID_ARG
    assert reserve(n=0) == m.MOE_ERR_WORKSPACE

    def write(T=3, k=P, ks=256, v=P, vs=256, kc=P, vc=P, n=need):
        return lib.moe_cache_write(C.byref(s), C.byref(i), None, T, k, ks, v, vs, kc, vc, P, n,
                                   None)
    assert write(T=0) == m.MOE_ERR_UNSUPPORTED_SHAPE
    assert write(k=None) == m.MOE_ERR_INVALID_ARG
    assert write(v=ODD) == m.MOE_ERR_INVALID_ARG
    assert write(ks=255) == m.MOE_ERR_INVALID_ARG  # tokens overlap
    assert write(vs=260) == m.MOE_ERR_INVALID_ARG  # tokens not 16-byte aligned
    assert write(kc=None) == m.MOE_ERR_INVALID_ARG
    assert write(n=16) == m.MOE_ERR_WORKSPACE

    assert lib.moe_cache_compact(C.byref(s), C.byref(i), C.byref(o), None, pp, 2, P, need,
                                 None) == m.MOE_ERR_INVALID_ARG
    assert lib.moe_cache_compact(C.byref(s), C.byref(i), C.byref(i), P, pp, 2, P, need,
                                 None) == m.MOE_ERR_INVALID_ARG

    def copy(n=4, src=P, dst=P, a=pp, b=pp, k=2, n_to=100, have=need):
        return lib.moe_cache_copy_pages(C.byref(s), n, src, dst, a, b, k, n_to, P, have, None)
    for bad in (dict(n=0), dict(src=None), dict(dst=None), dict(a=None), dict(b=None), dict(k=0),
                dict(n_to=0)):
        assert copy(**bad) == m.MOE_ERR_INVALID_ARG, bad
    assert copy(have=1) == m.MOE_ERR_WORKSPACE


def test_verify_argument_errors(lib):
    ok = m.make_verify_shape(4, 3, 1000, "fp32")
    need = lib.moe_verify_workspace_bytes(C.byref(ok))
    assert need > 0
    for bad in ((0, 3, 1000, 2), (4097, 3, 1000, 2), (4, 0, 1000, 2), (4, 32, 1000, 2),
                (4, 3, 0, 2), (4, 3, 2**20 + 1, 2), (4, 3, 1000, 3), (4, 3, 1000, -1)):
        s = m.VerifyShape(*bad)
        assert lib.moe_verify_workspace_bytes(C.byref(s)) == 0
        assert lib.moe_verify_drafts(C.byref(s), P, P, P, P, P, P, P, P, 1 << 30,
                                     None) == m.MOE_ERR_UNSUPPORTED_SHAPE

    def call(p=P, q=P, draft=P, n=P, u=P, tok=P, acc=P, ws=P, have=need):
        return lib.moe_verify_drafts(C.byref(ok), p, q, draft, n, u, tok, acc, ws, have, None)
    for bad in (dict(p=None), dict(p=ODD), dict(q=ODD), dict(draft=None), dict(n=ODD), dict(u=None),
                dict(tok=None), dict(acc=None), dict(ws=None), dict(ws=C.c_void_p(0x10010))):
        assert call(**bad) == m.MOE_ERR_INVALID_ARG, bad
    assert call(have=need - 1) == m.MOE_ERR_WORKSPACE


def test_attention_argument_errors(lib):
    ok = dict(n_slots=4, T=2, n_q=16, n_kv=2, D=128, block=64, max_blocks=10, prefix_blocks=3,
              dtype=0)
    shape = m.AttnBatchShape(**ok)
    need = lib.moe_attn_batch_workspace_bytes(C.byref(shape))
    assert need > 0

    def call(s=shape, q=P, qs=2048, k=P, v=P, n=100, tab=P, pre=P, ln=P, nn=None, o=P, ws=P,
             have=need):
        return lib.moe_attn_batch(C.byref(s), q, qs, k, v, n, tab, pre, ln, nn, o, ws, have, None)
    for bad in (dict(n_slots=0), dict(n_slots=4097), dict(T=0), dict(T=9), dict(n_q=15),
                dict(n_kv=0), dict(D=96), dict(D=256), dict(block=32), dict(max_blocks=0),
                dict(max_blocks=2**18 + 1), dict(prefix_blocks=-1), dict(prefix_blocks=11),
                dict(dtype=2), dict(n_slots=4096, max_blocks=2**18)):
        s = m.AttnBatchShape(**{**ok, **bad})
        assert lib.moe_attn_batch_workspace_bytes(C.byref(s)) == 0, bad
        assert call(s=s) == m.MOE_ERR_UNSUPPORTED_SHAPE, bad
    eight = C.c_void_p(0x10008)
    for bad in (dict(q=None), dict(q=eight), dict(qs=2047), dict(qs=2052), dict(k=None),
                dict(v=eight), dict(n=0), dict(n=2**24), dict(tab=None), dict(pre=None),
                dict(ln=None), dict(nn=ODD), dict(o=None), dict(o=eight), dict(ws=None),
                dict(ws=C.c_void_p(0x10040))):
        assert call(**bad) == m.MOE_ERR_INVALID_ARG, bad
    assert call(have=need - 1) == m.MOE_ERR_WORKSPACE


# ---- the references on states worked by hand
def test_reference_fork():
    table = np.array([[3, 1, -1], [2, -1, -1]], np.int32)
    lens = np.array([70, 64], np.int32)
    refs = np.array([0, 1, 1, 1], np.int32)
    t, n, r = ref.fork(table, lens, refs, [0, 0], [1 << 30, 64])
    assert t.tolist() == [[3, 1, -1], [3, -1, -1]] and n.tolist() == [70, 64]
    assert r.tolist() == [0, 1, 0, 2]
    t, n, r = ref.fork(table, lens, refs, [-1, 0], None)
    assert t.tolist() == [[-1, -1, -1], [3, 1, -1]] and n.tolist() == [0, 70]
    assert r.tolist() == [0, 1, 0, 1]


def test_reference_reserve_copies_and_refuses():
    # two slots share page 2, filled to 10; pages 0, 1 and 3 are free
    table = np.array([[2, -1], [2, -1]], np.int32)
    pools = np.arange(4, dtype=np.int16).reshape(1, 4, 1, 1, 1) * np.ones((1, 4, 1, 64, 8), np.int16)
    t, n, r, g = ref.reserve(table, np.array([10, 10], np.int32), np.array([0, 0, 2, 0], np.int32),
                             [60, 60], pools)
    # slot 0: the copy in 0, a new block in 1; slot 1 would need two of one page
    assert t.tolist() == [[0, 1], [2, -1]] and n.tolist() == [70, 10] and g.tolist() == [60, 0]
    assert r.tolist() == [1, 1, 1, 0]
    assert pools[0, 0, 0, :10].tolist() == pools[0, 2, 0, :10].tolist()
    assert pools[0, 0, 0, 10:].max() == 0


def test_reference_compact():
    table = np.array([[4, 1], [4, -1]], np.int32)
    pools = np.arange(5, dtype=np.int16).reshape(1, 5, 1, 1, 1) * np.ones((1, 5, 1, 64, 8), np.int16)
    t, n, r, L = ref.compact(table, np.array([128, 64], np.int32),
                             np.array([0, 1, 0, 0, 2], np.int32), pools)
    assert L == 2 and t.tolist() == [[0, 1], [0, -1]] and r.tolist() == [2, 1, 0, 0, 0]
    assert pools[0, 0, 0, 0, 0] == 4


def test_reference_verify():
    p = np.array([[[0.5, 0.5, 0.0], [0.25, 0.25, 0.5]]])
    q = np.array([[[0.25, 0.75, 0.0]]])
    # accepted: u q = 0.9 * 0.25 < 0.5; then the second row, 0.6 past 0.5
    t, a = ref.verify(p, q, np.array([[0]]), [1], np.array([[0.9, 0.6]]))
    assert t.tolist() == [[0, 2]] and a.tolist() == [1]
    # rejected: 0.9 * 0.75 >= 0.5; only token 0 has more than the draft gave
    t, a = ref.verify(p, q, np.array([[1]]), [1], np.array([[0.9, 0.6]]))
    assert t.tolist() == [[0, -1]] and a.tolist() == [0]
    # a certain draft that is rejected leaves its own token out
    t, a = ref.verify(p, None, np.array([[1]]), [1], np.array([[0.9, 0.99]]))
    assert t.tolist() == [[0, -1]]


def test_reference_verify_keeps_the_targets_distribution():
    """q(x) min(1, p(x) / q(x)) + P(rejected) w(x) / sum w = p(x): the
    acceptance's border is p / q, and the new token's borders are the running
    sums of w = max(p - q, 0)."""
    p, q = np.array([1, 2, 3, 10]) / 16, np.array([4, 6, 2, 4]) / 16  # exact in binary
    w = np.maximum(p - q, 0)
    assert np.array_equal(np.minimum(p, q) + (1 - np.minimum(p, q).sum()) * w / w.sum(), p)

    def one(x, u0, u1):
        t, a = ref.verify(np.array([[p, p]]), np.array([[q]]), np.array([[x]]), [1],
                          np.array([[u0, u1]]))
        return t[0].tolist(), int(a[0])
    below = lambda x: np.nextafter(x, 0.0)  # noqa: E731
    assert one(0, below(0.25), 0.0) == ([0, 0], 1) and one(0, 0.25, 0.0) == ([2, -1], 0)
    assert one(3, below(1.0), 0.999) == ([3, 3], 1)
    assert one(1, 0.9, below(1 / 7)) == ([2, -1], 0)  # w = (0, 0, 1, 6) / 16
    assert one(1, 0.9, 1 / 7 + 1e-15) == ([3, -1], 0)
