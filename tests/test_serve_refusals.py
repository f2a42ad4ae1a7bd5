"""Host checks of the batch serving calls, beside test_serve_abi: refusals are
returned before anything is enqueued (no GPU needed)."""
import ctypes as C

import pytest

import bit_moe_expert_histogram_gb300 as m

P = C.c_void_p(0x10000)
ODD = C.c_void_p(0x10002)


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return m.load()


def test_compaction_with_a_map(lib):
    s = m.CacheShape(8, 16, 100, 2, 128, 64)
    need = lib.moe_cache_workspace_bytes(C.byref(s))
    i, o = m.CacheMetaPtrs(0x1000, 0x2000, 0x3000), m.CacheMetaPtrs(0x4000, 0x5000, 0x6000)
    pools = C.cast((C.c_void_p * 2)(0x10000, 0x20000), C.c_void_p)

    def call(s=s, o=o, live=P, moved=P, pools=pools, k=2, have=need):
        return lib.moe_cache_compact_map(C.byref(s), C.byref(i), C.byref(o), live, moved, pools, k,
                                         P, have, None)
    assert call(moved=ODD) == m.MOE_ERR_INVALID_ARG
    assert call(live=None) == m.MOE_ERR_INVALID_ARG
    assert call(o=i) == m.MOE_ERR_INVALID_ARG
    assert call(pools=None) == m.MOE_ERR_INVALID_ARG
    assert call(k=129) == m.MOE_ERR_INVALID_ARG
    assert call(have=need - 1) == m.MOE_ERR_WORKSPACE
    assert call(s=m.CacheShape(8, 16, 0, 2, 128, 64)) == m.MOE_ERR_UNSUPPORTED_SHAPE


def test_a_states_tensors_cannot_be_exchanged():
    """The addresses were taken when the state was made: another tensor put in
    a tensor's place would not be read, and the old one's memory would be."""
    state = m.CacheMeta.__new__(m.CacheMeta)
    for name in ("table", "lens", "refs"):
        with pytest.raises(AttributeError):
            setattr(state, name, None)
