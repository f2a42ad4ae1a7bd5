"""Host checks of the 4-bit cache's calls and of token log probabilities: every
refusal is returned before anything is enqueued (no GPU needed), and the
references that the GPU tests use agree with rows worked by hand."""
import ctypes as C

import numpy as np
import pytest

import bit_moe_expert_histogram_gb300 as m
import q4_ref as ref

P = C.c_void_p(0x10000)
ODD = C.c_void_p(0x10002)   # 2-byte aligned
OFF = C.c_void_p(0x10008)   # 8-byte aligned


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return m.load()


def test_units(lib):
    assert [lib.moe_cache_q4_units(d) for d in (64, 128, 0, 32, 96, 256, -64)] == [24, 40, 0, 0, 0, 0, 0]
    assert m.q4_page_shape(m.make_cache_shape(3, 4, 5, 2, 128)).D == 40
    with pytest.raises(m.MoeError):
        m.moe_cache_q4_units(256)


def test_write_and_read_refusals(lib):
    s = m.CacheShape(8, 16, 100, 2, 128, 64)
    need = lib.moe_cache_workspace_bytes(C.byref(s))
    meta = m.CacheMetaPtrs(0x1000, 0x2000, 0x3000)

    def write(s=s, meta=meta, n=P, T=4, dt=0, k=P, ks=256, v=P, vs=256, kc=P, vc=P, ws=P, have=need):
        return lib.moe_cache_write_q4(C.byref(s) if s else None, C.byref(meta) if meta else None, n, T,
                                      dt, k, ks, v, vs, kc, vc, ws, have, None)

    def read(s=s, meta=meta, first=P, n=P, T=4, kc=P, vc=P, dt=0, k=P, ks=256, v=P, vs=256, ws=P, have=need):
        return lib.moe_cache_read_q4(C.byref(s) if s else None, C.byref(meta) if meta else None, first, n,
                                     T, kc, vc, dt, k, ks, v, vs, ws, have, None)
    for call in (write, read):
        for bad in (dict(s=None), dict(T=0), dict(T=(1 << 18) + 1), dict(dt=3), dict(dt=-1),
                    dict(s=m.CacheShape(8, 16, 100, 2, 96, 64)),
                    dict(s=m.CacheShape(8, 16, 100, 2, 256, 64)),
                    dict(s=m.CacheShape(0, 16, 100, 2, 128, 64)),
                    dict(s=m.CacheShape(8, 16, 100, 65, 128, 64)),
                    dict(s=m.CacheShape(8, 16, 100, 2, 128, 32))):
            assert call(**bad) == m.MOE_ERR_UNSUPPORTED_SHAPE, bad
        for bad in (dict(meta=None), dict(meta=m.CacheMetaPtrs(0, 0x2000, 0x3000)),
                    dict(meta=m.CacheMetaPtrs(0x1000, 0x2002, 0x3000)), dict(n=ODD), dict(k=None),
                    dict(k=OFF), dict(v=None), dict(v=OFF), dict(kc=None), dict(kc=OFF), dict(vc=None),
                    dict(vc=OFF), dict(ks=248), dict(vs=248), dict(ks=257), dict(vs=260), dict(ws=None),
                    dict(ws=C.c_void_p(0x10080))):
            assert call(**bad) == m.MOE_ERR_INVALID_ARG, bad
        assert call(have=need - 1) == m.MOE_ERR_WORKSPACE
    assert write(dt=2) == m.MOE_ERR_UNSUPPORTED_SHAPE  # fp32 rows are not written
    assert read(first=ODD) == m.MOE_ERR_INVALID_ARG
    assert read(dt=2, ks=258) == m.MOE_ERR_INVALID_ARG


def test_attention_refusals(lib):
    ok = dict(n_slots=4, T=2, n_q=16, n_kv=2, D=128, block=64, max_blocks=8, prefix_blocks=0, dtype=0)
    s = m.AttnBatchShape(**ok)
    need = lib.moe_attn_batch_q4_workspace_bytes(C.byref(s))
    assert need > 0 and lib.moe_attn_batch_q4_workspace_bytes(None) == 0

    def call(s=s, q=P, qs=2048, k=P, v=P, n_phys=100, table=P, lens=P, n=None, o=P, ws=P, have=need):
        return lib.moe_attn_batch_q4(C.byref(s) if s else None, q, qs, k, v, n_phys, table, lens, n, o,
                                     ws, have, None)
    assert call(s=None) == m.MOE_ERR_UNSUPPORTED_SHAPE
    for bad in (dict(n_slots=0), dict(n_slots=4097), dict(T=0), dict(T=9), dict(n_q=15), dict(n_kv=0),
                dict(D=96), dict(D=256), dict(block=32), dict(max_blocks=0), dict(prefix_blocks=1),
                dict(dtype=2), dict(n_slots=4096, n_kv=16, max_blocks=1 << 13, T=32)):
        t = m.AttnBatchShape(**{**ok, **bad})
        assert lib.moe_attn_batch_q4_workspace_bytes(C.byref(t)) == 0, bad
        assert call(s=t) == m.MOE_ERR_UNSUPPORTED_SHAPE, bad
    for bad in (dict(q=None), dict(q=OFF), dict(qs=2040), dict(qs=2049), dict(k=None), dict(k=OFF),
                dict(v=None), dict(v=OFF), dict(n_phys=0), dict(table=None), dict(table=ODD),
                dict(lens=None), dict(lens=ODD), dict(n=ODD), dict(o=None), dict(o=OFF), dict(ws=None),
                dict(ws=C.c_void_p(0x10080))):
        assert call(**bad) == m.MOE_ERR_INVALID_ARG, bad
    assert call(have=need - 1) == m.MOE_ERR_WORKSPACE


def test_logprobs_refusals(lib):
    s = m.LogprobsShape(4, 1000, 5, 0)
    need = lib.moe_logprobs_workspace_bytes(C.byref(s))
    assert need > 0 and lib.moe_logprobs_workspace_bytes(None) == 0

    def call(s=s, x=P, stride=1000, tok=P, lp=P, ent=None, ids=None, top=None, ws=P, have=need):
        return lib.moe_token_logprobs(C.byref(s) if s else None, x, stride, tok, lp, ent, ids, top, ws,
                                      have, None)
    assert call(s=None) == m.MOE_ERR_UNSUPPORTED_SHAPE
    for bad in ((0, 1000, 5, 0), ((1 << 20) + 1, 1000, 5, 0), (4, 0, 5, 0), (4, (1 << 20) + 1, 5, 0),
                (4, 1000, -1, 0), (4, 1000, 33, 0), (4, 1000, 5, 3), (4, 1000, 5, -1)):
        t = m.LogprobsShape(*bad)
        assert lib.moe_logprobs_workspace_bytes(C.byref(t)) == 0, bad
        assert call(s=t) == m.MOE_ERR_UNSUPPORTED_SHAPE, bad
    for bad in (dict(x=None), dict(x=C.c_void_p(0x10001)), dict(stride=999), dict(tok=None), dict(tok=ODD),
                dict(lp=None), dict(lp=ODD), dict(ent=ODD), dict(ids=ODD), dict(top=ODD), dict(ws=None),
                dict(ws=C.c_void_p(0x10080))):
        assert call(**bad) == m.MOE_ERR_INVALID_ARG, bad
    assert call(s=m.LogprobsShape(4, 1000, 5, 2), x=ODD) == m.MOE_ERR_INVALID_ARG
    assert call(have=need - 1) == m.MOE_ERR_WORKSPACE


def test_the_binding_wants_cuda_tensors(lib):
    import torch
    s = m.make_logprobs_shape(2, 10)
    with pytest.raises(ValueError):
        m.moe_token_logprobs(s, torch.zeros(2, 10), torch.zeros(2, dtype=torch.int32), torch.zeros(2),
                             torch.zeros(1, dtype=torch.uint8))
    c = m.make_cache_shape(1, 1, 1, 1, 64)
    for dt in (torch.float32, torch.int16):  # of what type int16 bits are would be a guess
        x = torch.zeros((1, 1, 1, 64), dtype=dt)
        with pytest.raises(ValueError):
            m.moe_cache_write_q4(c, None, None, x, x, x, x, x)


def test_a_row_by_hand():
    """0 .. 15 twice: step 1 from 0, every code itself; a half goes up."""
    x = np.tile(np.arange(16.0), 4)
    code, s, b = ref.quantise(x)
    assert np.array_equal(code, x) and np.all(s == 1) and np.all(b == 0)
    x[1], x[17], x[33] = 0.5, 1.5, 1.25
    assert [ref.quantise(x)[0][i] for i in (1, 17, 33)] == [1, 2, 1]
    row = ref.pack(code, s, b).view(np.uint16)
    # D = 64: unit u of a half: elements 2 u, 2 u + 1 of its first group, then of its second
    assert [hex(v) for v in row[:3]] == ["0x1010", "0x3232", "0x5454"]
    assert np.array_equal(row[16:], [0x3F80] * 4 + [0] * 4)
    y = np.arange(128.0) % 32  # 32 elements a group: max 31, step 31 / 15
    code, s, b = ref.quantise(y)
    row = ref.pack(code, s, b).view(np.uint16)
    assert s[0] == 2.0625 and row[0] == sum(int(code[i]) << 4 * i for i in range(4))
    np.testing.assert_array_equal(ref.values(row.view(np.int16), 128), code * s[0])


def test_roundings_of_scale_and_bias():
    """Ties of the scale go to the even number, the bias goes down."""
    for lo, want in ((241 / 256, 1.0), (211 / 256, 1 + 2 / 128)):  # (16 - lo) / 15 = 1 + 1/256, 1 + 3/256
        x = np.full(64, lo)
        x[::16] = 16.0
        _, s, b = ref.quantise(x)
        assert np.all(s == want) and np.all(b == lo)
    x = np.full(64, -1.0 - 2.0**-10)
    code, s, b = ref.quantise(x)
    assert np.all(b == -1.0 - 2.0**-7) and np.all(s > 0) and np.all(code == 15)


def test_the_log_probabilities_reference():
    x = np.log(np.array([[0.5, 0.25, 0.25, 0.0 + 1e-300], [0.1, 0.2, 0.3, 0.4]]))
    x[0, 3] = -np.inf
    lp, ent, ids, top = ref.logprobs(x, [1, -1], 4)
    np.testing.assert_allclose(lp, [np.log(0.25), 0.0])
    np.testing.assert_allclose(ent, [1.5 * np.log(2), -(np.array([.1, .2, .3, .4]) * np.log([.1, .2, .3, .4])).sum()])
    assert ids.tolist() == [[0, 1, 2, -1], [3, 2, 1, 0]] and top[0, 3] == -np.inf


def test_the_attention_reference():
    """Equal keys: the mean of what is visible; a page that is none is left out."""
    rng = np.random.default_rng(0)
    k = np.tile(ref.pack(*ref.quantise(rng.normal(size=64))), (3, 1, 64, 1))
    v = ref.pack(*ref.quantise(rng.normal(size=(3, 1, 64, 64))))
    q = rng.normal(size=(1, 2, 2, 64))
    table = np.array([[2, 9, 0]])
    o, tol = ref.attention(q, k, v, table, [150], [2])
    mean = np.concatenate([ref.values(v[2, 0], 64), ref.values(v[0, 0], 64)[:22]])
    np.testing.assert_allclose(o[0, 1, 0], mean.mean(0))
    np.testing.assert_allclose(o[0, 0, 1], mean[:-1].mean(0))
    assert tol.min() > 0 and not ref.attention(q, k, v, table, [1], [2])[0][0, 0].any()
