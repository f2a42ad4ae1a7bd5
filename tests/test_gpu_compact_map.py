"""Where moe_cache_compact's pages went: pages held by nobody's table, and the
pages of a shared prompt that a caller keeps a list of."""
import numpy as np
import pytest
import torch

import bit_moe_expert_histogram_gb300 as m
import serve_ref as ref
from test_gpu_cache import DEV, Cache, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    m.load()


@pytest.mark.parametrize("n_slots,max_blocks,n_phys", [(1, 1, 1), (9, 7, 100), (30, 10, 1024),
                                                       (80, 40, 3001)])
def test_map(n_slots, max_blocks, n_phys):
    """Held pages go where the rule sends them, some of them pinned only;
    free ones go nowhere."""
    c = Cache(n_phys, n_slots, max_blocks, n_phys, n_kv=1, D=8, pools=1, share=0.2, fill=0.5)
    table, lens, refs = c.host
    pinned = np.nonzero(refs == 0)[0][::3]
    refs[pinned] = 1 + pinned % 3
    c.upload()
    n_live = torch.empty(1, dtype=torch.int32, device=DEV)
    moved = torch.full((n_phys,), -7, dtype=torch.int32, device=DEV)
    before = c.pools.copy()
    m.moe_cache_compact(c.shape, c.meta, c.out, n_live, c.table, c.ws, moved=moved)
    *want, L = ref.compact(*c.host, c.pools)
    c.check(want)
    to, held = moved.cpu().numpy(), np.nonzero(refs)[0]
    assert (to[refs == 0] == -1).all() and sorted(to[held]) == list(range(L))
    np.testing.assert_array_equal(to[held[held < L]], held[held < L])
    np.testing.assert_array_equal(c.dpools.cpu().numpy()[:, to[held]], before[:, held])
    np.testing.assert_array_equal(want[2][to[held]], refs[held])


def test_attention_goes_on_under_a_prompt_that_moved():
    """The prompt's pages are the pool's last ones, pinned by the caller and in
    no table; after the compaction the call with the mapped list gives the bits
    it gave before, and the old list would name free pages."""
    B, n_q, n_kv, D, prefix, own, n_phys = 6, 16, 2, 128, 5, 2, 60
    rng, g = np.random.default_rng(0), torch.Generator(device=DEV).manual_seed(0)
    pool = lambda: torch.randn((n_phys, n_kv, 64, D), generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    k, v = pool(), pool()
    q = torch.randn((B, 1, n_q, D), generator=g, device=DEV).to(torch.bfloat16)
    pages = rng.permutation(n_phys - prefix - 1).astype(np.int32)
    table = np.full((B, prefix + own), -1, np.int32)
    # the slots' states know their own pages only, as blocks past the prompt
    table[:, prefix:] = pages[:B * own].reshape(B, own)
    kept = np.arange(n_phys - prefix, n_phys, dtype=np.int32)[::-1].copy()
    refs = np.zeros(n_phys, np.int32)
    refs[pages[:B * own]], refs[kept] = 1, 1
    lens = (64 * prefix + rng.integers(1, 64 * own + 1, B)).astype(np.int32)
    shape = m.make_attn_batch_shape(B, 1, n_q, n_kv, D, prefix + own, prefix)
    ws = m.alloc_attn_batch_workspace(shape, DEV)
    outs = [torch.empty_like(q) for _ in range(2)]
    m.moe_attn_batch(shape, q, k, v, dev(table), dev(lens), outs[0], ws, prefix=dev(kept))
    cache = m.make_cache_shape(B, own, n_phys, n_kv, D)
    cws = m.alloc_cache_workspace(cache, DEV)
    state = m.CacheMeta(dev(table[:, prefix:]), dev(lens - 64 * prefix), dev(refs))
    out, n_live = m.CacheMeta.empty(cache, DEV), torch.empty(1, dtype=torch.int32, device=DEV)
    moved = torch.empty(n_phys, dtype=torch.int32, device=DEV)
    m.moe_cache_compact(cache, state, out, n_live, m.pool_table([k, v]), cws, moved=moved)
    assert m.moe_query_device_status(cws) == 0 and n_live.item() == B * own + prefix
    now = moved[dev(kept).long()]
    assert (now < n_live).all() and (out.refs[dev(kept).long()] == 0).all()
    after = dev(table)
    after[:, prefix:] = out.table
    m.moe_attn_batch(shape, q, k, v, after, dev(lens), outs[1], ws, prefix=now)
    assert m.moe_query_device_status(ws) == 0
    assert torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16))


def test_binding_refuses_a_map_of_another_size():
    c = Cache(1, 3, 2, 9)
    n_live = torch.empty(1, dtype=torch.int32, device=DEV)
    for bad in (torch.empty(8, dtype=torch.int32, device=DEV),
                torch.empty(9, dtype=torch.int64, device=DEV), torch.empty(9, dtype=torch.int32)):
        with pytest.raises(ValueError):
            m.moe_cache_compact(c.shape, c.meta, c.out, n_live, c.table, c.ws, moved=bad)
