"""The binding copies rows as they are, so it refuses tensors of two types:
fp16 keys in a bf16 pool would be read as other numbers. int16 tensors are
bits of either type."""
import numpy as np
import pytest
import torch

import bit_moe_expert_histogram_gb300 as m

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    m.load()


def state(shape):
    ints = lambda a: torch.from_numpy(np.asarray(a, np.int32)).to(DEV)  # noqa: E731
    return m.CacheMeta(ints([[1, -1], [2, -1]]), ints([3, 1]), ints([0, 1, 1, 0]))


def test_write_wants_one_type():
    shape = m.make_cache_shape(2, 2, 4, 2, 64)
    ws, meta = m.alloc_cache_workspace(shape, DEV), state(shape)
    bf, fp, raw = torch.bfloat16, torch.float16, torch.int16
    for kn, vn, kc, vc, good in ((bf, bf, bf, bf, True), (fp, fp, fp, fp, True),
                                 (bf, fp, bf, fp, True), (raw, bf, bf, raw, True),
                                 (fp, bf, bf, bf, False), (bf, bf, bf, fp, False),
                                 (bf, fp, fp, bf, False)):
        new = [torch.full((2, 1, 2, 64), 1.0 + i, device=DEV).to(t) for i, t in enumerate((kn, vn))]
        pools = [torch.zeros((4, 2, 64, 64), dtype=t, device=DEV) for t in (kc, vc)]
        if not good:
            with pytest.raises(ValueError):
                m.moe_cache_write(shape, meta, None, *new, *pools, ws)
            assert not any(p.any() for p in pools)
            continue
        m.moe_cache_write(shape, meta, None, *new, *pools, ws)
        for p, x in zip(pools, new):
            for page, row in ((1, 2), (2, 0)):
                assert torch.equal(p[page, :, row].view(raw), x[page - 1, 0].view(raw))
    assert m.moe_query_device_status(ws) == 0


def test_page_copies_want_one_type():
    shape = m.make_cache_shape(2, 2, 4, 2, 64)
    ws = m.alloc_cache_workspace(shape, DEV)
    one = torch.zeros(1, dtype=torch.int32, device=DEV)
    pool = lambda t, v: torch.full((4, 2, 64, 64), v, dtype=t, device=DEV)  # noqa: E731
    a = m.pool_table([pool(torch.bfloat16, 1), pool(torch.bfloat16, 2)])
    with pytest.raises(ValueError):
        m.moe_cache_copy_pages(shape, one, one, a, m.pool_table(
            [pool(torch.bfloat16, 0), pool(torch.float16, 0)]), ws)
    to = [pool(torch.int16, 0), pool(torch.bfloat16, 0)]
    m.moe_cache_copy_pages(shape, one, one, a, m.pool_table(to), ws)
    assert m.moe_query_device_status(ws) == 0
    assert torch.equal(to[0].view(torch.bfloat16)[0], a.pools[0][0])
    assert torch.equal(to[1][0], a.pools[1][0]) and not to[1][1:].any()
