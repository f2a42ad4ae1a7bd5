"""moe_cache_fork: a parent that is no slot is recorded, on either side of the
slots' numbers; -1 is the way to leave a slot empty."""
import numpy as np
import pytest
import torch

import bit_moe_expert_histogram_gb300 as m
import serve_ref as ref
from test_gpu_cache import Cache, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    m.load()


@pytest.mark.parametrize("n_slots", [4, 300])  # one CTA, and a CTA a slot
@pytest.mark.parametrize("parent,status", [(-1, 0), (-2, m.MOE_ERR_BAD_INPUT),
                                           (-2 ** 31, m.MOE_ERR_BAD_INPUT),
                                           (2 ** 31 - 1, m.MOE_ERR_BAD_INPUT)])
def test_parent_out_of_range(n_slots, parent, status):
    c = Cache(7, n_slots, 5, 6 * n_slots, pools=1, D=8)
    parents = np.arange(n_slots, dtype=np.int32)
    parents[2] = parent
    m.moe_cache_fork(c.shape, c.meta, dev(parents), c.out, c.ws)
    c.check(ref.fork(*c.host, parents, None), status)
