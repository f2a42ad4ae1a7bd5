"""Attention over 4-bit pages where pairs are cut by many CTAs: what is joined is
what this call left in the workspace, never a part of the call before, and the
order in which the CTAs arrive changes nothing. Calls that differ in the queries
alone take turns on one workspace; each has to repeat, bit for bit, what it gives
with a workspace of its own."""
import numpy as np
import pytest
import torch

import bit_moe_expert_histogram_gb300 as m
from test_gpu_attn_q4 import Case, ints, some, wide

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    m.load()


CASES = {
    "one slot over all CTAs": (False, [(40000, 1)], 1, 16, 2, 128, "bf16"),
    "two rows of items a warp": (False, [(30000, 2), (5000, 1)], 2, 8, 2, 64, "fp16"),
    "sixteen rows": (True, [(9000, 4), (12000, 3)], 4, 16, 2, 128, "bf16"),
    "sixteen rows, D = 64": (True, [(9000, 4), (7000, 4)], 4, 12, 4, 64, "bf16"),
}


@pytest.mark.parametrize("name", list(CASES))
def test_parts_are_the_calls_own(name):
    w, slots, T, n_q, n_kv, D, dtype = CASES[name]
    c = Case(50 + len(name), slots, T, n_q, n_kv, D, dtype, k_std=0.3)
    c = wide(c) if w else c
    shape = c.shape()
    k, v = torch.from_numpy(c.k).to(DEV), torch.from_numpy(c.v).to(DEV)
    table, lens, new = ints(c.table), ints(c.lens), ints(c.new)
    qs = [c.q.to(DEV), -c.q.to(DEV), c.q.flip(-1).contiguous().to(DEV)]

    def call(q, o, ws):
        m.moe_attn_batch_q4(shape, q, k, v, table, lens, o, ws, n_new=new)

    alone = [torch.empty_like(q) for q in qs]
    for q, o in zip(qs, alone):
        call(q, o, m.alloc_attn_batch_q4_workspace(shape, DEV))
    c.check(o=alone[0])
    assert not torch.equal(alone[0], alone[1]) and not torch.equal(alone[0], alone[2])
    ws = m.alloc_attn_batch_q4_workspace(shape, DEV)
    turns = [(i * i + i // 7) % 3 for i in range(120)]
    got = torch.empty((len(turns), *c.q.shape), dtype=c.q.dtype, device=DEV)
    for i, j in enumerate(turns):  # back to back: nothing waits in between
        call(qs[j], got[i], ws)
    assert m.moe_query_device_status(ws) == 0
    for i, j in enumerate(turns):
        assert torch.equal(got[i], alone[j]), i


def test_more_slots_than_threads_in_tiles_of_sixteen():
    """Each thread of the scan has several slots, tiles have sixteen rows."""
    rng = np.random.default_rng(60)
    c = wide(Case(61, some(rng, 300, 250, 4), 4, 16, 2, 128, "bf16", 0.3))
    first = c.call()
    c.check(o=first)
    assert torch.equal(c.call(ws=c.ws), first)
    wide(Case(62, some(rng, 600, 120, 3), 3, 12, 4, 64, "fp16", 0.3)).check()
