"""Log probabilities of rows whose low ids cannot be: a grammar or a slice of the
vocabulary that forbids the first of a row's chunks, or all of a stretch where
rows are cut, so that the likeliest come from what follows nothing. Ordinary,
distinct logits behind it, few of them, or the type's lowest number in between."""
import pytest
import torch

import bit_moe_expert_histogram_gb300 as m
from test_gpu_logprobs import DEV, TYPES, call, check, logits

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    m.load()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n,V", [(6, 40000), (6, 131072), (640, 40000)])
@pytest.mark.parametrize("k", [1, 20, 32])
def test_rows_whose_first_ids_cannot_be(dtype, n, V, k):
    """Few rows are cut in stretches, 640 are not."""
    x = logits(80 + V + k, n, V, dtype)
    low = torch.finfo(TYPES[dtype]).min
    x[0, :V // 2] = -INF
    x[1, :16384] = -INF
    x[2, :V - 15] = -INF               # fewer than k are left, at the end
    x[3, 10:V - 10] = -INF             # at both ends
    x[4, :20000], x[4, 20000:V - 3] = -INF, low
    x[5, 5:V - 5000] = low             # a few, then the lowest number, then ordinary ones
    tokens = [(i * 7919 + V - 1) % V for i in range(n)]
    got = call(x, tokens, k)
    check(x[:6], tokens[:6], k, [y[:6] for y in got])


def test_a_bad_row_without_a_token():
    x = logits(90, 3, 500, "fp32")
    x[0, 7], x[1] = float("nan"), -INF
    lp, ent, ids, top = call(x, [-1, -1, -1], 2, status=m.MOE_ERR_BAD_INPUT)
    assert lp.tolist() == [0, 0, 0] and ent[:2].isnan().all() and ent[2].isfinite()
    assert (ids[:2] == -1).all() and (top[:2] == -INF).all()
