"""Attention over 4-bit pages with queries and keys at the ends of the range that
the documentation gives them: elements of queries of up to 2^100 beside keys so
small that scores are ordinary numbers, the other way round, and heads of either
kind in one call. Queries carry a power of two of their row, so that the bound of
tests/q4_ref.py holds as it stands: what a clamped power loses is below 2^-121 an
element, 2^-20 of the largest where that is 2^-100 or more, and the bound allows
136 2^-22 of the sum of the products' magnitudes."""
import numpy as np
import pytest
import torch

import bit_moe_expert_histogram_gb300 as m
import q4_ref as ref
from test_gpu_attn_q4 import Case, wide

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    m.load()


def keys_times(c, head, factor):
    """The keys of `head` times a power of two: scales and biases alone change."""
    D = c.dims[4]
    raw = np.ascontiguousarray(c.k[:, head, :, D // 4:]).view(np.uint16)
    with np.errstate(invalid="ignore", over="ignore"):
        x = ref.bf16_of(raw) * np.float32(factor)
    c.k[:, head, :, D // 4:] = ref.bf16_bits(x).view(np.int16)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [1, 4])
@pytest.mark.parametrize("power", [-100, -60, 60, 96])
def test_queries_and_keys_far_from_1(D, T, power):
    # elements of normal rows are below 2^4 here: 2^96 keeps them below 2^100
    c = Case(70 + D + T, [(300, T), (64, 1), (129, min(T, 2))], T, 8, 2, D, "bf16", k_std=0.5)
    assert c.q.abs().max() < 16
    if T > 1:
        c = wide(c)
    for head, p in ((0, power), (1, -power if -power <= 96 else 96)):
        c.q[:, :, 4 * head:4 * head + 4] = (c.q[:, :, 4 * head:4 * head + 4].double() * 2.0**p).to(torch.bfloat16)
        keys_times(c, head, 2.0**-p)
    c.check()
