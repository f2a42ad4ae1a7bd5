"""moe_verify_drafts at the ends of fp32's range: rows need not sum to 1, but
a sum that is no number of the type decides nothing."""
import numpy as np
import pytest
import torch

import bit_moe_expert_histogram_gb300 as m
from test_gpu_verify import check, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    m.load()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V", [40, 9000])
@pytest.mark.parametrize("apart", [1, 7, 33])
def test_a_sum_past_the_range_is_recorded(dtype, V, apart):
    """Slot 1's row sums to 4.5e38, in one thread, warp or over several; the
    others' tokens are as ever. Rejected and accepted drafts alike."""
    dt = {"fp32": torch.float32, "bf16": torch.bfloat16}[dtype]
    p = torch.softmax(torch.randn((3, 2, V), generator=torch.Generator().manual_seed(V)), -1).to(dt)
    u = np.float32([[0.5, 0.3]] * 3)
    want, acc = check(p, None, np.full((3, 1), 2), [1, 0, 1], u, dtype)
    p[1, :, 0], p[1, :, apart] = 3e38, 1.5e38
    got = run(p, None, np.full((3, 1), 2), [1, 0, 1], u, dtype, m.MOE_ERR_BAD_INPUT)
    assert got[0][1].tolist() == [-1, -1]
    np.testing.assert_array_equal(got[0][[0, 2]], want[[0, 2]])
    np.testing.assert_array_equal(got[1], acc)
    # drafted and rejected: the difference from the certain draft still sums to it
    got = run(p, None, np.full((3, 1), 2), [1, 1, 1], np.float32([[0.999, 0.3]] * 3), dtype,
              m.MOE_ERR_BAD_INPUT)
    assert got[0][1].tolist() == [-1, -1] and got[1][1] == 0


def test_large_and_small_sums():
    """Just below the largest number, and 2^-100: thresholds as ever."""
    V = 5000
    p = torch.zeros((4, 2, V))
    p[0, :, 17], p[0, :, 4500] = 1.6e38, 1.7e38
    p[1] = 2.0 ** 114  # 1.04e38 in all
    p[2] = 2.0 ** -112
    p[3, :, 1], p[3, :, 4999] = 2.0 ** -101, 2.0 ** -101
    for u1 in (0.0, 0.25, 0.4999, 0.50001, 0.99999):
        check(p, None, np.zeros((4, 1)), np.zeros(4, np.int32), np.float32([[0.5, u1]] * 4), "fp32")
