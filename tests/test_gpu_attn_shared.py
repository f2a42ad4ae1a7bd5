"""The shared part of the batch's attention (attn_prefix_kernel) at sizes that
take it, against a plain evaluation in 64 bits. Few slots or short prompts are
read by every slot for itself, so each test here also looks at the kernels
that its call launched.

Tolerance: the one of test_gpu_attn_batch, 2 h |o| + h A + 2^-14 A with
A = sum w_j |v_j|, holds for scores of up to 40 in log2 units. A score
x = log2(e) q.k / sqrt(D) is a sum of D fp32 products, off by at most
D 2^-23 X with X = log2(e) sum |q_d k_d| / sqrt(D) (2^-23: an addition may cut
instead of rounding), and 2^x by ln 2 times that, in the weights and in their
sum; so 2 ln(2) D 2^-23 X A comes on top, X being the row's largest."""
import numpy as np
import pytest
import torch

import bit_moe_expert_histogram_gb300 as m
from test_gpu_attn_batch import DEV, TYPES, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    m.load()


def kernels_of(fn):
    """Names of the kernels that fn launches, [] where none were recorded."""
    from torch.autograd import DeviceType
    from torch.profiler import ProfilerActivity, profile
    for _ in range(2):  # the first trace of a process can come back empty
        torch.cuda.synchronize()
        with profile(activities=[ProfilerActivity.CUDA]) as prof:
            fn()
            torch.cuda.synchronize()
        names = [e.name for e in prof.events() if e.device_type == DeviceType.CUDA]
        if names:
            break
    return names


class Shared(Case):
    """A case whose prefix is read once for all slots."""

    def largest(self):
        """X of each row, spread over its elements."""
        B, T, n_q, n_kv, D, P, _ = self.dims
        k, q = self.k.double().abs().numpy(), self.q.double().abs().numpy()
        X, G = np.zeros((B, T, n_q, D)), n_q // n_kv
        for s in range(B):
            L = int(self.lens[s])
            blocks = [self.prefix[j] if j < P else self.table[s, j] for j in range(-(-L // 64))]
            for h in range(n_kv):
                if L:
                    kk = np.concatenate([k[p, h] for p in blocks])[:L]
                    x = q[s, :, h * G:(h + 1) * G] @ kk.T
                    X[s, :, h * G:(h + 1) * G] = x.max(-1, keepdims=True)
        return X * np.log2(np.e) / np.sqrt(D)

    def check(self, skip=(), **kw):
        got = self.run(**kw)
        o, A = self.want(skip)
        D, dtype = self.dims[4], self.dims[6]
        h = torch.finfo(TYPES[dtype]).eps / 2
        assert np.isfinite(got).all()
        tol = 2 * h * np.abs(o) + (h + 2.0 ** -14 + 2 * np.log(2) * D * 2.0 ** -23 * self.largest()) * A
        off = np.abs(got - o) - tol
        assert off.max() <= 0, "over by %.3g at %s" % (off.max(),
                                                       np.unravel_index(off.argmax(), off.shape))
        names = kernels_of(lambda: self.run(**kw))
        assert not names or any("attn_prefix_kernel" in n for n in names), names
        return got


SHAPES = [(1, 16, 2, 128, 17), (3, 12, 4, 64, 18), (4, 16, 2, 128, 17), (8, 8, 1, 64, 41)]
BOTH = pytest.mark.parametrize("dtype", ["bf16", "fp16"])
EACH = pytest.mark.parametrize("T,n_q,n_kv,D,prefix", SHAPES)


@BOTH
@EACH
@pytest.mark.parametrize("short", [0, 10, 64, 94, 129, -1])
def test_pages_past_every_slot_hold_anything(short, T, n_q, n_kv, D, prefix, dtype):
    """No slot reaches the prefix's last `short` positions (-1: all but 70),
    whose keys and values are NaN and infinities, as in pages not written yet:
    the ends lie in either page of a step, at a page's border, and early."""
    last = 70 if short < 0 else prefix * 64 - short
    rng = np.random.default_rng(last)
    pairs = [(int(n), int(rng.integers(0, T + 1))) for n in rng.integers(0, last + 1, 64)]
    pairs[7], pairs[40] = (last, T), (last, 1)
    c = Shared(last + T, pairs, T, n_q, n_kv, D, prefix=prefix, dtype=dtype)
    for j, p in enumerate(c.prefix):
        rows = max(0, min(64, last - 64 * j))
        c.k[p, :, rows:], c.v[p, :, rows:] = float("nan"), float("nan")
        c.v[p, :, rows::2] = float("inf")
        if rows < 64:
            c.k[p, 0, rows] = float("-inf")
    c.check()
