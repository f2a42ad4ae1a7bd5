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


@BOTH
@EACH
def test_slots_that_end_on_every_side_of_the_prefix(T, n_q, n_kv, D, prefix, dtype):
    """Past it, with it, inside it, in its first page, nothing at all."""
    P = prefix * 64
    pairs = [(P + 5, T), (P + 200, T), (P + 64, 1), (P, T), (P - 10, T), (T, T), (0, 0), (P + 1, 1)]
    Shared(prefix + T, pairs * 8, T, n_q, n_kv, D, prefix=prefix, dtype=dtype).check()


# the height of each step's scores (two pages), in log2 units above the first
LEVELS = [0, 5, 9.5, 9.5, 4, 18, 18, 14, 18.25]


@BOTH
@pytest.mark.parametrize("D", [64, 128])
def test_scores_that_rise_past_the_lag(D, dtype):
    """Half of the heads see scores that rise by more than 2^8 from one step
    to a later one, so that what was summed before has to be scaled, while the
    other half's fall; within the lag and below nothing is scaled. The values
    shrink as the scores of the rising half grow, so that the early steps weigh
    as much in its outputs as the last."""
    n_kv, T, prefix = 8, 4, 18
    c = Shared(D, [(64 * prefix + 40 + s, T) for s in range(64)], T, 64, n_kv, D, prefix=prefix,
               dtype=dtype, scale=0.2)
    slope = np.sqrt(D) / np.log2(np.e) / 8  # of k[0] per unit of height, q[0] being 8

    def level(page, at):
        seen = ~torch.isnan(c.k[page, :, :, 0])
        c.k[page, :, :, 0] = torch.where(seen, at * slope, float("nan")).to(c.k.dtype)
        c.v[page] = (c.v[page].double() * 2.0 ** (13 - at)).to(c.v.dtype)
    for j, p in enumerate(c.prefix):
        level(p, LEVELS[j // 2])
    for s in range(64):
        level(c.table[s, prefix], LEVELS[-1])
    c.q[..., 0] = torch.where(torch.arange(64) % 2 == 0, 8.0, -8.0).to(c.q.dtype)
    c.check()


@BOTH
def test_sharp_flat_and_large_scores(dtype):
    """All scores alike (the mean of the values); one position that takes
    everything, in the prefix or past it; scores far past what an exponential
    without its maximum could hold."""
    prefix = 18
    pairs = [(64 * prefix + 70, 1), (500, 1)] * 32
    Shared(9, pairs, 1, 16, 2, 128, prefix=prefix, dtype=dtype, scale=0.0).check()
    c = Shared(10, pairs, 1, 16, 2, 128, prefix=prefix, dtype=dtype, scale=3.0)
    for s in range(0, 64, 2):
        c.q[s, 0, 0] = (c.k[c.prefix[s // 4], 0, 3].double() * 2).to(c.q.dtype)
        c.q[s, 0, 15] = (c.k[c.table[s, prefix + 1], 1, 5].double() * 2).to(c.q.dtype)
    c.check()
    Shared(11, pairs, 1, 16, 2, 128, prefix=prefix, dtype=dtype, scale=20.0).check()


@BOTH
@pytest.mark.parametrize("where", [0, 1, 8, 16])
def test_a_bad_prefix_page_is_recorded_and_left_out(where, dtype):
    """In either half of a step, alone in the last one, below the pool and
    past it."""
    prefix = 17
    pairs = [(64 * prefix + 20, 2), (64 * prefix - 5, 1), (64 * where + 64, 2), (1, 1)] * 16
    c = Shared(where, pairs, 2, 16, 2, 128, prefix=prefix, dtype=dtype)
    for wrong in (-3, c.k.shape[0], 1 << 30):
        pre = c.prefix.copy()
        gone, pre[where] = pre[where], wrong
        c.check(skip=(gone,), prefix=pre, status=m.MOE_ERR_BAD_INPUT)
    pre = np.full_like(c.prefix, -1)  # nothing of the prefix is left
    c.check(skip=tuple(c.prefix), prefix=pre, status=m.MOE_ERR_BAD_INPUT)


@BOTH
def test_replays_with_other_lengths(dtype):
    """Three kernels captured once, whose second starts beside the first. Own
    lines that are long, short, gone or those of a few slots divide the SMs
    otherwise; each replay has to give the bits of a call made then."""
    prefix, T = 18, 3
    c = Shared(18, [(64 * prefix + 600, T)] * 64, T, 16, 2, 128, prefix=prefix, dtype=dtype)
    B, _, n_q, n_kv, D, P, _ = c.dims
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    shape = m.make_attn_batch_shape(B, T, n_q, n_kv, D, c.table.shape[1], P, dtype)
    ws = m.alloc_attn_batch_workspace(shape, DEV)
    q, k, v, tab, pre = c.q.to(DEV), c.k.to(DEV), c.v.to(DEV), up(c.table), up(c.prefix)
    ln, nn, o = up(c.lens), up(c.n_new), torch.empty_like(c.q, device=DEV)
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=side):
        m.moe_attn_batch(shape, q, k, v, tab, ln, o, ws, n_new=nn, prefix=pre)
    rng = np.random.default_rng(5)
    for own in (np.full(B, 600), np.full(B, 3), rng.integers(1, 601, B), np.full(B, -64),
                np.where(np.arange(B) == 9, 600, 1), rng.integers(-64 * prefix, 601, B)):
        c.lens = (64 * prefix + own).astype(np.int32)
        c.n_new = np.minimum(rng.integers(0, T + 1, B), c.lens).astype(np.int32)
        ln.copy_(up(c.lens))
        nn.copy_(up(c.n_new))
        o.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(o.cpu().double().numpy(), c.check())
    assert m.moe_query_device_status(ws) == 0
