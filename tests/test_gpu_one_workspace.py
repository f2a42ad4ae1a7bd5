"""One workspace for a server whose batch grows and shrinks: calls of several
shapes in turn, in a workspace of the largest size, give the results that each
gives in one of its own."""
import numpy as np
import pytest
import torch

import bit_moe_expert_histogram_gb300 as m
import serve_ref as ref
from test_gpu_attn_batch import DEV, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    m.load()


def test_attention():
    """What a call leaves in the workspace must not count as the next one's
    arrivals, with and without a shared prompt. Pairs of few blocks on borders
    of the CTAs' shares are joined by counters; the others' parts could lie
    where a larger shape has its counters."""
    rng = np.random.default_rng(50)
    cases = [Case(50, [(2000, 2), (900, 1), (64, 1)] * 3, 2, 16, 2, 128),
             Case(51, [(int(n), 1) for n in rng.integers(1, 129, 128)], 1, 16, 2, 128),
             Case(52, [(64 * 20 + 90, 3)] * 40, 3, 16, 2, 128, prefix=20),
             Case(53, [(int(n), 2) for n in rng.integers(2, 129, 300)], 2, 8, 4, 64, dtype="fp16"),
             Case(54, [(100, 1)], 1, 16, 2, 128)]
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV)  # noqa: E731
    want, work = [c.check() for c in cases], []
    for c in cases:
        B, T, n_q, n_kv, D, P, dtype = c.dims
        shape = m.make_attn_batch_shape(B, T, n_q, n_kv, D, c.table.shape[1], P, dtype)
        work.append((shape, c.q.to(DEV), c.k.to(DEV), c.v.to(DEV), up(c.table), up(c.lens),
                     up(c.n_new), up(c.prefix) if P else None))
    need = [m.load().moe_attn_batch_workspace_bytes(w[0]) for w in work]
    ws = torch.empty(max(need), dtype=torch.uint8, device=DEV)
    m.moe_workspace_init(ws)
    order = [0, 1, 0, 1, 2, 1, 3, 2, 3, 4, 3, 0, 3, 1, 4, 2, 0]
    outs = [torch.full_like(work[i][1], 7.0) for i in order]
    for i, o in zip(order, outs):
        shape, q, k, v, tab, ln, nn, pre = work[i]
        m.moe_attn_batch(shape, q, k, v, tab, ln, o, ws, n_new=nn, prefix=pre)
    assert m.moe_query_device_status(ws) == 0
    for i, o in zip(order, outs):
        np.testing.assert_array_equal(o.cpu().double().numpy(), want[i], err_msg=str(i))


def test_verification():
    """Segments' sums of a small batch with a large vocabulary could lie where
    a large batch has its counters. Every output is written and right, however
    the batch changes."""
    g = torch.Generator().manual_seed(60)
    work, want = [], []
    for B, T, V, dtype in ((4, 2, 90000, "fp32"), (512, 3, 9000, "fp32"), (40, 1, 40000, "bf16"),
                           (1, 31, 5, "fp16"), (2000, 1, 300, "bf16")):
        dt = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
        p = torch.softmax(3 * torch.randn((B, T + 1, V), generator=g), -1).to(dt)
        draft = p[:, :T].float().argmax(-1).to(torch.int32)
        n = torch.randint(0, T + 1, (B,), generator=g, dtype=torch.int32)
        u = torch.rand((B, T + 1), generator=g)
        want.append(ref.verify(p.double().numpy(), None, draft.numpy(), n.numpy(),
                               u.double().numpy()))
        work.append((m.make_verify_shape(B, T, V, dtype), p.to(DEV), draft.to(DEV), n.to(DEV),
                     u.to(DEV)))
    need = [m.load().moe_verify_workspace_bytes(w[0]) for w in work]
    ws = torch.empty(max(need), dtype=torch.uint8, device=DEV)
    m.moe_workspace_init(ws)
    order, outs = [0, 1, 0, 1, 2, 1, 4, 0, 4, 3, 1, 2, 4, 1, 0], []
    for i in order:
        shape, p, draft, n, u = work[i]
        tokens = torch.full(u.shape, -7, dtype=torch.int32, device=DEV)
        acc = torch.full(n.shape, -7, dtype=torch.int32, device=DEV)
        m.moe_verify_drafts(shape, p, None, draft, n, u, tokens, acc, ws)
        outs.append((tokens, acc))
    assert m.moe_query_device_status(ws) == 0
    for i, (tokens, acc) in zip(order, outs):
        np.testing.assert_array_equal(tokens.cpu().numpy(), want[i][0], err_msg=str(i))
        np.testing.assert_array_equal(acc.cpu().numpy(), want[i][1], err_msg=str(i))
