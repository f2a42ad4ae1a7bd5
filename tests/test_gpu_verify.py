"""GPU parity of draft verification (moe_verify_drafts) with the plain
reference in 64 bits: token ids and counts, all equal. The values of the
inputs are exact in 64 bits, and the sums of both sides are off by less than
2^-40 of the total, so only a threshold that close to a border could tell
them apart; the drawn numbers are fixed by their seeds."""
import numpy as np
import pytest
import torch

import bit_moe_expert_histogram_gb300 as m
import serve_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    m.load()


def run(p, q, draft, n_draft, u, dtype, want_status=0):
    """p, q: torch tensors of the type; the rest numpy."""
    B, T1, V = p.shape
    shape = m.make_verify_shape(B, T1 - 1, V, dtype)
    ws = m.alloc_verify_workspace(shape, DEV)
    tokens = torch.full((B, T1), -7, dtype=torch.int32, device=DEV)
    acc = torch.full((B,), -7, dtype=torch.int32, device=DEV)
    d = torch.from_numpy(np.ascontiguousarray(draft, np.int32)).to(DEV)
    n = None if n_draft is None else torch.from_numpy(np.asarray(n_draft, np.int32)).to(DEV)
    ut = torch.from_numpy(np.ascontiguousarray(u, np.float32)).to(DEV)
    for _ in range(2):  # the second call finds the counters as the first left them
        m.moe_verify_drafts(shape, p.to(DEV), None if q is None else q.to(DEV), d, n, ut, tokens,
                            acc, ws)
        assert m.moe_query_device_status(ws) == want_status
    return tokens.cpu().numpy(), acc.cpu().numpy()


def check(p, q, draft, n_draft, u, dtype, want_status=0):
    got = run(p, q, draft, n_draft, u, dtype, want_status)
    B, T1, _ = p.shape
    want = ref.verify(p.double().numpy(), None if q is None else q.double().numpy(),
                      np.asarray(draft, np.int32), np.full(B, T1 - 1) if n_draft is None else n_draft,
                      np.asarray(u, np.float32).astype(np.float64))
    np.testing.assert_array_equal(got[1], want[1])
    np.testing.assert_array_equal(got[0], want[0])
    return got


def draws(seed, B, T, V, dtype, sharp=3.0):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn((B, T + 1, V), generator=g) * sharp
    p = torch.softmax(z, -1)
    q = torch.softmax(z[:, :T] + 0.7 * torch.randn((B, T, V), generator=g), -1)
    draft = torch.multinomial(q.view(-1, V), 1, generator=g).view(B, T).numpy().astype(np.int32)
    n = torch.randint(0, T + 1, (B,), generator=g).numpy().astype(np.int32)
    u = torch.rand((B, T + 1), generator=g).numpy()
    return p.to(TYPES[dtype]), q.to(TYPES[dtype]), draft, n, u


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("B,T,V", [(1, 1, 1), (3, 2, 17), (40, 4, 4096), (9, 8, 4097), (5, 31, 1000),
                                   (17, 3, 32000), (2, 2, 131071), (64, 1, 255)])
def test_verify(B, T, V, dtype):
    p, q, draft, n, u = draws(B * 1000 + T, B, T, V, dtype)
    check(p, q, draft, n, u, dtype)
    check(p, q, draft, None, u, dtype)
    check(p, None, draft, n, u, dtype)


def test_many_thresholds_on_a_flat_row():
    """Every weight alike: the token is floor(u V), for thresholds at the very
    borders too (the sums of equal powers of two are exact)."""
    V, B = 8192, 512
    p = torch.full((B, 2, V), 1.0 / V)
    u = np.zeros((B, 2), np.float32)
    u[:, 1] = (np.arange(B) * 16) / V
    got, acc = check(p, None, np.zeros((B, 1)), np.zeros(B, np.int32), u, "fp32")
    assert got[:, 0].tolist() == [16 * i for i in range(B)] and not acc.any()


def test_zero_weights_are_never_drawn():
    V = 10000
    p = torch.zeros((4, 2, V))
    p[0, :, 9999] = 1.0     # the last
    p[1, :, 0] = 1.0        # the first
    p[2, :, 4096] = 0.5     # a segment's first
    p[2, :, 4095] = 0.5     # a segment's last
    p[3, :, 5000] = 1e-40   # a subnormal alone
    for u1 in (0.0, 0.4999, 0.5, 0.99999994, 1.0):  # 1.0 is out of range: the last that weighs
        got, _ = check(p, None, np.zeros((4, 1)), np.zeros(4, np.int32),
                       np.tile(np.float32([0.5, u1]), (4, 1)), "fp32")
        assert got[:, 0].tolist() == [9999, 0, 4095 if u1 < 0.5 else 4096, 5000]


def test_difference_that_leaves_nothing_falls_back_to_the_target():
    V = 6000
    p = torch.softmax(torch.randn((2, 2, V), generator=torch.Generator().manual_seed(1)), -1)
    q = p[:, :1] * 2  # nowhere below p
    check(p, q, np.array([[5], [700]]), [1, 1], np.float32([[0.9, 0.3], [0.5, 0.7]]), "fp32")


def test_borders_of_acceptance():
    """u q = p is a rejection, the number before it is not; one-hot rows
    (greedy decoding) accept their token whatever u is and no other."""
    p = torch.tensor([[[0.25, 0.75], [0.5, 0.5]]] * 2)
    q = torch.tensor([[[0.5, 0.5]]] * 2)
    u = np.float32([[0.5, 0.1], [np.nextafter(np.float32(0.5), np.float32(0)), 0.1]])
    _, acc = check(p, q, np.zeros((2, 1)), [1, 1], u, "fp32")
    assert acc.tolist() == [0, 1]
    hot = torch.zeros((1, 4, 50))
    for t, x in enumerate((7, 9, 11, 13)):
        hot[0, t, x] = 1.0
    got, acc = check(hot, None, np.array([[7, 9, 12]]), [3],
                     np.float32([[0.999, 0.0, 0.0, 0.6]]), "fp32")
    assert got.tolist() == [[7, 9, 11, -1]] and acc.tolist() == [2]


def test_what_is_not_finite_weighs_nothing():
    p = torch.full((3, 1 + 1, 5000), 1e-4)
    p[0, :, 10] = float("nan")
    p[1, :, 20] = float("inf")
    p[2, :, 30] = -1.0
    q = torch.zeros((3, 1, 5000))
    q[0, 0, 40] = float("nan")
    q[1, 0, 50] = float("inf")
    for x in (3, 10, 20):
        check(p, q, np.full((3, 1), x), [1, 1, 0], np.float32([[0.5, 0.002]] * 3), "fp32")


def test_bad_ids_counts_and_rows_are_recorded():
    p, q, draft, _, u = draws(3, 4, 2, 300, "fp32")
    draft[0, 0], draft[1, 1] = 300, -1
    u[1, 0] = 0.0  # slot 1 gets as far as its second draft
    check(p, q, draft, [2, 2, 2, 2], u, "fp32", m.MOE_ERR_BAD_INPUT)
    check(p, None, draft, [2, 2, 2, 2], u, "fp32", m.MOE_ERR_BAD_INPUT)
    p[2] = 0.0
    got, acc = run(p, q, np.zeros((4, 2)), [0, 0, 0, 0], u, "fp32", m.MOE_ERR_BAD_INPUT)
    assert got[2].tolist() == [-1, -1, -1] and acc[2] == 0
    # a count out of range is brought into it
    got, acc = run(p[:2], q[:2], np.zeros((2, 2)), [-4, 9], u[:2], "fp32", m.MOE_ERR_BAD_INPUT)
    want = ref.verify(p[:2].double().numpy(), q[:2].double().numpy(), np.zeros((2, 2), int), [0, 2],
                      u[:2].astype(np.float64))
    np.testing.assert_array_equal(got, want[0])


def test_rows_at_odd_addresses():
    """p and q as slices that start one element into their storage."""
    p, q, draft, n, u = draws(8, 6, 3, 5001, "bf16")
    shape = m.make_verify_shape(6, 3, 5001, "bf16")
    ws = m.alloc_verify_workspace(shape, DEV)

    def shifted(t):
        s = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)[1:]
        return s.copy_(t.reshape(-1)).view(t.shape)
    tokens = torch.empty((6, 4), dtype=torch.int32, device=DEV)
    acc = torch.empty(6, dtype=torch.int32, device=DEV)
    m.moe_verify_drafts(shape, shifted(p), shifted(q), torch.from_numpy(draft).to(DEV),
                        torch.from_numpy(n).to(DEV), torch.from_numpy(u).to(DEV), tokens, acc, ws)
    want = ref.verify(p.double().numpy(), q.double().numpy(), draft, n, u.astype(np.float64))
    np.testing.assert_array_equal(tokens.cpu().numpy(), want[0])
    np.testing.assert_array_equal(acc.cpu().numpy(), want[1])


def test_graph_replays_with_new_numbers():
    """Captured once; the random numbers of the time decide."""
    p, q, draft, n, u = draws(9, 40, 4, 20000, "fp32")
    shape = m.make_verify_shape(40, 4, 20000, "fp32")
    ws = m.alloc_verify_workspace(shape, DEV)
    tokens = torch.empty((40, 5), dtype=torch.int32, device=DEV)
    acc = torch.empty(40, dtype=torch.int32, device=DEV)
    dp, dq, dd, dn = p.to(DEV), q.to(DEV), torch.from_numpy(draft).to(DEV), torch.from_numpy(n).to(DEV)
    du = torch.from_numpy(u).to(DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        m.moe_verify_drafts(shape, dp, dq, dd, dn, du, tokens, acc, ws)
    for seed in range(4):
        u = np.random.default_rng(seed).random((40, 5), np.float32)
        du.copy_(torch.from_numpy(u))
        g.replay()
        torch.cuda.synchronize()
        want = ref.verify(p.double().numpy(), q.double().numpy(), draft, n, u.astype(np.float64))
        np.testing.assert_array_equal(tokens.cpu().numpy(), want[0])
        np.testing.assert_array_equal(acc.cpu().numpy(), want[1])


def test_binding_refuses_wrong_tensors():
    shape = m.make_verify_shape(2, 2, 100, "fp32")
    ws = m.alloc_verify_workspace(shape, DEV)
    f = lambda *s: torch.zeros(s, device=DEV)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)  # noqa: E731
    good = [f(2, 3, 100), f(2, 2, 100), i(2, 2), i(2), f(2, 3), i(2, 3), i(2)]
    for k, bad in ((0, f(2, 2, 100)), (0, f(2, 3, 100).half()), (1, f(2, 3, 100)), (2, i(2, 3)),
                   (2, i(2, 2).long()), (4, f(2, 2)), (5, i(2, 2)), (6, i(3)),
                   (0, f(3, 2, 100).transpose(0, 1))):
        args = list(good)
        args[k] = bad
        with pytest.raises(ValueError):
            m.moe_verify_drafts(shape, *args, ws)
