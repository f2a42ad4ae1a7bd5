"""Log probabilities of given tokens, entropies and likeliest tokens against 64
bits. Bound: an element's exponential is off by 2^-22 (its approximation) and
2^-22 |d| e^d <= 2^-23 of the largest (roundings of d); a thread adds up to
V / 512 of them and 16 such sums follow, 2^-24 each: ln Z is off by less than
2^-20 + (V / 512 + 16) 2^-24, log probabilities by that and two roundings of
their own, entropies by that times 2 + H (A / Z) and a rounding."""
import numpy as np
import pytest
import torch

import bit_moe_expert_histogram_gb300 as m
import q4_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    m.load()


def call(x, tokens, k, ws=None, status=0, parts=True):
    n, V = x.shape
    name = {v: a for a, v in TYPES.items()}[x.dtype]
    shape = m.make_logprobs_shape(n, V, k, name)
    if ws is None:
        ws = m.alloc_logprobs_workspace(shape, DEV)
    f = lambda *s: torch.full(s, 7.0, device=DEV)  # noqa: E731
    lp, ent = f(n), f(n) if parts else None
    ids = torch.full((n, k), -7, dtype=torch.int32, device=DEV) if k and parts else None
    top = f(n, k) if k and parts else None
    m.moe_token_logprobs(shape, x, torch.tensor(tokens, dtype=torch.int32, device=DEV), lp, ws,
                         entropy=ent, top_ids=ids, top_logp=top)
    if status is not None:
        assert m.moe_query_device_status(ws) == status
    return lp, ent, ids, top


def check(x, tokens, k, got=None):
    V = x.shape[1]
    lp, ent, ids, top = call(x, tokens, k) if got is None else got
    wlp, went, wids, wtop = ref.logprobs(x.cpu().double().numpy(), tokens, k)
    z = 2.0**-20 + (V / 512 + 16) * 2.0**-24
    near = lambda a, b, t: np.all((np.abs(a.cpu().double().numpy() - b) <= t) | (a.cpu().double().numpy() == b))  # noqa: E731
    with np.errstate(invalid="ignore"):
        assert near(lp, wlp, z + 2.0**-23 * np.abs(np.where(np.isinf(wlp), 0, wlp)) + 2.0**-23 * 12)
        assert near(ent, went, (2 + went) * (z + 2.0**-22))
        if k:
            np.testing.assert_array_equal(ids.cpu().numpy(), wids)
            assert near(top, wtop, z + 2.0**-23 * np.abs(np.where(np.isinf(wtop), 0, wtop)) + 2.0**-23 * 12)


def logits(seed, n, V, dtype, std=3.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((n, V), generator=g) * std).to(TYPES[dtype]).to(DEV)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n,V,k", [(1, 1, 1), (3, 2, 5), (2, 31, 32), (5, 33, 20), (4, 1000, 32), (2, 8191, 7),
                                   (3, 16385, 20), (1, 70001, 32), (40, 5000, 1), (700, 333, 4), (2, 131072, 0)])
def test_against_64_bits(dtype, n, V, k):
    x = logits(n + V, n, V, dtype)
    tokens = [(i * 7919 + 5) % V if i % 4 != 3 else -1 for i in range(n)]
    check(x, tokens, k)


def test_a_large_vocabulary():
    check(logits(1, 2, 1 << 20, "fp32"), [5, (1 << 20) - 1], 32)
    check(logits(2, 1, 1 << 20, "bf16"), [77], 20)


@pytest.mark.parametrize("dtype,offset,pad", [("bf16", 0, 1), ("bf16", 3, 5), ("fp16", 7, 0), ("fp32", 1, 2),
                                              ("fp32", 3, 0), ("bf16", 1, 7)])
def test_rows_that_lie_apart_and_start_anywhere(dtype, offset, pad):
    n, V = 5, 20011
    full = logits(3, n, offset + V + pad, dtype)
    full[:, :offset], full[:, offset + V:] = float("nan"), float("inf")  # must not be seen
    x = full[:, offset:offset + V]
    check(x, [0, V - 1, 17, -1, 3], 9, call(x, [0, V - 1, 17, -1, 3], 9))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [100, 5000, 40000])
def test_equal_logits_go_to_the_lower_id(dtype, V):
    g = torch.Generator().manual_seed(V)
    few = torch.randint(0, 6, (4, V), generator=g).float()     # six different numbers
    flat = torch.zeros((1, V))                                 # one
    two = torch.zeros((1, V))
    two[0, V // 2:] = 1.0                                      # the upper half ahead
    x = torch.cat([few, flat, two, -two]).to(TYPES[dtype]).to(DEV)
    for k in (1, 20, 32):
        check(x, [1] * 7, k)


@pytest.mark.parametrize("dtype,V", [("fp32", 30000), ("bf16", 60000), ("fp16", 2000)])
def test_sorted_and_crowded_logits(dtype, V):
    """Rising logits bring every chunk's elements into the list, and strong
    ones that one thread reads alone crowd it."""
    up = torch.linspace(-30, 30, V)
    crowd = torch.randn(V, generator=torch.Generator().manual_seed(1))
    for i in range(0, V, 4096):
        crowd[i:i + 130] = 20 + torch.rand(len(crowd[i:i + 130]))
    late = torch.full((V,), -5.0)
    late[-3:] = torch.tensor([1.0, 2.0, 1.0])
    x = torch.stack([up, up.flip(0), crowd, late]).to(TYPES[dtype]).to(DEV)
    for k in (1, 5, 32):
        check(x, [0, V - 1, 2, V - 1], k)


def test_many_above_the_bar():
    """One group of threads holds the thousand largest: more than the list."""
    V = 65536
    x = torch.randn(V, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    ids = torch.arange(V)
    group = (ids // 8 % 512) < 64  # the first two warps' vectors, every chunk
    y = torch.where(group, x.abs() + 30, x)
    check(torch.stack([y, x]).to(DEV), [3, 4], 32)
    z = torch.full((V,), -float("inf"), dtype=torch.bfloat16)
    z[group & (ids % 8 < 6)] = y[group & (ids % 8 < 6)]
    check(torch.stack([z, y.flip(0)]).to(DEV), [0, 1], 20)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_tokens_that_cannot_be(dtype):
    x = logits(6, 4, 9000, dtype)
    x[0, 3:] = -float("inf")     # three are left
    x[1, :8999] = -float("inf")  # one
    x[2, ::2] = -float("inf")
    check(x, [1, 8999, 1, 0], 10)
    lp, _, ids, top = call(x, [5, 0, 2, 0], 10)
    assert lp[:3].tolist() == [-float("inf")] * 3
    assert ids[0].tolist()[3:] == [-1] * 7 and ids[1].tolist() == [8999] + [-1] * 9
    assert top[1, 0] == 0 and top[1, 1] == -float("inf")


def test_rows_without_a_distribution_are_recorded():
    x = logits(7, 4, 3000, "fp32")
    x[0], x[1, 5], x[2, 6] = -float("inf"), float("nan"), float("inf")
    lp, ent, ids, top = call(x, [1, 2, 3, 4], 3, status=m.MOE_ERR_BAD_INPUT)
    assert lp[:3].isnan().all() and ent[:3].isnan().all() and (ids[:3] == -1).all()
    assert (top[:3] == -float("inf")).all()
    check(x[3:], [4], 3, (lp[3:], ent[3:], ids[3:], top[3:]))


def test_ids_out_of_range_are_recorded():
    x = logits(8, 4, 100, "bf16")
    lp, *_ = call(x, [100, -2, -1, 99], 0, status=m.MOE_ERR_BAD_INPUT)
    assert lp[:2].isnan().all() and lp[2] == 0 and lp[3].isfinite()


def test_far_logits():
    """e^d underflows for nearly all; large offsets cancel."""
    x = logits(9, 3, 5000, "fp32", std=100.0)
    x[1] += 1e6
    x[2] -= 3e4
    check(x, [1, 2, 3], 5)


def test_outputs_may_be_left_out():
    x = logits(10, 3, 4000, "bf16")
    full = call(x, [1, 2, 3], 5)
    assert torch.equal(call(x, [1, 2, 3], 5, parts=False)[0], full[0])
    shape = m.make_logprobs_shape(3, 4000, 5, "bf16")
    ids = torch.empty((3, 5), dtype=torch.int32, device=DEV)
    lp = torch.empty(3, device=DEV)
    m.moe_token_logprobs(shape, x, torch.tensor([1, 2, 3], dtype=torch.int32, device=DEV), lp,
                         m.alloc_logprobs_workspace(shape, DEV), top_ids=ids)
    assert torch.equal(ids, full[2]) and torch.equal(lp, full[0])


def test_one_workspace_every_shape_and_the_same_bits():
    work = [(logits(20 + i, n, V, d), [i % V] * n, k)
            for i, (n, V, d, k) in enumerate(((1, 200000, "bf16", 32), (300, 4000, "fp32", 5), (7, 70000, "fp16", 20),
                                              (64, 131072, "bf16", 20), (2, 5, "fp32", 0)))]
    ws = m.alloc_logprobs_workspace(m.make_logprobs_shape(1, 1), DEV)
    alone = [call(*w) for w in work]
    for i in (0, 1, 0, 2, 3, 2, 4, 3, 0, 1, 4, 2):
        for a, b in zip(call(*work[i], ws=ws), alone[i]):
            assert a is None or torch.equal(a, b)


def test_a_captured_call_takes_new_logits():
    shape = m.make_logprobs_shape(3, 50000, 5, "bf16")
    x, tok = logits(30, 3, 50000, "bf16"), torch.zeros(3, dtype=torch.int32, device=DEV)
    out = [torch.empty(3, device=DEV), torch.empty(3, device=DEV),
           torch.empty((3, 5), dtype=torch.int32, device=DEV), torch.empty((3, 5), device=DEV)]
    ws = m.alloc_logprobs_workspace(shape, DEV)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            m.moe_token_logprobs(shape, x, tok, out[0], ws, entropy=out[1], top_ids=out[2], top_logp=out[3])
    for seed in range(3):
        x.copy_(logits(40 + seed, 3, 50000, "bf16"))
        tok.fill_(seed + 9)
        graph.replay()
        torch.cuda.synchronize()
        check(x, [seed + 9] * 3, 5, out)


def test_rows_past_32_bits_of_bytes():
    n, V = 33000, 70000  # 4.6 GB
    x = torch.zeros((n, V), dtype=torch.bfloat16, device=DEV)
    some = [0, 1, n // 2, n - 1]
    x[some] = logits(50, 4, V, "bf16")
    lp, ent, ids, top = call(x, [3] * n, 4)
    check(x[some], [3] * 4, 4, (lp[some], ent[some], ids[some], top[some]))
    assert ids[2].tolist() == [0, 1, 2, 3]


@pytest.mark.parametrize("dtype,vec", [("bf16", 8), ("fp32", 4)])
@pytest.mark.parametrize("first,more", [(256, 0), (256, 1), (255, 1), (250, 40), (256, 300), (257, 5)])
@pytest.mark.parametrize("chunks", [2, 3])
@pytest.mark.parametrize("n", [3, 900])
def test_a_list_that_is_about_full(dtype, vec, first, more, chunks, n):
    # the first chunk (1024 vectors) brings as many as the list holds or nearly,
    # in all of the 64 groups of four threads that the bar comes from; what
    # follows overfills it
    chunk = 1024 * vec
    x = torch.full((n, chunks * chunk), -3.0)
    at = torch.arange(first)
    x[:, (at % 64) * 4 * vec + at // 64 % 4 * vec + at // 256] = 5.0
    for c in range(1, chunks):
        x[:, c * chunk + 7 * torch.arange(more)] = 5.0 + c
    x = x.to(TYPES[dtype]).to(DEV)
    tokens = [(i * 7919) % x.shape[1] for i in range(n)]
    if n <= 3:
        check(x, tokens, 32)
        return
    lp, ent, ids, top = call(x, tokens, 32)
    _, _, wids, _ = ref.logprobs(x[:1].cpu().double().numpy(), tokens[:1], 32)
    assert torch.equal(ids, torch.from_numpy(wids).to(ids).expand_as(ids))
    assert torch.equal(top, top[:1].expand_as(top)) and torch.equal(ent, ent[:1].expand_as(ent))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n,V", [(6, 9000), (6, 70001), (700, 9000)])
def test_masks_of_the_lowest_number(dtype, n, V):
    """Rows of which whole threads', warps' and stretches' shares are the
    type's lowest number, alone or beside -inf: it weighs nothing beside an
    ordinary logit, but it is listed, and alone it is a distribution."""
    low = torch.finfo(TYPES[dtype]).min
    x = logits(10, n, V, dtype)
    x[0, 100:] = low
    x[1, :] = low
    x[2, :], x[2, 1::2] = low, -float("inf")
    x[3, :], x[3, V - 1] = low, -3.0
    x[4, :V // 2], x[4, V // 2:] = -float("inf"), low
    x[5, :-5] = low
    tokens = [(i * 7919) % V for i in range(n)]
    got = call(x, tokens, 8)
    check(x[:6], tokens[:6], 8, [y[:6] for y in got])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,V", [(6, 70001), (640, 20000)])
def test_rows_whose_large_numbers_lie_together(dtype, n, V):
    """Sorted and smooth rows, cut and uncut: the list is overfilled early, late
    or throughout."""
    g = torch.Generator().manual_seed(12)
    r = torch.randn(V, generator=g)
    at = torch.arange(V) / 900.0
    rows = [torch.sort(r)[0], torch.sort(r, descending=True)[0], torch.sin(at), torch.sin(at) * torch.cos(7 * at),
            torch.floor(at), torch.where(at > at[-1] / 2, torch.floor(at) % 3, torch.zeros(()))]
    x = torch.stack([rows[i % 6] for i in range(n)]).to(TYPES[dtype]).to(DEV)
    tokens = [(i * 7919) % V for i in range(n)]
    for k in (1, 20, 32):
        got = call(x, tokens, k)
        check(x[:6], tokens[:6], k, [y[:6] for y in got])
        assert all(torch.equal(y[6:12], y[:6]) for y in got[1:] if n > 12)
