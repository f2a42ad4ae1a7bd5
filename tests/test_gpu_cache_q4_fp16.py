"""4-bit rows read back as fp16: s c + b rounded once, to the nearest fp16 number,
ties to even. Rows are packed as they are wanted: twelve-bit products s c that
are ties of fp16 beside biases too small for fp32 to see next to them, products
that all but cancel their bias, results among fp16's subnormal numbers and past
its largest. The wanted numbers are exact in 64 bits (a product of twelve bits
and a bias of eight, less than 40 binary places apart), which numpy rounds once."""
import numpy as np
import pytest
import torch

import bit_moe_expert_histogram_gb300 as m
import q4_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    m.load()


def scales_and_biases():
    """[groups] each, bf16 numbers."""
    s, b = [], []
    for top in range(128, 256):  # all significands
        for sign in (1.0, -1.0):
            for place in (-40, -30, -26, -24, -21, -18, 0, 8):
                s.append(top / 128.0)
                b.append(sign * (1 + top % 128 / 128.0) * 2.0**place)
    rng = np.random.default_rng(0)
    for _ in range(4096):
        e = rng.integers(-30, 14)
        s.append((1 + rng.integers(128) / 128) * 2.0**e)
        b.append(rng.choice([1, -1]) * (1 + rng.integers(128) / 128) * 2.0**(e + rng.integers(-27, 28)))
    for c in range(1, 16):  # s c + b = 0 exactly
        s.append(1.25)
        b.append(-1.25 * c)
    s += [0.0, 0.0, 4096.0, 4368.0, 4368.0]  # the last: up to 65520, a tie with infinity
    b += [-0.0, 2.0**-25, 0.0, 0.0, -2.0**-20]
    while len(s) % 4:
        s.append(1.0)
        b.append(0.0)
    return np.array(s), np.array(b)


@pytest.mark.parametrize("D", [64, 128])
def test_fp16_rows_are_rounded_once(D):
    s, b = scales_and_biases()
    n = len(s) // 4
    s, b = s.reshape(n, 4), b.reshape(n, 4)
    code = np.tile(np.arange(16, dtype=np.uint8), D // 16)
    rows = ref.pack(np.broadcast_to(code, (n, D)), s, b)
    want = ref.values(rows, D)
    blocks = -(-n // 64)
    shape = m.make_cache_shape(1, blocks, blocks, 1, D)
    k, v = m.alloc_q4_pool(shape, DEV), m.alloc_q4_pool(shape, DEV)
    for pool, r in ((k, rows), (v, rows[::-1])):
        pool.view(-1, pool.shape[-1])[:n] = torch.from_numpy(r.copy()).to(DEV)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    meta = m.CacheMeta(ints([list(range(blocks))]), ints([n]), ints([1] * blocks))
    ws = m.alloc_cache_workspace(shape, DEV)
    out = [torch.full((1, n, 1, D), 7.0, dtype=torch.float16, device=DEV) for _ in range(2)]
    m.moe_cache_read_q4(shape, meta, None, None, k, v, *out, ws)
    assert m.moe_query_device_status(ws) == 0
    with np.errstate(over="ignore"):
        want = want.astype(np.float16)
    for got, w in zip(out, (want, want[::-1])):
        got = got.cpu().numpy().reshape(n, D)
        bad = np.argwhere(got.view(np.uint16) != w.view(np.uint16))
        assert len(bad) == 0, (len(bad), [(got[tuple(i)], w[tuple(i)]) for i in bad[:4]])
