"""The serving example over a cache in 4 bits, and its answers' log
probabilities: pages taken, forked, copied on write and cut as 4-bit pools, rows
quantised as they are written, attention over the codes.

With temperature 0 every token has to be the likeliest one when the text is read
one token at a time through a 4-bit cache, too. The two ways quantise rows of
activations that differ by roundings (some 2^-8 of unit scale), and a code that
falls to another side moves a value by a step, a fifteenth of its group's range
(some 0.3), for one element in a hundred or so: beside the 0.03 of 16-bit
activations a logit is uncertain by some 0.3 / sqrt(100) on top. A token counts
as the likeliest within 0.25; as in the 16-bit test, routing can differ where
two experts are that close, and nine in ten have to be right."""
import os
import sys

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    import __graft_entry__
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import speculative_serving
    speculative_serving.m.load()
    return speculative_serving


@pytest.mark.parametrize("prompt,requests,drafts", [(300, 5, 3), (65, 2, 1), (20, 3, 7), (130, 4, 0)])
def test_decoding_over_4_bits(example, prompt, requests, drafts):
    model = example.Model(seed=prompt)
    tokens = np.random.default_rng(prompt).integers(0, example.VOCAB, prompt).tolist()
    logps = []
    got, steps, held = example.decode(model, tokens, requests, 40, drafts, bits=4, logps=logps)
    assert steps <= 40 and all(r == got[0] for r in got)
    gaps = example.shortfall(model, tokens, got[0], bits=4)
    assert len(gaps) == 40 and sum(x <= 0.25 for x in gaps) >= 36, gaps
    shared = (prompt - 1) // 64
    own = -(-(prompt + 40 + drafts) // 64) - shared
    assert held <= shared + requests * own
    # the likeliest of 512 has at least a 512th
    assert all(len(s) == 40 and all(-np.log(512) - 1e-4 <= x <= 0 for x in s) for s in logps)


def test_log_probabilities_of_the_16_bit_answers(example):
    """Against the logits of the text read one token at a time."""
    model = example.Model(seed=3)
    tokens = np.random.default_rng(3).integers(0, example.VOCAB, 90).tolist()
    logps = []
    got, _, _ = example.decode(model, tokens, 2, 20, 2, logps=logps)
    ints = lambda a: torch.tensor(a, dtype=torch.int32, device=model.dev)  # noqa: E731
    text = tokens + got[0]
    server = example.Server(model, 1, len(text), -(-len(text) // 64) + 1)
    want = []
    for i, t in enumerate(text[:-1]):
        logits = server.step(ints([[t]]), ints([1]))[0, 0].double()
        if i >= len(tokens) - 1:
            want.append(float(torch.log_softmax(logits, -1)[text[i + 1]]))
    # logits differ by some 0.03 (the 16-bit test's reckoning) but for a routing
    # that differs, once in ten
    near = [abs(a - b) <= 0.25 for a, b in zip(logps[0], want)]
    assert len(near) == 20 and sum(near) >= 18, list(zip(logps[0], want))
