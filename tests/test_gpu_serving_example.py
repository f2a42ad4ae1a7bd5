"""The serving example end to end: the calls of a batch's step together
(pages, attention under a shared prompt, MoE layer, verification).

With temperature 0 every drafted token has to be the likeliest one when the
text is read one token at a time. The two ways round 16-bit activations
differently: about ten roundings of 2^-9 on a residual of unit scale give a
logit (unit scale, 512 of them) an uncertainty of some 0.03, so a token counts
as the likeliest within 0.125. Where two experts' router logits are that close
the routing itself can differ (a few tokens in a hundred for two layers of 2
of 16 experts) and with it the logits: nine tokens in ten have to be right."""
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


@pytest.mark.parametrize("prompt,requests,drafts", [(300, 5, 3), (65, 2, 1), (20, 3, 7)])
def test_drafted_tokens_are_the_likeliest(example, prompt, requests, drafts):
    model = example.Model(seed=prompt)
    tokens = np.random.default_rng(prompt).integers(0, example.VOCAB, prompt).tolist()
    got, steps, held = example.decode(model, tokens, requests, 40, drafts)
    assert steps <= 40 and all(r == got[0] for r in got)
    gaps = example.shortfall(model, tokens, got[0])
    assert len(gaps) == 40 and sum(x <= 0.125 for x in gaps) >= 36, gaps
    # the prompt's whole pages once, and each request's own
    shared = (prompt - 1) // 64
    own = -(-(prompt + 40 + drafts) // 64) - shared
    assert held <= shared + requests * own


def test_sampled_decoding_runs(example):
    model = example.Model(seed=1)
    tokens = np.random.default_rng(1).integers(0, example.VOCAB, 130).tolist()
    got, _, _ = example.decode(model, tokens, 4, 20, 2, temperature=1.0)
    assert all(len(r) == 20 and all(0 <= t < example.VOCAB for t in r) for r in got)
    assert len({tuple(r) for r in got}) > 1
