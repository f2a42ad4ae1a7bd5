"""A batch of requests over one page pool, decoded with drafted tokens.

    python examples/speculative_serving.py [--requests 8] [--new 48] [--temperature 0.0] [--cache 4]

One prompt is read once into a slot's pages and forked to every request
(moe_cache_fork), so its pages are shared; each step then takes room for the
current token and its drafts (moe_cache_reserve), runs the layers (keys and
values into their pages with moe_cache_write, moe_attn_batch with the prompt's
whole pages as the shared prefix, the MoE layer with moe_layer_w4), checks the
drafts against the model's probabilities (moe_verify_drafts) and gives the
rejected tail back (moe_cache_fork with `keep`). The model is a small
random-weight one: 2 layers of 8 query heads on 2 key/value heads of 64, 16
experts. Drafts are what followed the current token the last time it came up.
With --cache 4 keys and values are held in 4 bits: the same steps with
moe_cache_write_q4 and moe_attn_batch_q4, where the prompt's pages are shared
through the slots' tables. The answers' log probabilities come from
moe_token_logprobs.

With temperature 0 the probabilities are one-hot, and every token has to be the
likeliest one when the same text is read one token at a time (up to the
roundings of 16-bit activations, which depend on how many tokens go through a
layer at once); main() prints how far they are from that.
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bit_moe_expert_histogram_gb300 as m  # noqa: E402
import synth  # noqa: E402

BLOCK = 64
N_Q, N_KV, D, LAYERS, VOCAB = 8, 2, 64, 2, 512


class Model:
    """Random weights and one layer call for N tokens."""

    def __init__(self, seed=0, dev="cuda"):
        self.dev = torch.device(dev)
        g = torch.Generator().manual_seed(seed)
        w = synth.CONFIGS["tiny"]
        self.S, H = w.shape, w.shape.H
        rnd = lambda *s: (torch.randn(s, generator=g) / s[0] ** 0.5).to(torch.bfloat16).to(dev)  # noqa: E731
        self.embed = torch.randn((VOCAB, H), generator=g).to(torch.bfloat16).to(dev)
        self.qkv = [rnd(H, (N_Q + 2 * N_KV) * D) for _ in range(LAYERS)]
        self.out = [rnd(N_Q * D, H) for _ in range(LAYERS)]
        self.head = rnd(H, VOCAB)
        self.moe = []
        for layer in range(LAYERS):
            L = synth.gen_layer(1, self.S, seed=seed + layer)
            router = torch.from_numpy(np.ascontiguousarray(L.w_router).view(np.int16)).to(dev)
            self.moe.append((router, m.ExpertWeights.from_numpy(
                L.q_gate_up, L.s_gate_up, L.b_gate_up, L.q_down, L.s_down, L.b_down, dev),
                m.ExpertWeights.from_numpy(L.sh_q_gate_up, L.sh_s_gate_up, L.sh_b_gate_up,
                                           L.sh_q_down, L.sh_s_down, L.sh_b_down, dev)))
        self.ws = {}

    @staticmethod
    def norm(x):
        x = x.float()
        return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)

    def experts(self, layer, x):
        n, s = x.shape[0], self.S
        if n not in self.ws:
            shape = m.make_shape(n, s.H, s.E, s.K, s.I, s.n_shared, 128)
            self.ws[n] = (shape, m.alloc_workspace(shape, self.dev))
        shape, ws = self.ws[n]
        router, ex, sh = self.moe[layer]
        y = torch.empty_like(x)
        m.moe_layer_w4(shape, x, router, None, ex, sh, y, ws)
        # 4-bit test weights are large: the layer's output comes at unit scale
        return self.norm(y)


class Server:
    """Slots, their pages and the calls of a step."""

    def __init__(self, model, n_slots, max_len, n_phys, bits=16):
        self.model, self.B, dev = model, n_slots, model.dev
        self.bits = bits
        self.width = -(-max_len // BLOCK)
        self.shape = m.make_cache_shape(n_slots, self.width, n_phys, N_KV, D)
        # what the page calls move: pages of 16-bit rows, or of 4-bit ones
        self.page_shape = m.q4_page_shape(self.shape) if bits == 4 else self.shape
        self.cache_ws = m.alloc_cache_workspace(self.shape, dev)
        self.meta, self.spare = m.CacheMeta.empty(self.shape, dev), m.CacheMeta.empty(self.shape, dev)
        if bits == 4:
            pool = lambda: m.alloc_q4_pool(self.shape, dev)  # noqa: E731
        else:
            pool = lambda: torch.empty((n_phys, N_KV, BLOCK, D), dtype=torch.bfloat16, device=dev)  # noqa: E731
        self.k, self.v = [pool() for _ in range(LAYERS)], [pool() for _ in range(LAYERS)]
        self.pools = m.pool_table(self.k + self.v)
        self.granted = torch.empty(n_slots, dtype=torch.int32, device=dev)
        self.attn = {}
        self.prefix = None

    def fork(self, parent, keep=None):
        m.moe_cache_fork(self.page_shape, self.meta, parent, self.spare, self.cache_ws, keep=keep)
        self.meta, self.spare = self.spare, self.meta

    def share_prefix(self, slot, blocks):
        """The first `blocks` pages of `slot` are every slot's from here on."""
        if self.bits == 16:
            self.prefix = self.meta.table[slot, :blocks].clone() if blocks else None

    def step(self, tokens, n_new):
        """tokens int32 [B][T], n_new int32 [B]: their logits [B][T][VOCAB]."""
        B, T = tokens.shape
        m.moe_cache_reserve(self.page_shape, self.meta, n_new, self.spare, self.granted, self.pools,
                            self.cache_ws)
        self.meta, self.spare = self.spare, self.meta
        P = 0 if self.prefix is None else len(self.prefix)
        if (T, P) not in self.attn:
            shape = m.make_attn_batch_shape(B, T, N_Q, N_KV, D, self.width, P)
            alloc = m.alloc_attn_batch_q4_workspace if self.bits == 4 else m.alloc_attn_batch_workspace
            self.attn[T, P] = (shape, alloc(shape, self.model.dev),
                               torch.empty((B, T, N_Q, D), dtype=torch.bfloat16,
                                           device=self.model.dev))
        shape, ws, o = self.attn[T, P]
        x = self.model.embed[tokens.long()].view(B * T, -1)
        for layer in range(LAYERS):
            qkv = (self.model.norm(x) @ self.model.qkv[layer]).view(B, T, N_Q + 2 * N_KV, D)
            q, k, v = qkv[:, :, :N_Q], qkv[:, :, N_Q:N_Q + N_KV], qkv[:, :, N_Q + N_KV:]
            pools = self.k[layer], self.v[layer]
            if self.bits == 4:
                m.moe_cache_write_q4(self.shape, self.meta, self.granted, k, v, *pools, self.cache_ws)
                m.moe_attn_batch_q4(shape, q, *pools, self.meta.table, self.meta.lens, o, ws,
                                    n_new=self.granted)
            else:
                m.moe_cache_write(self.shape, self.meta, self.granted, k, v, *pools, self.cache_ws)
                m.moe_attn_batch(shape, q, *pools, self.meta.table, self.meta.lens, o, ws,
                                 n_new=self.granted, prefix=self.prefix)
            x = x + o.view(B * T, -1) @ self.model.out[layer]
            x = x + self.model.experts(layer, self.model.norm(x))
        return (self.model.norm(x) @ self.model.head).float().view(B, T, VOCAB)


def probabilities(logits, temperature):
    if temperature > 0:
        return torch.softmax(logits / temperature, -1)
    return torch.nn.functional.one_hot(logits.argmax(-1), VOCAB).float()


def look_up(history, n):
    """What followed the last token of `history` the last time it came up."""
    for i in range(len(history) - 2, -1, -1):
        if history[i] == history[-1]:
            return history[i + 1:i + 1 + n]
    return []


def decode(model, prompt, requests, new, drafts, temperature=0.0, seed=0, bits=16, logps=None):
    """Token lists of every request, how many steps they took and how many pages
    were held. logps: a list that takes the tokens' log probabilities (of the
    model as it is, whatever the temperature), a list a request."""
    dev = model.dev
    max_len = len(prompt) + new + drafts + BLOCK
    per_slot = -(-(new + drafts + BLOCK) // BLOCK) + 1
    server = Server(model, requests, max_len, -(-len(prompt) // BLOCK) + requests * per_slot, bits)
    ints = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731
    # the prompt, sixteen tokens at a time, into slot 0; its last token starts
    # every request
    for i in range(0, len(prompt) - 1, 16):
        part = prompt[i:min(i + 16, len(prompt) - 1)]
        tokens = torch.zeros((requests, 16), dtype=torch.int32, device=dev)
        tokens[0, :len(part)] = ints(part)
        server.step(tokens, ints([len(part)] + [0] * (requests - 1)))
    server.fork(ints([0] * requests))
    server.share_prefix(0, (len(prompt) - 1) // BLOCK)
    T = drafts + 1
    shape = m.make_verify_shape(requests, max(drafts, 1), VOCAB)
    ws = m.alloc_verify_workspace(shape, dev)
    out = torch.empty((requests, max(drafts, 1) + 1), dtype=torch.int32, device=dev)
    n_acc = torch.empty(requests, dtype=torch.int32, device=dev)
    everyone = ints(list(range(requests)))
    g = torch.Generator(device=dev).manual_seed(seed)
    history = [list(prompt) for _ in range(requests)]
    lshape = m.make_logprobs_shape(requests * T, VOCAB)
    lws, logp = m.alloc_logprobs_workspace(lshape, dev), torch.empty(requests * T, device=dev)
    said = [[] for _ in range(requests)]
    steps = 0
    while min(len(h) for h in history) < len(prompt) + new:
        tokens = torch.zeros((requests, T), dtype=torch.int32, device=dev)
        draft = torch.zeros((requests, max(drafts, 1)), dtype=torch.int32, device=dev)
        counts = []
        for b, h in enumerate(history):
            d = look_up(h, drafts) if len(h) < len(prompt) + new else []
            counts.append(len(d))
            tokens[b, :1 + len(d)] = ints([h[-1]] + d)
            if d:
                draft[b, :len(d)] = ints(d)
        n_draft = ints(counts)
        lens = server.meta.lens.clone()
        logits = server.step(tokens, n_draft + 1)
        p = probabilities(logits, temperature)
        if drafts == 0:  # verification wants room for one draft
            p = torch.cat([p, p], 1).contiguous()
        u = torch.rand(out.shape, generator=g, device=dev)
        m.moe_verify_drafts(shape, p, None, draft, n_draft, u, out, n_acc, ws)
        server.fork(everyone, keep=lens + 1 + n_acc)  # what was rejected goes back
        steps += 1
        # row t of a request's logits is what its t-th token here was drawn from
        m.moe_token_logprobs(lshape, logits.view(requests * T, VOCAB), out[:, :T].contiguous().view(-1),
                             logp, lws)
        for h, s, row, lp in zip(history, said, out.tolist(), logp.view(requests, T).tolist()):
            h += [t for t in row if t >= 0]
            s += [x for x, t in zip(lp, row) if t >= 0]
    for w in (server.cache_ws, ws, lws, *[a[1] for a in server.attn.values()]):
        status = m.moe_query_device_status(w)
        if status != 0:
            raise RuntimeError("device status %d" % status)
    if logps is not None:
        logps += [s[:new] for s in said]
    held = int((server.meta.refs > 0).sum())
    return [h[len(prompt):len(prompt) + new] for h in history], steps, held


def shortfall(model, prompt, text, bits=16):
    """For every token of `text` after `prompt`, read one token at a time: the
    largest logit less the token's own."""
    ints = lambda a: torch.tensor(a, dtype=torch.int32, device=model.dev)  # noqa: E731
    tokens = list(prompt) + list(text)
    server = Server(model, 1, len(tokens), -(-len(tokens) // BLOCK) + 1, bits)
    gaps = []
    for i, t in enumerate(tokens[:-1]):
        logits = server.step(ints([[t]]), ints([1]))[0, 0]
        if i >= len(prompt) - 1:
            gaps.append(logits.max() - logits[tokens[i + 1]])
    return torch.stack(gaps).tolist()


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--new", type=int, default=48)
    ap.add_argument("--drafts", type=int, default=3)
    ap.add_argument("--prompt", type=int, default=300)
    ap.add_argument("--temperature", type=float, default=0.0)
    ap.add_argument("--cache", type=int, choices=(16, 4), default=16, help="bits of keys and values")
    args = ap.parse_args()
    m.load()
    model = Model()
    prompt = np.random.default_rng(0).integers(0, VOCAB, args.prompt).tolist()
    logps = []
    got, steps, held = decode(model, prompt, args.requests, args.new, args.drafts, args.temperature,
                              bits=args.cache, logps=logps)
    print("%d requests x %d tokens in %d steps, %d pages held, %.2f nats a token" % (
        args.requests, args.new, steps, held, -np.mean(logps)))
    if args.temperature == 0:
        gaps = shortfall(model, prompt, got[0], args.cache)
        print("read one at a time: %d of %d tokens the likeliest, the others short by up to %.3f" % (
            sum(x <= 0 for x in gaps), len(gaps), max(gaps)))


if __name__ == "__main__":
    main()
