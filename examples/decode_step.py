#!/usr/bin/env python3
"""A small decoder around the activation-sparse layer: prompts, then tokens one
by one, then the gradient of their log probabilities.

Every step runs, on the current stream and without a synchronisation,

    twell_kv_plan       which cache pages the step's tokens go to
    twell_block_norm    the first norm
    per layer:  projections (torch), twell_kv_append, twell_kv_attention,
                output projection (torch), twell_block_norm (residual sum and next norm),
                twell_ffn_fwd (the sparse layer), twell_block_norm
    twell_logprobs      log probability, entropy and best alternatives of the answer

for requests of different lengths in one batch: their prompts in the first step,
one token each afterwards, a finished request giving its pages back on the
way.  Weights are random: what comes out means nothing, but a token's log
probabilities must not depend on how the steps were cut, and that is checked.

    python examples/decode_step.py
"""
from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import activation_sparse_transformer_gb300 as tw

D_MODEL, D_FF, LAYERS, Q_HEADS, KV_HEADS, HEAD_DIM, VOCAB = 512, 2048, 2, 8, 2, 64, 1000
TILE, CAP, PAGE = 64, 8, 16
EPS = torch.finfo(torch.float32).eps  # of the norms, as torch's rms_norm of fp32 rows has it


class Decoder:
    """Weights, caches and the buffers that live from step to step."""

    def __init__(self, max_requests: int, max_len: int, fmt=tw.KV_E4M3, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: (torch.randn(s, generator=g, device="cuda") * s[-1] ** -0.5).bfloat16()  # noqa: E731
        self.embed, self.unembed = 8 * rand(VOCAB, D_MODEL), 4 * rand(VOCAB, D_MODEL)
        width = (Q_HEADS + 2 * KV_HEADS) * HEAD_DIM
        self.layers = [dict(qkv=rand(width, D_MODEL), out=rand(D_MODEL, Q_HEADS * HEAD_DIM), w_in=rand(D_FF, D_MODEL),
                            # a bias that leaves about one unit in twenty active
                            b=torch.full((D_FF,), -1.65, device="cuda").bfloat16(), w_down=rand(D_FF, D_MODEL))
                       for _ in range(LAYERS)]
        blocks = -(-max_len // PAGE)
        n_pages = max_requests * blocks
        self.caches = [tw.alloc_kv_cache(n_pages, PAGE, KV_HEADS, HEAD_DIM, fmt) for _ in range(LAYERS)]
        self.ring, self.pool = tw.alloc_page_ring(n_pages)
        self.table = torch.zeros((max_requests, blocks), dtype=torch.int32, device="cuda")
        self.lens = torch.zeros((max_requests,), dtype=torch.int32, device="cuda")
        self.norm = torch.ones(D_MODEL, device="cuda").bfloat16()
        self.max_len = max_len

    def ffn(self, x, layer):
        n = x.shape[0]
        h = tw.alloc_packed(n, D_FF, TILE, CAP, n)
        ws = torch.empty(tw.fwd_workspace_bytes(n, D_MODEL, D_FF, TILE, CAP, n), dtype=torch.uint8, device="cuda")
        y = torch.empty_like(x)
        tw.twell_ffn_fwd(x, layer["w_in"], layer["b"], layer["w_down"], h, y, ws)
        return y

    def step(self, tokens, new, max_new: int):
        """One step: `tokens` of all requests in order, new[r] of each (-1: request
        r is finished).  Returns the logits of every token and the step's plan."""
        n, requests = tokens.numel(), self.lens.numel()
        plan = tw.alloc_kv_plan(requests, n)
        tw.twell_kv_plan(self.lens, new, self.table, self.ring, self.pool, PAGE, plan)
        x = self.embed[tokens]
        hidden = torch.empty_like(x)
        tw.twell_block_norm(x, None, None, hidden, w_pre=self.norm, eps=EPS)
        o = torch.empty((n, Q_HEADS, HEAD_DIM), dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(tw.kv_attention_workspace_bytes(n, requests, Q_HEADS, KV_HEADS, HEAD_DIM), dtype=torch.uint8,
                         device="cuda")
        for layer, cache in zip(self.layers, self.caches):
            qkv = (hidden @ layer["qkv"].T).view(n, Q_HEADS + 2 * KV_HEADS, HEAD_DIM)
            q, k, v = qkv.split((Q_HEADS, KV_HEADS, KV_HEADS), 1)
            tw.twell_kv_append(k, v, plan.cu_q, plan.slots, cache)
            tw.twell_kv_attention(q, cache, self.table, plan.cu_q, plan.positions, plan.kv_lens, self.max_len,
                                  max_new, HEAD_DIM ** -0.5, o, ws)
            tw.twell_block_norm(x, o.view(n, -1) @ layer["out"].T, x, hidden, w_pre=self.norm, eps=EPS)
            tw.twell_block_norm(x, self.ffn(hidden, layer), x, hidden, w_pre=self.norm, eps=EPS)
        self.lens, self.pool = plan.kv_lens, plan.pool
        return hidden @ self.unembed.T, hidden, plan

    def status(self) -> list:
        return [tw.twell_kv_read_status(c) for c in self.caches]


def answer(logits, targets, top: int):
    """(log probabilities of targets, entropy, lse, best log probabilities, their tokens)"""
    n = logits.shape[0]
    f = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
    out = None if targets is None else f(n), f(n), f(n), f(n, top), torch.empty((n, top), dtype=torch.int32, device="cuda")
    tw.twell_logprobs(logits, targets, 1.0, *out)
    return out


def run(prompt_lens=(37, 5, 130, 64), steps: int = 12, fmt=tw.KV_E4M3) -> dict:
    g = torch.Generator(device="cuda").manual_seed(1)
    requests, longest = len(prompt_lens), max(prompt_lens)
    prompts = [torch.randint(VOCAB, (n,), generator=g, device="cuda") for n in prompt_lens]
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731

    # the prompts in one step, then greedy tokens one by one; the second request ends half way
    model = Decoder(requests, longest + steps + 1, fmt)
    logits, _, plan = model.step(torch.cat(prompts), i32(prompt_lens), longest)
    last = plan.cu_q[1:].long() - 1
    texts, scores = [list(p.tolist()) for p in prompts], [[] for _ in prompts]
    live = list(range(requests))
    for step in range(steps):
        _, _, _, best, token = answer(logits[last].contiguous(), None, 1)
        for row, r in enumerate(live):
            texts[r].append(int(token[row, 0]))
            scores[r].append(float(best[row, 0]))
        new = [1 if r in live else 0 for r in range(requests)]
        if step == steps // 2 and requests > 1:
            live.remove(1)
            new[1] = -1
        logits, _, plan = model.step(torch.tensor([texts[r][-1] for r in live], device="cuda"), i32(new), 1)
        last = torch.arange(len(live), device="cuda")
    assert model.status() == [0] * LAYERS

    # the same sequences in one step each: the same log probabilities, up to the
    # cache's scales (a page written token by token may have moved to a larger one)
    again = Decoder(requests, longest + steps + 1, fmt)
    lens = [len(t) - 1 for t in texts]
    logits, hidden, plan = again.step(torch.tensor([t for x in texts for t in x[:-1]], device="cuda"), i32(lens),
                                      max(lens))
    targets = i32([t for x in texts for t in x[1:]])
    logprob, entropy, lse, _, _ = answer(logits, targets, 1)
    first, off = 0, 0.0
    for r, n in enumerate(lens):
        mine = logprob[first + prompt_lens[r] - 1:first + n].tolist()
        off = max([off] + [abs(a - b) for a, b in zip(mine, scores[r])])
        first += n

    # one policy-gradient step's gradient: the answers' tokens weighted alike, a little entropy
    weight = torch.cat([torch.cat([torch.zeros(p - 1), torch.ones(n - p + 1)]) for p, n in zip(prompt_lens, lens)])
    weight = -(weight / weight.sum()).cuda()
    d_logits = torch.empty_like(logits)
    tw.twell_logprobs_bwd(logits, targets, 1.0, lse, entropy, weight, -0.01 * weight.abs(), d_logits)
    d_unembed = d_logits.T @ hidden
    return dict(texts=texts, scores=scores, off=off, entropy=float(entropy.mean()), d_unembed=d_unembed,
                d_logits=d_logits, free=int(model.pool[1]), pages=model.ring.numel(), lens=model.lens.tolist())


if __name__ == "__main__":
    out = run()
    for text, score in zip(out["texts"], out["scores"]):
        print(f"{len(text):4d} tokens, the answer's log probability {sum(score):8.2f}: {text[-len(score):]}")
    print(f"token by token against one step: log probabilities within {out['off']:.3f}; mean entropy "
          f"{out['entropy']:.2f}; gradient of the output weights {out['d_unembed'].float().norm():.4f}")
