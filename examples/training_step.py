#!/usr/bin/env python3
"""A training step around the activation-sparse layer: a stack of blocks, from the tokens' embeddings to
the log probabilities of the next ones and back to every weight's gradient.

Forward, on the current stream and without a synchronisation:

    twell_block_norm       the first norm
    per block:  twell_ffn_fwd (the sparse layer), twell_block_norm (norm behind it, gate, residual
                sum, norm before the next block)
    twell_linear_logprobs  log probabilities and entropies of the targets; no logits in memory

and backward the gradients of the same calls in reverse order:

    twell_linear_logprobs_bwd;  per block twell_block_norm_bwd, twell_ffn_bwd;  twell_block_norm_bwd

    python examples/training_step.py
"""
from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import activation_sparse_transformer_gb300 as tw

D_MODEL, D_FF, BLOCKS, VOCAB, TILE, CAP = 512, 2048, 2, 1000, 64, 8
EPS, BRANCH_SCALE = 1e-6, (2 * BLOCKS) ** -0.5


class Model:
    """Weights, and the buffers that live from step to step."""

    def __init__(self, n_tokens: int, stream=torch.float32, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: (torch.randn(s, generator=g, device="cuda") * s[-1] ** -0.5).bfloat16()  # noqa: E731
        near_one = lambda: (1 + 0.1 * torch.randn(D_MODEL, generator=g, device="cuda")).bfloat16()  # noqa: E731
        self.embed, self.unembed = 8 * rand(VOCAB, D_MODEL), 3 * rand(VOCAB, D_MODEL)
        self.norm = [near_one() for _ in range(BLOCKS + 1)]  # before each block, and the last one
        self.blocks = [dict(w_in=rand(D_FF, D_MODEL),
                            # a bias that leaves about one unit in twenty active
                            b=torch.full((D_FF,), -1.65, device="cuda").bfloat16(), w_down=rand(D_FF, D_MODEL),
                            post=near_one(), gate=near_one()) for _ in range(BLOCKS)]
        self.n, self.stream = n_tokens, stream
        new = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
        rows = lambda dtype=torch.bfloat16: new(n_tokens, D_MODEL, dtype=dtype)  # noqa: E731
        self.x = [rows(stream) for _ in range(BLOCKS + 1)]   # the residual stream before each block, and behind the last
        self.h = [rows() for _ in range(BLOCKS + 1)]         # its norms
        self.y = [rows() for _ in range(BLOCKS)]             # the blocks' outputs
        self.rstd = [new(n_tokens) for _ in range(BLOCKS + 1)]
        self.rstd_post = [new(n_tokens) for _ in range(BLOCKS)]
        self.packed = [tw.alloc_packed(n_tokens, D_FF, TILE, CAP, n_tokens) for _ in range(BLOCKS)]
        self.logprob, self.entropy, self.lse = (new(n_tokens) for _ in range(3))
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        shape = (n_tokens, D_MODEL, D_FF, TILE, CAP, n_tokens)
        self.workspace = new(max(tw.fwd_workspace_bytes(*shape), tw.bwd_workspace_bytes(*shape),
                                 tw.block_norm_bwd_workspace_bytes(n_tokens, D_MODEL),
                                 tw.linear_logprobs_workspace_bytes(n_tokens, D_MODEL, VOCAB),
                                 tw.linear_logprobs_bwd_workspace_bytes(n_tokens, D_MODEL, VOCAB)), dtype=torch.uint8)

    def forward(self, tokens, targets):
        """Log probabilities of targets and entropies; what the backward pass needs stays in the buffers."""
        self.x[0].copy_(self.embed[tokens])
        tw.twell_block_norm(self.x[0], None, None, self.h[0], w_pre=self.norm[0], eps=EPS, rstd_pre=self.rstd[0])
        for i, w in enumerate(self.blocks):
            tw.twell_ffn_fwd(self.h[i], w["w_in"], w["b"], w["w_down"], self.packed[i], self.y[i], self.workspace)
            tw.twell_block_norm(self.x[i], self.y[i], self.x[i + 1], self.h[i + 1], w_post=w["post"], gate=w["gate"],
                                w_pre=self.norm[i + 1], branch_scale=BRANCH_SCALE, eps=EPS,
                                rstd_post=self.rstd_post[i], rstd_pre=self.rstd[i + 1])
        tw.twell_linear_logprobs(self.h[-1], self.unembed, targets, 1.0, self.logprob, self.entropy, self.lse,
                                 self.workspace, self.status)
        return self.logprob, self.entropy

    def backward(self, tokens, targets, d_logprob, d_entropy) -> dict:
        """Gradients of sum(d_logprob logprob + d_entropy entropy) by the weights' names."""
        f32 = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
        grads = {"unembed": torch.empty_like(self.unembed)}
        d_h = torch.empty_like(self.h[-1])
        tw.twell_linear_logprobs_bwd(self.h[-1], self.unembed, targets, 1.0, self.lse, self.entropy, d_logprob,
                                     d_entropy, d_h, grads["unembed"], self.workspace, self.status)
        d_x = None  # the last norm is all that reads the stream behind the last block
        for i in reversed(range(BLOCKS)):
            w, g = self.blocks[i], {k: f32(D_MODEL) for k in ("post", "gate")}
            norm = f32(D_MODEL)
            d_before, d_y = torch.empty_like(self.x[i]), torch.empty_like(self.y[i])
            tw.twell_block_norm_bwd(d_h, d_x, self.x[i + 1], self.y[i], d_before, d_y, w_post=w["post"], gate=w["gate"],
                                    w_pre=self.norm[i + 1], branch_scale=BRANCH_SCALE, rstd_post=self.rstd_post[i],
                                    rstd_pre=self.rstd[i + 1], dw_post=g["post"], dgate=g["gate"], dw_pre=norm,
                                    workspace=self.workspace)
            d_x, d_h = d_before, torch.empty_like(d_h)
            g.update(w_in=f32(D_FF, D_MODEL), w_down=f32(D_FF, D_MODEL), b=f32(D_FF))
            tw.twell_ffn_bwd(self.h[i], w["w_in"], w["w_down"], self.packed[i], d_y, 0.0, d_h, g["w_in"], g["w_down"],
                             g["b"], self.workspace)
            grads.update({f"{k}{i}": t for k, t in g.items()})
            grads[f"norm{i + 1}"] = norm
        grads["norm0"] = f32(D_MODEL)
        tw.twell_block_norm_bwd(d_h, d_x, self.x[0], None, d_x, None, w_pre=self.norm[0], rstd_pre=self.rstd[0],
                                dw_pre=grads["norm0"], workspace=self.workspace)
        grads["embed"] = torch.zeros(VOCAB, D_MODEL, device="cuda").index_add_(0, tokens, d_x.float())
        return grads

    def ok(self) -> bool:
        return int(self.status) == 0 and all(tw.twell_read_status(p) == 0 for p in self.packed)


def batch(n_tokens: int, seed: int = 1):
    """Tokens, the next ones (the last has none) and the weight of each log probability."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    tokens = torch.randint(VOCAB, (n_tokens,), generator=g, device="cuda")
    targets = torch.roll(tokens, -1).to(torch.int32)
    targets[-1] = -1
    return tokens, targets, torch.full((n_tokens,), -1.0 / n_tokens, device="cuda")


def run(n_tokens: int = 300, stream=torch.float32) -> dict:
    model = Model(n_tokens, stream)
    tokens, targets, weight = batch(n_tokens)
    logprob, entropy = model.forward(tokens, targets)
    d_entropy = 0.01 * weight
    grads = model.backward(tokens, targets, weight, d_entropy)
    assert model.ok()
    return dict(model=model, tokens=tokens, targets=targets, weight=weight, d_entropy=d_entropy, grads=grads,
                logprob=logprob, entropy=entropy)


if __name__ == "__main__":
    out = run()
    print(f"mean log probability {float(out['logprob'].mean()):.3f}, entropy {float(out['entropy'].mean()):.3f}")
    for name, grad in out["grads"].items():
        print(f"{name:10s} {str(tuple(grad.shape)):14s} gradient's norm {float(grad.float().norm()):.3e}")
