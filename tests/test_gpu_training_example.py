"""The training step's calls together, as examples/training_step.py uses them: norms, sparse layers,
residual sums and log probabilities forward, and every weight's gradient backward, against a 64-bit
model of the same weights differentiated by autograd."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    import __graft_entry__ as g
    g.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import training_step
    return training_step


def model_in_64_bits(example, torch, out):
    """(logprob, entropy, gradients) with the sparse layer as its definition, ReLU(h W_in + b) W_down, where the units
    that are on are those that the layer stored: its backward goes by them, and a unit near zero that is on in one model
    only brings a whole term of w_in's gradient (one of 150 does, which would be 8 % of the norm)."""
    import activation_sparse_transformer_gb300 as tw
    m = out["model"]
    on = []
    for packed in m.packed:
        dense = torch.empty((m.n, example.D_FF), dtype=torch.bfloat16, device="cuda")
        tw.twell_unpack(packed, dense)
        on.append((dense != 0).double())
    leaf = lambda t: t.double().requires_grad_()  # noqa: E731
    w = {"embed": leaf(m.embed), "unembed": leaf(m.unembed)}
    w.update({f"norm{i}": leaf(t) for i, t in enumerate(m.norm)})
    for i, block in enumerate(m.blocks):
        w.update({f"{k}{i}": leaf(t) for k, t in block.items()})

    def norm(x, weight):
        return x * torch.rsqrt(x.square().mean(1, keepdim=True) + example.EPS) * weight

    x = w["embed"][out["tokens"]]
    h = norm(x, w["norm0"])
    for i in range(example.BLOCKS):
        y = (on[i] * (h @ w[f"w_in{i}"].T + w[f"b{i}"])) @ w[f"w_down{i}"]
        x = x + example.BRANCH_SCALE * w[f"gate{i}"] * norm(y, w[f"post{i}"])
        h = norm(x, w[f"norm{i + 1}"])
    logp = torch.log_softmax(h @ w["unembed"].T, 1)
    t = out["targets"].long()
    logprob = torch.where(t >= 0, logp.gather(1, t.clamp(min=0)[:, None])[:, 0], 0.0)
    entropy = -(logp.exp() * logp).sum(1)
    loss = (out["weight"].double() * logprob + out["d_entropy"].double() * entropy).sum()
    return logprob.detach(), entropy.detach(), dict(zip(w, torch.autograd.grad(loss, list(w.values()))))


@pytest.mark.parametrize("n_tokens,stream", [(300, "float32"), (77, "bfloat16")])
def test_training_example(example, n_tokens, stream):
    import torch
    out = example.run(n_tokens, getattr(torch, stream))
    logprob, entropy, want = model_in_64_bits(example, torch, out)
    # a block rounds h, its activations, y and (bf16 streams) x to bf16, each by 2^-8 at most; the logits, of size 3, move
    # with the last h
    bound = 4 * example.BLOCKS * 2.0 ** -8
    assert float((out["logprob"] - logprob).abs().max()) <= 4 * bound
    assert float((out["entropy"] - entropy).abs().max()) <= 4 * bound
    assert set(out["grads"]) == set(want)
    for name, got in out["grads"].items():
        assert torch.isfinite(got.float()).all(), name
        # as many roundings again on the way back, of G, d_h, d_y and d_x
        off = float((got.double() - want[name]).norm() / want[name].norm())
        assert off <= 2 * bound, f"{name}: {off:.3f}"


def test_training_step_in_a_graph(example):
    """One captured step, replayed with other tokens in its buffers, is the eager step of those tokens."""
    import torch
    eager = example.run(130)
    model = example.Model(130)
    tokens, targets, weight = example.batch(130, seed=5)
    d_entropy = 0.01 * weight
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        model.forward(tokens, targets)
        model.backward(tokens, targets, weight, d_entropy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        model.forward(tokens, targets)
        grads = model.backward(tokens, targets, weight, d_entropy)
    tokens.copy_(eager["tokens"])
    targets.copy_(eager["targets"])
    graph.replay()
    torch.cuda.synchronize()
    assert model.ok()
    assert torch.equal(model.logprob, eager["logprob"]) and torch.equal(model.entropy, eager["entropy"])
    for name, got in grads.items():
        if name == "embed":  # torch's index_add_ has no fixed order
            assert (got - eager["grads"][name]).norm() <= 1e-5 * got.norm()
        else:
            assert torch.equal(got, eager["grads"][name]), name
