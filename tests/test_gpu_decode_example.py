"""The decode step's calls together, as examples/decode_step.py uses them: the
tables, the cache, the attention, the sparse layer, the log probabilities and their gradient."""
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
    import decode_step
    return decode_step


@pytest.mark.parametrize("fmt", ["KV_E4M3", "KV_INT8"])
def test_decode_example(example, fmt):
    import torch
    import activation_sparse_transformer_gb300 as tw
    out = example.run(fmt=getattr(tw, fmt))
    # answers of 12 tokens, 7 for the request that ended half way, whose pages are free again
    assert [len(s) for s in out["scores"]] == [12, 7, 12, 12]
    assert out["lens"] == [37 + 12, 0, 130 + 12, 64 + 12]
    held = sum(-(-n // example.PAGE) for n in out["lens"])
    assert out["free"] + held == out["pages"]
    # a token's log probability does not depend on how the steps were cut: bf16
    # projections and 8-bit codes of a page that may have moved to a larger scale, two
    # layers, log probabilities of size 1 to 7
    assert out["off"] < 0.25
    # gradients of a log-softmax sum to zero over the vocabulary (bf16 entries: half a
    # unit of 2^-8 of each)
    d = out["d_logits"].float()
    assert torch.isfinite(d).all() and d.abs().sum() > 0
    assert (d.sum(1).abs() <= 2.0 ** -8 * d.abs().sum(1) + 1e-12).all()
    assert torch.isfinite(out["d_unembed"].float()).all()
