"""The decoder's norms (examples/decode_step.py) are torch's rms_norm of the same rows, its eps included."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_norms_of_the_decoder(monkeypatch):
    import torch
    import __graft_entry__ as g
    g.build()
    monkeypatch.syspath_prepend(os.path.join(ROOT, "examples"))
    sys.modules.pop("decode_step", None)
    import decode_step
    tw, norm, seen = decode_step.tw, decode_step.tw.twell_block_norm, []

    def spy(x, y, x_out, h, **given):
        z = x.float() if y is None else x.float() + y.float()
        norm(x, y, x_out, h, **given)
        want = torch.nn.functional.rms_norm(z, z.shape[1:])
        # two roundings to bf16 of values that differ by fp32's: a step of bf16 for some, most equal
        seen.append((given["eps"], float((h.float() - want.bfloat16().float()).abs().max() / want.abs().max()),
                     float((h != want.bfloat16()).float().mean())))

    monkeypatch.setattr(tw, "twell_block_norm", spy)
    decode_step.run(prompt_lens=(9, 3), steps=2)
    assert seen
    for eps, off, differ in seen:
        assert eps == torch.finfo(torch.float32).eps
        assert off <= 2.0 ** -7 and differ <= 2.0 ** -8
