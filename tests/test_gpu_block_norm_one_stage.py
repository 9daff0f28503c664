"""Norms of fp32 streams at widths where one row at a time is on its way to a group of threads (4096 and 8192 columns, and
their neighbours), with numbers of rows that do not fill the last round."""
import pytest
import test_gpu_block_norm as base
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tw():
    import activation_sparse_transformer_gb300 as m
    m.load_library()
    return m


SIZES = [(701, 4096), (305, 4096), (401, 8192), (153, 8192), (3, 8192), (350, 4088), (350, 4104), (200, 8184)]


@pytest.mark.parametrize("flags", ["ypgrn", "yn", "ypr", "n"])
@pytest.mark.parametrize("rows,dim", SIZES)
def test_forward_and_gradient(tw, rows, dim, flags):
    i = base.make(rows, dim, torch.float32, flags, 41, pad=8)
    base.check_forward(i, base.run(tw, i, 0.75, -1.25), 0.75, -1.25)
    out, want, size, call = base.backward(tw, i, 0.75, -1.25, 42)
    base.check_backward(out, want, size, rows)
    first = {k: v.clone() for k, v in out.items() if v is not None}
    call()
    for k in first:
        assert torch.equal(out[k], first[k]), k
