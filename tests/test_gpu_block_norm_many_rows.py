"""Norms of as many rows as the call's int32 can count (2^31 - 1 of 8 columns, 34 GB): all SMs take their share."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tw():
    import activation_sparse_transformer_gb300 as m
    m.load_library()
    return m


@pytest.mark.parametrize("rows", [2 ** 31 - 1, 2 ** 31 - 32, 2 ** 31 - 160])
def test_rows_up_to_the_last_number(tw, rows):
    if torch.cuda.mem_get_info()[0] < 50 << 30:
        pytest.skip("34 GB beside what others hold")
    x = torch.full((rows, 8), 2.0, dtype=torch.bfloat16, device="cuda")
    marks = [0, 1, 31, 1 << 30, rows - 33, rows - 2, rows - 1]
    for k, r in enumerate(marks):
        x[r] = float(k + 4)
    ends = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
    ends[0].record()
    tw.twell_block_norm(x, None, x, skip_scale=0.5)       # in place: a half
    ends[1].record()
    tw.twell_block_norm_bwd(None, x, None, None, x, skip_scale=4.0)  # and four times that
    ends[2].record()
    torch.cuda.synchronize()
    for k, r in enumerate(marks):
        assert (x[r] == 2 * (k + 4)).all(), r
        x[r] = 4.0
    assert float(x.min()) == 4.0 and float(x.max()) == 4.0
    # 69 GB there and back, 10 ms; one CTA alone takes more than a minute
    assert ends[0].elapsed_time(ends[1]) < 2000 and ends[1].elapsed_time(ends[2]) < 2000
