"""layer_norm on tensors that start between 16-byte boundaries: parameters that are
slices of one buffer, and rows that are no whole number of 16-byte vectors.
"""
import pytest
import torch

import gated_delta_rule_bwd_gb300 as gdn
from test_layer_norm import compare, make

gpu = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 257, 1024, 8192])
def test_parameters_in_one_buffer(D, dtype):
    x, w, b, dy = make(5, D, dtype, seed=D)
    flat = torch.cat([w[:1], w, b])
    got = compare(x, flat[1:D + 1], flat[D + 1:], dy)
    assert all(torch.equal(s, t) for s, t in zip(got, compare(x, w, b, dy)))
    y, mean, rstd = gdn.layer_norm_fwd(x, w, b)
    stats = torch.cat([mean[:1], mean, rstd])
    dx, dw, db = gdn.layer_norm_bwd(x, w, stats[1:6], stats[6:], dy)
    assert torch.equal(dx, got[1]) and torch.equal(dw, got[2]) and torch.equal(db, got[3])


@gpu
@pytest.mark.parametrize("D,dtype", [(257, BF16), (1001, BF16), (12, BF16), (257, F32), (6, F32)])
def test_rows_between_boundaries(D, dtype):
    x, w, b, dy = make(8, D, dtype, seed=D)
    assert x[1:].data_ptr() % 16
    compare(x[1:], w, b, dy[1:])


@gpu
def test_whole_vectors_stay_refused():
    flat = torch.zeros(1 + 4 * 64, dtype=BF16, device="cuda")
    w = torch.ones(64, device="cuda")
    with pytest.raises(gdn.GdnError, match="aligned"):
        gdn.layer_norm_fwd(flat[1:].view(4, 64), w)
