"""GPU tests of the feed-forward operators at the ends of their ranges.  Tolerances as in
test_gpu_feedforward.py."""
from __future__ import annotations

import pytest
import torch

from test_gpu_feedforward import _gen, _norm_inputs, _normal, _ok, test_residual_norm_backward as _check_backward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,D", [(1, 8200), (2, 16384), (73, 9000), (75, 16384)])
def test_norm_backward_rows_shared_by_two_blocks(wq, M, D):
    """Wide rows, one or two to a pair of blocks, so that a pair's first exchange comes right
    after its start; the same bits every time."""
    _check_backward(wq, M, D, M, "all")
    _check_backward(wq, M, D, 1, "noy")
    g = _gen(M + D)
    x, y, gate, wp, wn = _norm_inputs(g, M, D, M)
    dr, dh = _normal(g, M, D), _normal(g, M, D)
    _, _, rp, rn = wq.residual_norm(x, y, gate, wp, wn, save=True)
    first = wq.residual_norm_backward(dr, dh, x, y, gate, wp, wn, rp, rn)
    for _ in range(20):
        again = wq.residual_norm_backward(dr, dh, x, y, gate, wp, wn, rp, rn)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    _ok(wq)
