"""Derivatives that the feed-forward helpers do not have are refused, not dropped."""
from __future__ import annotations

import pytest
import torch
from torch.autograd import forward_ad

from mixed_gemm_b200 import feedforward


def test_tangents_are_seen():
    x, q = torch.ones(4, 64), torch.zeros(4, 64, dtype=torch.int8)
    assert feedforward._dual_level() < 0
    with forward_ad.dual_level():
        assert feedforward._dual_level() >= 0
        d = forward_ad.make_dual(x, torch.ones_like(x))
        assert not d.requires_grad
        feedforward._no_tangents("f", (x, q, None, 3.0, "silu"))
        for ts in ((d,), (x, None, d), (q, d[:2])):
            with pytest.raises(ValueError, match="tangent"):
                feedforward._no_tangents("f", ts)
    assert feedforward._dual_level() < 0


def _calls(wq, t, q):
    """Each helper with ``t`` as one of its floating-point inputs."""
    s, v = t[:, 0].float(), t[0]
    plain = forward_ad.unpack_dual(t).primal.detach().clone()  # (detach keeps a tangent)
    assert forward_ad.unpack_dual(plain).tangent is None
    return {"gated_ff": lambda: wq.gated_ff(plain, t, plain),
            "gated_ff_save": lambda: wq.gated_ff(t, plain, plain, save=True),
            "gated_ff_bias": lambda: wq.gated_ff(plain, plain, plain, b_up=v),
            "gated_ff_backward": lambda: wq.gated_ff_backward(t, plain, plain, plain, plain, plain),
            "residual_norm": lambda: wq.residual_norm(plain, plain, w_pre=v),
            "residual_norm_save": lambda: wq.residual_norm(plain, y=t, w_pre=plain[0], save=True),
            "residual_norm_codes": lambda: wq.residual_norm(t, w_pre=plain[0], quantize=True),
            "residual_norm_backward": lambda: wq.residual_norm_backward(
                plain, None, plain, t, None, None, None, None, None),
            "quantize_rows_int8": lambda: wq.quantize_rows_int8(t),
            "matmul_i8": lambda: wq.matmul_i8(q, s, q, plain[0].float()),
            "out": lambda: wq.residual_norm(plain, plain, out=t)}


@pytest.mark.gpu
def test_forward_mode_is_refused(wq):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.empty(64, 64, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    q = torch.zeros(64, 64, device="cuda", dtype=torch.int8)
    want = wq.gated_ff(x, x, x)
    with forward_ad.dual_level():
        d = forward_ad.make_dual(x, torch.ones_like(x))
        for name, call in _calls(wq, d, q).items():
            with pytest.raises(ValueError, match="tangent"):
                call()
                pytest.fail(f"{name} was taken")
        # tensors without a tangent are taken inside a level too, and so is a primal
        assert torch.equal(wq.gated_ff(x, x, x), want)
        assert torch.equal(wq.gated_ff(forward_ad.unpack_dual(d).primal, x, x), want)
    torch.cuda.synchronize()
    assert wq.wq_device_error() == 0


@pytest.mark.gpu
def test_quantize_rows_int8_of_a_recorded_tensor(wq):
    """Codes and scales have no gradient: an input that requires one is refused unless the
    caller says that none is wanted."""
    x = torch.ones(4, 64, device="cuda", dtype=torch.bfloat16)
    want = wq.quantize_rows_int8(x)
    p = x.clone().requires_grad_(True)
    with pytest.raises(ValueError, match="detach"):
        wq.quantize_rows_int8(p)
    with pytest.raises(ValueError, match="detach"):
        wq.quantize_rows_int8(p * 2)
    taken = [wq.quantize_rows_int8(p.detach())]
    with torch.no_grad():
        taken.append(wq.quantize_rows_int8(p))
    for got in taken:
        assert all(torch.equal(a, b) and not a.requires_grad for a, b in zip(got, want))
