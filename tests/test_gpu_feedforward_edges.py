"""GPU tests of the feed-forward operators at the ends of their ranges.  Tolerances as in
test_gpu_feedforward.py."""
from __future__ import annotations

import pytest
import torch

from test_gpu_feedforward import (B, TINY, _gen, _norm64, _norm_inputs, _normal, _ok, _within,
                                  test_residual_norm_backward as _check_backward)

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


def _codes_are_the_definition(wq, x, y, gate, wp, wn, per, scale, eps=1e-6):
    """Codes and scales equal those of 64 bits, clamped to +-127; returns them."""
    r, q, s = wq.residual_norm(x, y, gate, wp, wn, rows_per_gate=per, scale=scale, eps=eps, quantize=True)
    _ok(wq)
    R, H, _, _ = _norm64(x, y, gate, per, wp, wn, scale, eps)
    S = (H.abs().amax(1) / 127).float()
    Q = torch.where(S[:, None] > 0, H / S.double()[:, None], torch.zeros_like(H)).round().clamp(-127, 127)
    assert torch.equal(s, S), (s, S)
    assert torch.equal(q, Q.to(torch.int8)), (q != Q).nonzero()[:4]
    assert ((r.double() - R).abs() <= B * R.abs() + TINY).all()
    return q, s


@pytest.mark.parametrize("D", [8, 264, 2048, 4096])
def test_codes_of_a_subnormal_scale(wq, D):
    """A scale that is subnormal is rounded by up to a half: codes stop at +-127 in place of
    changing their sign.  Rows enough for every form of the kernel."""
    bf = torch.bfloat16
    for M in (3, 700):
        x = torch.full((M, D), 3.0, device="cuda", dtype=bf)
        x[:, 0] = 0.05
        wn = torch.zeros(D, device="cuda", dtype=bf)
        wn[0] = 1e-40
        q, s = _codes_are_the_definition(wq, x, None, None, None, wn, M, 1.0)
        assert (s > 0).all() and (s < 2.0 ** -126).all()
        # D = 8 (rms 2.81): amax / 127 is 9.2 x 2^-149, the scale 9, the quotient 129.9.  From
        # D = 264 on (rms 2.99) amax / 127 is 8.6 x 2^-149, the scale 9 too, the code 122
        assert D > 8 or (q[:, 0] == 127).all()
        _codes_are_the_definition(wq, -x, None, None, None, wn, M, 1.0)
        # tiny rows under an ordinary weight: from scales just above the normal range to none
        zero = torch.zeros(M, D, device="cuda", dtype=bf)
        y = (torch.linspace(0.2, 1.0, D, device="cuda") * 1e-30).to(bf).expand(M, D).contiguous()
        one = torch.ones(D, device="cuda", dtype=bf)
        for scale in (2e-9, 7e-10, 3e-12, 7e-15, 2.5e-16, 1.6e-16, 9e-17, 1e-17):
            _codes_are_the_definition(wq, zero, y, None, None, one, M, scale)


# magnitudes of y, gate and w_post whose product leaves fp32's normal range, or comes near its ends
FAR = [(1e35, 100.0, 100.0), (1e35, 1e-36, 1e-20), (1e-35, 1e-10, 1.0), (1e-30, 1e-14, 1e-3), (1e30, 1e30, 1e-30),
       (1e-39, 1e30, 1.0), (1e13, 1e12, 1e12), (1e-13, 1e-12, 1e-12), (1.0, 1e25, 1e-25), (1e-20, 1e-20, 1e20)]


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("D,M,per", [(8, 3, 1), (1032, 5, 2), (264, 700, 1), (4096, 700, 64), (2048, 400, 1)])
def test_codes_where_gate_and_norm_leave_fp32(wq, D, M, per, post):
    """Codes are the definition's whatever the magnitudes of y, gate and w_post; rows whose r is
    the far product alone among them, zeros and ordinary columns beside far ones."""
    g = _gen(D + M)
    for big, gt, wt in FAR:
        x, y, gate, wp, wn = _norm_inputs(g, M, D, per)
        x[::2] = 0
        y, gate, wp = (y.float() * big).bfloat16(), (gate.float() * gt).bfloat16(), (wp.float() * wt).bfloat16()
        y[:, 3::16] = 0
        y[:, 5::32] = 1.0
        gate[:, 6::16] = 0
        gate[:, 1::32] = -0.5
        R, _, _, _ = _norm64(x, y, gate, per, wp if post else None, wn, 0.7, 1e-30)
        if not (R.abs() < 3e38).all():  # r itself is no number of its type
            continue
        _codes_are_the_definition(wq, x, y, gate, wp if post else None, wn, per, 0.7, eps=1e-30)


def test_codes_and_bf16_agree_on_a_far_row(wq):
    """y near 1e35 with gate and w_post near 100: r and h are ordinary numbers in both forms."""
    g = _gen(5)
    x, y, gate, wp, wn = _norm_inputs(g, 6, 512, 3)
    y, gate, wp = (y.float() * 1e35).bfloat16(), (gate.float() * 100).bfloat16(), (wp.float() * 100).bfloat16()
    r, h = wq.residual_norm(x, y, gate, wp, wn, rows_per_gate=3)
    r2, q, s = wq.residual_norm(x, y, gate, wp, wn, rows_per_gate=3, quantize=True)
    _ok(wq)
    assert torch.isfinite(h).all() and torch.isfinite(s).all()
    # bf16 of both, and half a step of the codes
    assert ((q.double() * s.double()[:, None] - h.double()).abs() <= 0.51 * s.double()[:, None] + 2 * B * h.double().abs()).all()
    assert ((r.double() - r2.double()).abs() <= 2 * B * r.double().abs()).all()


@pytest.mark.parametrize("per", [1, 3])
@pytest.mark.parametrize("D", [264, 8200])
def test_norm_backward_of_far_y_and_small_gates(wq, D, per):
    """y near bf16's largest numbers under small gates: yhat is ordinary, and so is r / rms(r)
    where r is the gated norm alone.  (1 / rms(y) may be subnormal in fp32: 2^-21 relative.)"""
    M, scale, eps = 7, 0.7, 1e-30
    g = _gen(D + per)
    x, y, gate, wp, wn = _norm_inputs(g, M, D, per)
    x[::2] = 0
    y, gate = (y.float().clamp(-1.5, 1.5) * 2e38).bfloat16(), (gate.float() * 1e-7).bfloat16()
    dr, dh = _normal(g, M, D), _normal(g, M, D)
    _, _, rp, rn = wq.residual_norm(x, y, gate, wp, wn, rows_per_gate=per, scale=scale, eps=eps, save=True)
    dx, _, dgate, dwp, dwn = wq.residual_norm_backward(dr, dh, x, y, gate, wp, wn, rp, rn, rows_per_gate=per,
                                                       scale=scale)
    _ok(wq)
    rows = torch.arange(M, device="cuda") // per
    Y, G = y.double(), gate.double()[rows]
    RP = (Y.square().mean(1, keepdim=True) + eps).rsqrt()
    yh = Y * RP
    R = x.double() + scale * G * yh * wp.double()
    RN = (R.square().mean(1, keepdim=True) + eps).rsqrt()
    rh, a = R * RN, dh.double() * wn.double()
    ref = dr.double() + RN * (a - rh * (a * rh).mean(1, keepdim=True))
    size = dr.double().abs() + RN * (a.abs() + rh.abs() * (a * rh).abs().mean(1, keepdim=True))
    small = 2.0 ** -17
    _within(dx, ref, B * ref.abs() + small * size, "dx")
    t, s = dh.double() * rh, (dh.double() * rh).abs()
    _within(dwn, t.sum(0), B * t.sum(0).abs() + small * s.sum(0), "dw_pre")
    t, s = scale * ref * G * yh, scale * size * (G * yh).abs()
    _within(dwp, t.sum(0), B * t.sum(0).abs() + small * s.sum(0), "dw_post")
    t, s = scale * ref * yh * wp.double(), scale * size * (yh * wp.double()).abs()
    zero = torch.zeros(gate.shape, device="cuda", dtype=torch.float64)
    want = zero.index_add(0, rows, t)
    _within(dgate, want, B * want.abs() + small * zero.index_add(0, rows, s), "dgate")


def test_i8_extreme_codes_longest_k_many_tokens(wq):
    """-128 x -128 over the longest K with more tokens than the narrow kernels take; exact in fp32
    (2^14 K and -127 x 2^7 K are K times whole numbers below 2^15, K = 2^17 - 16)."""
    M, N, K = 200, 48, 131056
    xq = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    xq[3::7] = 127
    w = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    w[1::2] = 127
    one = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    y = wq.matmul_i8(xq, one[0], w, one[1], out_dtype=torch.float32)
    _ok(wq)
    assert torch.equal(y, ((xq[:, :1].double() * K) * w[:, 0].double()).float())


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_i8_nan_scale_stays_in_its_row_of_many(wq, out_dtype):
    g = _gen(6)
    M, N, K = 200, 80, 64
    xq = torch.randint(-128, 128, (M, K), device="cuda", generator=g).to(torch.int8)
    w = torch.randint(-128, 128, (N, K), device="cuda", generator=g).to(torch.int8)
    sx, sw = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    sx[2], sw[5] = float("nan"), float("nan")
    y = wq.matmul_i8(xq, sx, w, sw, out_dtype=out_dtype)
    _ok(wq)
    rows, cols = torch.arange(M, device="cuda") != 2, torch.arange(N, device="cuda") != 5
    assert torch.isnan(y[2]).all() and torch.isnan(y[:, 5]).all() and torch.isfinite(y[rows][:, cols]).all()


@pytest.mark.parametrize("K", [8, 64, 4104])
@pytest.mark.parametrize("bad", [float("nan"), -float("nan"), float("inf"), -float("inf")])
def test_quantize_rows_of_non_finite_values(wq, K, bad):
    """A row with a NaN or an infinity has no scale: NaN, and codes 0 (as the norms' codes); the
    product then shows it.  The other rows are the definition's, bf16's largest values among them."""
    g = _gen(K)
    x = _normal(g, 6, K)
    x[1, K - 1] = x[4, 0] = bad
    x[5] = torch.finfo(torch.bfloat16).max
    x[2] = 0
    q, s = wq.quantize_rows_int8(x)
    _ok(wq)
    good = torch.tensor([0, 2, 3, 5], device="cuda")
    assert torch.isnan(s[[1, 4]]).all() and not q[[1, 4]].any()
    X = x[good].double()
    S = (X.abs().amax(1) / 127).float()
    Q = torch.where(S[:, None] > 0, X / S.double()[:, None], torch.zeros_like(X)).round().clamp(-127, 127)
    assert torch.equal(s[good], S) and torch.equal(q[good], Q.to(torch.int8))
    if K % 16 == 0:
        w, sw = wq.quantize_rows_int8(_normal(g, 24, K))
        y = wq.matmul_i8(q, s, w, sw, out_dtype=torch.float32)
        _ok(wq)
        assert torch.isnan(y[[1, 4]]).all() and not torch.isnan(y[good]).any()
