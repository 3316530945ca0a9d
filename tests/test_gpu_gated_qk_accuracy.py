"""Accuracy where the other tests' bounds are wide: angles near zero and far
away, rows of extreme size, convex weights, and sums over many rows.  Units
are half steps of fp32, 2^-24."""
import pytest
import torch

import plain64

pytestmark = pytest.mark.gpu

F32 = torch.float32
UNIT = plain64.UNIT


@pytest.mark.parametrize("size", [1e14, 1e-14, 1e17, 1e-17])
@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("dk,Hq", [(128, 3), (16, 5)])
def test_rows_of_any_size_have_their_gradient(dk, Hq, norm, size):
    # the norm's inverse cubed is beyond fp32's range, the gradient is not
    from bayesian_scan_gb300 import kdn
    g = torch.Generator().manual_seed(dk)
    x = torch.randn(2, 33, Hq, dk, generator=g) * size
    go, w = torch.randn(2, Hq, 33, dk, generator=g), 1 + 0.3 * torch.randn(dk, generator=g)
    inv = (1e4 ** (-torch.arange(dk // 2) / (dk // 2))).float()
    theta = plain64.rotation_angles(torch.arange(33).expand(1, 2, 33), inv, None)
    got = kdn.qk_norm_rope_bwd(x.cuda(), None, go.cuda(), None, inv_freq=inv.cuda(), wq=w.cuda(), norm=norm, eps=0.0)
    gx, ex, gw, ew = plain64.qk_bwd(x, w, go, theta, dk, False, norm, 0.0)
    scaled = got["q"].cpu().double() * size                  # (of order one, whatever the rows' size)
    assert scaled.isfinite().all()
    assert ((scaled - gx * size).abs() <= (ex + UNIT * (gx.abs() + ex)) * size).all()
    plain64.assert_within(got["wq"], gw, ew)
