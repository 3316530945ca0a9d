"""The residual's norm at the edges of its types and layouts."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
TINY = 2.0 ** -149                                           # fp32's smallest number


@pytest.fixture(scope="module")
def kdn():
    from bayesian_scan_gb300 import kdn as k
    return k


@pytest.mark.parametrize("C", [256, 257, 640, 2048, 2049, 20000])
@pytest.mark.parametrize("rows", [3, 1300])
def test_8_bits_of_groups_that_all_but_vanish(kdn, rows, C):
    # rows of 1 and -1, so 1 / rms is 1 - 5e-7 and y is the weight: n TINY less 5e-7 of it and one rounding is
    # n TINY again (n < 1000).  A group's largest / 448 is 0 up to 224 TINY, 1 TINY up to 672.
    sign = torch.where(torch.arange(rows * C).view(rows, C) % 3 == 0, -1.0, 1.0)
    w = torch.ones(C)
    some = torch.tensor([0, 1, 70, 224] * 32)
    w[:128] = some * TINY                                    # scale 1, all zeros
    w[128:256] = torch.tensor([0, 5, 225, 448] * 32) * TINY  # scale TINY
    y, _, scale = kdn.add_rms_norm_fwd(sign.cuda(), weight=w.cuda(), out_dtype=E4M3)
    y, scale = y.float().cpu(), scale.cpu()
    assert (scale[:, 0] == 1).all() and (y[:, :128] == 0).all()
    assert (scale[:, 1] == TINY).all()
    assert torch.equal(y[:, 128:256], sign[:, 128:256] * (w[128:256] / TINY).to(E4M3).float())
    if C > 256:
        # |y| = 1 - 5e-7 everywhere: the largest, 448 units of its scale within a rounding or two
        assert (y[:, 256:].abs() == 448).all() and ((scale[:, 2:] * 448 - 1).abs() < 1e-6).all()


@pytest.mark.parametrize("rows,C,wide,first", [(60, 96, 200, 40), (60, 96, 201, 41), (5, 2048, 6144, 2048)])
@pytest.mark.parametrize("given_stream", [False, True])
def test_a_slice_that_is_its_own_sum_goes_back(kdn, rows, C, wide, first, given_stream):
    # without a residual the forward returns x itself, a column slice too; the backward takes what it returned
    g = torch.Generator().manual_seed(C)
    x = torch.randn(rows, wide, generator=g).to(BF16).cuda()[:, first:first + C]
    w, gy = torch.randn(C, generator=g).cuda(), torch.randn(rows, C, generator=g).to(BF16).cuda()
    gs = torch.randn(rows, C, generator=g).to(BF16).cuda()
    want = kdn.add_rms_norm_bwd(x.contiguous(), gy, weight=w, grad_sum=gs)
    side = torch.cuda.Stream() if given_stream else None
    torch.cuda.synchronize()
    _, s, _ = kdn.add_rms_norm_fwd(x, weight=w, stream=side)
    assert s is x
    got = kdn.add_rms_norm_bwd(s, gy, weight=w, grad_sum=gs, stream=side)
    torch.cuda.synchronize()
    assert all(got[n].is_contiguous() and torch.equal(got[n], want[n]) for n in want)
    with pytest.raises(ValueError, match="adjacent channels"):
        kdn.add_rms_norm_bwd(x[:, ::2], gy[:, ::2].contiguous())
