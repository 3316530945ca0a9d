"""The residual's addition and its norm on the GPU against 64 bits.

Bounds, in units of 2^-24: a sum of C squares is within C/2 + 5 of itself (the
terms are positive; lanes and warps add in trees), its root half of that; the
other factors of y add at most 8.  The backward's second sum, over t . s, is
within C units of the sum of its magnitudes."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
UNIT = 2.0 ** -24
EPS = 1e-6


@pytest.fixture(scope="module")
def kdn():
    from bayesian_scan_gb300 import kdn as k
    return k


def half(t):
    return torch.finfo(t).eps / 2


def draw(rows, C, dt, rt, seed, weight=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, C, generator=g).to(dt)
    r = (torch.exp(2 * torch.randn(rows, 1, generator=g)) * torch.randn(rows, C, generator=g)).to(rt)
    w = 1 + 0.5 * torch.randn(C, generator=g) if weight else None
    return x, r, w, g


def norm64(s, w, eps=EPS):
    n = s / torch.sqrt(s.square().mean(-1, keepdim=True) + eps)
    return n if w is None else n * w.double()


SIZES = [(1, 1), (3, 7), (1, 128), (5, 136), (2, 1000), (7, 257), (9, 2048), (4, 4096), (3, 8192), (2, 20000), (2, 20001),
         (1, 40000), (1300, 64), (1300, 512), (2500, 1000), (1220, 2048), (1501, 129)]
TYPES = [(BF16, BF16, BF16), (BF16, F32, BF16), (F32, F32, F32), (F32, BF16, F32), (BF16, BF16, F32)]


@pytest.mark.parametrize("rows,C", SIZES)
@pytest.mark.parametrize("dt,rt,ot", TYPES)
def test_forward(kdn, rows, C, dt, rt, ot):
    x, r, w, _ = draw(rows, C, dt, rt, rows + C)
    y, s, scale = kdn.add_rms_norm_fwd(x.cuda(), r.cuda(), weight=w.cuda(), eps=EPS, out_dtype=ot)
    assert scale is None and y.dtype == ot and s.dtype == rt
    assert torch.equal(s.cpu(), (x.float() + r.float()).to(rt))
    want = norm64(s.cpu().double(), w)
    assert ((y.cpu().double() - want).abs() <= (((C / 4 + 11) * UNIT) + half(ot)) * want.abs() + 1e-40).all()
    y, s, _ = kdn.add_rms_norm_fwd(x.cuda(), eps=EPS)        # no residual, no weight
    want = norm64(x.double(), None)
    assert torch.equal(s.cpu(), x)
    assert ((y.cpu().double() - want).abs() <= (((C / 4 + 11) * UNIT) + half(dt)) * want.abs() + 1e-40).all()


@pytest.mark.parametrize("rows,C", SIZES)
@pytest.mark.parametrize("dt,rt", [(BF16, BF16), (BF16, F32), (F32, F32)])
def test_8_bits(kdn, rows, C, dt, rt):
    x, r, w, _ = draw(rows, C, dt, rt, rows + C)
    x[0], r[0] = 0, 0                                        # a row of zeros
    w[-1] = 0
    y, s, scale = kdn.add_rms_norm_fwd(x.cuda(), r.cuda(), weight=w.cuda(), eps=EPS, out_dtype=E4M3)
    assert y.dtype == E4M3 and scale.shape == (rows, -(-C // 128)) and torch.equal(s.cpu(), (x.float() + r.float()).to(rt))
    want = norm64(s.cpu().double(), w)
    pad = torch.nn.functional.pad(want, (0, -C % 128)).unflatten(-1, (-1, 128))
    top = pad.abs().amax(-1)
    e = (C / 4 + 13) * UNIT
    sc = scale.cpu().double()
    assert (sc[top == 0] == 1).all()
    assert ((sc - top / 448).abs()[top > 0] <= e * (top / 448)[top > 0]).all()
    # in units of the scale: half a step of the value (2^-4 of it), of 2^-9 below the normal range
    got = y.cpu().float().double()
    q = (pad / sc.unsqueeze(-1)).flatten(-2)[:, :C]
    assert got.isfinite().all()
    assert ((got - q).abs() <= torch.maximum(q.abs() * (2.0 ** -4 + 3 * e), torch.tensor(2.0 ** -10)) * (1 + 1e-5)).all()
    assert (got[0] == 0).all() and (got[:, -1] == 0).all()


@pytest.mark.parametrize("rows,C", SIZES)
@pytest.mark.parametrize("dt,rt,ot", TYPES)
def test_backward(kdn, rows, C, dt, rt, ot):
    x, s, w, g = draw(rows, C, dt, rt, 3 * rows + C)
    gy = torch.randn(rows, C, generator=g).to(ot)
    gs = torch.randn(rows, C, generator=g).to(rt)
    s64, w64 = s.double().requires_grad_(), w.double().requires_grad_()
    (norm64(s64, w64) * gy.double()).sum().backward()
    want = s64.grad + gs.double()
    got = kdn.add_rms_norm_bwd(s.cuda(), gy.cuda(), weight=w.cuda(), grad_sum=gs.cuda(), eps=EPS, x_dtype=dt)
    r = 1 / torch.sqrt(s.double().square().mean(-1, keepdim=True) + EPS)
    n, t = s.double() * r, gy.double() * w.double()
    e = (C / 4 + 16) * UNIT
    mag = r * (t.abs() + n.abs() * (t * n).abs().mean(-1, keepdim=True) * (1 + 4 * C * UNIT / e)) + gs.double().abs()
    for name, ty in (("residual", rt), ("x", dt)):
        assert got[name].dtype == ty
        assert ((got[name].cpu().double() - want).abs() <= 3 * e * mag + half(ty) * want.abs() + 1e-40).all(), name
    mag = (gy.double() * n).abs().sum(0)
    assert ((got["weight"].cpu().double() - w64.grad).abs() <= (2 * e + rows * UNIT) * mag + 1e-40).all()
    got = kdn.add_rms_norm_bwd(s.cuda(), gy.cuda(), eps=EPS, grad_weight=True)      # no weight, no other gradient
    mag = r * (gy.double().abs() + n.abs() * (gy.double() * n).abs().mean(-1, keepdim=True) * (1 + 4 * C * UNIT / e))
    s64 = s.double().requires_grad_()
    (norm64(s64, None) * gy.double()).sum().backward()
    assert ((got["x"].cpu().double() - s64.grad).abs() <= 3 * e * mag + half(rt) * s64.grad.abs() + 1e-40).all()
    assert got["x"] is got["residual"]
    want, mag = (gy.double() * n).sum(0), (gy.double() * n).abs().sum(0)
    assert ((got["weight"].cpu().double() - want).abs() <= (2 * e + rows * UNIT) * mag + 1e-40).all()


def test_column_slices_and_batches(kdn):
    x, r, w, _ = draw(60, 96, BF16, BF16, 1)
    wide = torch.zeros(3, 20, 200, dtype=BF16)
    wide[..., 40:136] = x.view(3, 20, 96)
    wide[..., :40] = wide[..., 136:] = torch.nan
    want, s, _ = kdn.add_rms_norm_fwd(x.cuda(), r.cuda(), weight=w.cuda())
    y, s2, _ = kdn.add_rms_norm_fwd(wide.cuda()[..., 40:136], r.cuda().view(3, 20, 96), weight=w.cuda())
    assert torch.equal(y.view(60, 96), want) and torch.equal(s2.view(60, 96), s)
    wide = torch.zeros(3, 20, 201, dtype=BF16)                # rows that 16-byte loads cannot read
    wide[..., 41:137] = x.view(3, 20, 96)
    y, s2, _ = kdn.add_rms_norm_fwd(wide.cuda()[..., 41:137], r.cuda().view(3, 20, 96), weight=w.cuda())
    assert torch.equal(s2.view(60, 96), s)
    a, b = y.view(60, 96).float(), want.float()              # the sum of squares in another order
    assert ((a - b).abs() <= 2 ** -7 * b.abs()).all()


def test_in_place(kdn):
    x, r, w, g = draw(50, 264, BF16, F32, 2)
    res = r.cuda()
    want, s, _ = kdn.add_rms_norm_fwd(x.cuda(), res, weight=w.cuda())
    y, s2, _ = kdn.add_rms_norm_fwd(x.cuda(), res, weight=w.cuda(), sum_out=res)
    assert s2 is res and torch.equal(res, s) and torch.equal(y, want)
    gy, gs = torch.randn(50, 264, generator=g).to(BF16).cuda(), torch.randn(50, 264, generator=g).cuda()
    a = kdn.add_rms_norm_bwd(s, gy, weight=w.cuda(), grad_sum=gs, x_dtype=BF16)
    b = kdn.add_rms_norm_bwd(s, gy, weight=w.cuda(), grad_sum=gs, x_dtype=BF16, grad_residual=gs)
    assert b["residual"] is gs and all(torch.equal(a[n], b[n]) for n in a)
    for C in (30000, 30001):                                 # rows that the registers do not hold
        x, r, w, g = draw(3, C, BF16, F32, C)
        gy, gs = torch.randn(3, C, generator=g).to(BF16).cuda(), torch.randn(3, C, generator=g).cuda()
        a = kdn.add_rms_norm_bwd(r.cuda(), gy, weight=w.cuda(), grad_sum=gs, x_dtype=BF16)
        b = kdn.add_rms_norm_bwd(r.cuda(), gy, weight=w.cuda(), grad_sum=gs, x_dtype=BF16, grad_residual=gs)
        assert all(torch.equal(a[n], b[n]) for n in a)
        res = r.cuda()
        want, s, _ = kdn.add_rms_norm_fwd(x.cuda(), res, weight=w.cuda())
        y, s2, _ = kdn.add_rms_norm_fwd(x.cuda(), res, weight=w.cuda(), sum_out=res)
        assert torch.equal(res, s) and torch.equal(y, want)


def test_nothing(kdn):
    x = torch.empty(0, 64, device="cuda")
    y, s, _ = kdn.add_rms_norm_fwd(x, x)
    assert y.shape == (0, 64) and s.shape == (0, 64)
    y, s, scale = kdn.add_rms_norm_fwd(x, x, out_dtype=E4M3)
    assert scale.shape == (0, 1)
    got = kdn.add_rms_norm_bwd(x, x, grad_weight=True)
    assert got["x"].shape == (0, 64) and (got["weight"] == 0).all()


def test_what_is_not_finite_stays_in_its_row(kdn):
    x, r, w, _ = draw(2500, 512, F32, F32, 4)
    clean = kdn.add_rms_norm_fwd(x.cuda(), r.cuda(), weight=w.cuda(), out_dtype=E4M3)
    x[3, 5], x[1000, 7] = torch.nan, torch.inf
    y, s, scale = kdn.add_rms_norm_fwd(x.cuda(), r.cuda(), weight=w.cuda(), out_dtype=E4M3)
    rest = torch.ones(2500, dtype=torch.bool)
    rest[3] = rest[1000] = False
    for a, b in zip((y.float(), s, scale), (clean[0].float(), clean[1], clean[2])):
        assert torch.equal(a.cpu()[rest], b.cpu()[rest])
    assert y.float()[3].isnan().all() and y.float()[1000, 7].isnan()


@pytest.mark.parametrize("rows,C", [(3000, 512), (5, 2048)])
def test_streams_graphs_and_the_same_again(kdn, rows, C):
    x, r, w, g = draw(rows, C, BF16, BF16, 6)
    x, r, w = x.cuda(), r.cuda(), w.cuda()
    gy = torch.randn(rows, C, generator=g).to(BF16).cuda()
    y, s, _ = kdn.add_rms_norm_fwd(x, r, weight=w)
    gr = kdn.add_rms_norm_bwd(s, gy, weight=w, grad_sum=gy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, s2, _ = kdn.add_rms_norm_fwd(x, r, weight=w, stream=side)
    gr2 = kdn.add_rms_norm_bwd(s2, gy, weight=w, grad_sum=gy, stream=side)
    side.synchronize()
    assert torch.equal(y, y2) and all(torch.equal(gr[n], gr2[n]) for n in gr)
    graph, static = torch.cuda.CUDAGraph(), x.clone()
    with torch.cuda.graph(graph):
        y3, s3, _ = kdn.add_rms_norm_fwd(static, r, weight=w)
        gr3 = kdn.add_rms_norm_bwd(s3, gy, weight=w, grad_sum=gy)
    static.mul_(3)
    graph.replay()
    torch.cuda.synchronize()
    y4, s4, _ = kdn.add_rms_norm_fwd(static, r, weight=w)
    gr4 = kdn.add_rms_norm_bwd(s4, gy, weight=w, grad_sum=gy)
    assert torch.equal(y3, y4) and torch.equal(s3, s4) and all(torch.equal(gr3[n], gr4[n]) for n in gr4)
