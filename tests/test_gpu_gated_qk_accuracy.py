"""Accuracy where the other tests' bounds are wide: angles near zero and far
away, rows of extreme size, convex weights, and sums over many rows.  Units
are half steps of fp32, 2^-24."""
import math
from fractions import Fraction

import pytest
import torch

import plain64

pytestmark = pytest.mark.gpu

F32 = torch.float32
UNIT = plain64.UNIT
TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534")


def turned(pos, inv):
    """cos and sin of pos x inv as the kernels have them: pairs (1, 0) turned."""
    from bayesian_scan_gb300 import kdn
    T, dk = len(pos), 128
    x = torch.zeros(1, T, 1, dk, device="cuda")
    x[..., :dk // 2] = 1
    o = kdn.qk_norm_rope_fwd(x, None, torch.tensor(pos, dtype=torch.int32, device="cuda")[None], inv.cuda(),
                             norm="none")[0][0, 0].cpu().double()
    return o[:, :dk // 2], o[:, dk // 2:]


def exact(pos, inv):
    """(cos, sin) from the angle modulo a turn in rational arithmetic."""
    c, s = (torch.zeros(len(pos), len(inv), dtype=torch.float64) for _ in range(2))
    for j, f in enumerate(inv.tolist()):
        for i, p in enumerate(pos):
            a = Fraction(f) * p
            a = float(a - round(a / TWO_PI) * TWO_PI)
            c[i, j], s[i, j] = math.cos(a), math.sin(a)
    return c, s


# An angle in turns is a 64-bit fraction: a frequency's is within 2^-63 turns, so that of position pos
# within |pos| 2^-63 turns, |pos| 2^-60 radians.  Beyond that cos and sin are within 6 units of
# themselves: the conversion and the product by x one each, its square's effect less than one, the
# polynomials 1.5 and their roundings 1.5.
VALUE = 6 * UNIT


def test_small_angles_keep_their_sine():
    # frequencies down to those of long-context bases
    inv = torch.logspace(-9, 0, 64, base=10.0)
    pos = [0, 1, 2, 3, 7, 100, 1001, 65535, -1, -2, -5, -333, 1 << 20]
    c, s = turned(pos, inv)
    rc, rs = exact(pos, inv)
    for got, ref in ((c, rc), (s, rs)):
        lim = VALUE * ref.abs() + torch.tensor(pos).abs().double()[:, None] * 2.0 ** -60
        assert ((got - ref).abs() <= lim).all(), float(((got - ref).abs() / lim).nan_to_num(0).max())


def test_fast_frequencies_at_far_positions():
    # frequencies above one: a turn or many per token
    g = torch.Generator().manual_seed(1)
    inv = torch.cat([torch.logspace(0, 6, 60, base=10.0), torch.tensor([1.0, 402.12387, 2.0 ** 20, 2.0 ** 40])])
    pos = [2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1, 12345, 1] + torch.randint(-2 ** 31, 2 ** 31, (20,), generator=g).tolist()
    c, s = turned(pos, inv)
    rc, rs = exact(pos, inv)
    for got, ref in ((c, rc), (s, rs)):
        lim = VALUE * ref.abs() + torch.tensor(pos).abs().double()[:, None] * 2.0 ** -60
        assert ((got - ref).abs() <= lim).all(), float(((got - ref).abs() / lim).max())


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


def test_convex_weights():
    # w = 1 - exp(-d) alone (A = 1, x = 1, no state), fp32 in and out.  The exponent is within 1.5 units
    # of itself, which moves w by at most as much of itself; the polynomial branch adds 2, the hardware's
    # 2^x (2^-22, below a half) 4, a product one: 4.5 units, and 6.5 beyond a half
    from bayesian_scan_gb300 import kdn
    d = torch.cat([torch.logspace(-30, 0, 2000, base=2.0), torch.linspace(0.2, 1.2, 6000), torch.linspace(1.2, 20, 192)])
    ref = -torch.expm1(-d.double())
    C = len(d)
    ones, A = torch.ones(1, C, device="cuda"), torch.ones(C, device="cuda")
    got = {"step": kdn.gated_step(ones, d.cuda()[None], A, torch.zeros_like(ones), leak=True)[0]}
    o, f = kdn.gated_scan_fwd(ones[:, None], d.cuda()[None, None], A, leak=True)
    got["out"], got["final"] = o[0, 0], f[0]
    b = kdn.gated_scan_bwd(ones[:, None], d.cuda()[None, None], A, o, ones[:, None], leak=True)
    got["grad_x"] = b["x"][0, 0]
    for n, v in got.items():
        off = (v.cpu().double() - ref).abs() / (UNIT * ref)
        assert off[ref < 0.5].max() <= 4.5 and off.max() <= 6.5, (n, float(off[ref < 0.5].max()), float(off.max()))


@pytest.mark.parametrize("B,C", [(70000, 3), (4096 + 1, 33), (129, 70), (128, 5), (97, 64), (33, 1), (2, 130)])
@pytest.mark.parametrize("packed", [False, True])
def test_sums_over_rows_are_complete(B, C, packed):
    # alpha = 1 and small whole numbers: every product and sum is exact in fp32, so that a row left out
    # or taken twice shows; every row has a share of its own
    from bayesian_scan_gb300 import kdn
    g = torch.Generator().manual_seed(B)
    draw = lambda lo, hi, *shape: torch.randint(lo, hi + 1, shape, generator=g).float()
    T = 2
    d, go, out, h0 = draw(1, 2, B, T, C), draw(1, 2, B, T, C), draw(1, 3, B, T, C), draw(1, 3, B, C)
    A = torch.zeros(C)
    u = torch.stack([go[:, 0] + go[:, 1], go[:, 1]], 1)
    share = d * u * torch.stack([h0, out[:, 0]], 1)
    assert share.min() >= 1 and share.double().sum((0, 1)).max() < 2 ** 24
    off = torch.arange(0, B * T + 1, T, dtype=torch.int32)
    shaped = (lambda t: t.reshape(1, B * T, C).cuda()) if packed else (lambda t: t.cuda())
    got = kdn.gated_scan_bwd(shaped(d), shaped(d), A.cuda(), shaped(out), shaped(go), h0=h0.cuda(),
                             offsets=off.cuda() if packed else None)
    assert torch.equal(got["A"].cpu(), -share.sum((0, 1)))
    assert torch.equal(got["h0"].cpu(), u[:, 0])


@pytest.mark.parametrize("B,T,Hq,Hk", [(1, 1, 1, 1), (3, 7, 3, 1), (2, 997, 5, 2), (8, 700, 16, 16), (1, 5000, 1, 1)])
def test_sums_of_weights_gradients_are_complete(B, T, Hq, Hk):
    # no norm and no rotation: grad w = sum of x g, whole numbers again
    from bayesian_scan_gb300 import kdn
    g = torch.Generator().manual_seed(T)
    draw = lambda *shape: torch.randint(1, 4, shape, generator=g).float()
    q, k, gq, gk = draw(B, T, Hq, 64), draw(B, T, Hk, 64), draw(B, Hq, T, 64), draw(B, Hk, T, 64)
    got = kdn.qk_norm_rope_bwd(*(t.cuda() for t in (q, k, gq, gk)), norm="none", grad_w=True)
    for n, x, go in (("wq", q, gq), ("wk", k, gk)):
        want = (x * go.transpose(1, 2)).sum((0, 1, 2), dtype=torch.float64)
        assert want.max() < 2 ** 24
        assert torch.equal(got[n].cpu().double(), want)


@pytest.mark.parametrize("leak", [False, True])
@pytest.mark.parametrize("in_dtype", [F32, torch.bfloat16])
def test_what_bf16_states_cost(in_dtype, leak):
    # the gradients from a bf16 forward's own output against those of the states before their rounding:
    # grad d = -A u (h - leak x) moves by A u times the rounding of h, half a step of bf16, and by that of
    # the states that the kernel made (GATE's units); the others do not see it, but grad A does through d
    from bayesian_scan_gb300 import kdn
    g = torch.Generator().manual_seed(9)
    B, T, C = 2, 300, 64
    x = torch.randn(B, 1, T, C, generator=g).to(in_dtype)
    d = torch.nn.functional.softplus(torch.randn(B, 1, T, C, generator=g)).to(in_dtype)
    A = torch.exp(torch.empty(1, C).uniform_(math.log(1e-3), 0.0, generator=g))
    go = torch.randn(B, 1, T, C, generator=g).bfloat16()
    out, _ = kdn.gated_scan_fwd(x.cuda(), d.cuda(), A.cuda(), leak=leak, out_dtype=torch.bfloat16)
    got = kdn.gated_scan_bwd(x.cuda(), d.cuda(), A.cuda(), out, go.cuda(), leak=leak)
    states, _, off, _ = plain64.gated_fwd(x, d, A, None, leak)
    val, err = plain64.gated_bwd(x, d, A, states, go, None, leak)
    u, rounding = torch.zeros(B, 1, C, dtype=torch.float64), torch.zeros_like(states)
    for t in range(T - 1, -1, -1):
        u = torch.exp(-A.double() * d[:, :, t].double()) * (go[:, :, t].double() + u)
        if t:
            off_t = off[:, :, t - 1] + plain64.half_step(torch.bfloat16) * (states[:, :, t - 1].abs() + off[:, :, t - 1])
            rounding[:, :, t] = A.double() * u.abs() * off_t
    plain64.assert_within(got["x"], val["x"], err["x"], "grad_x")
    plain64.assert_within(got["d"], val["d"], err["d"] + rounding, "grad_d")
    plain64.assert_within(got["A"], val["A"], err["A"] + (rounding * d.double() / A.double().unsqueeze(1)).sum((0, 2)),
                          "grad_A")


def test_negative_frequencies_turn_the_other_way():
    # as exact as positive ones: slow and fast, near and far
    inv = -torch.cat([torch.logspace(-9, 0, 40, base=10.0), torch.logspace(0.1, 6, 24, base=10.0)])
    pos = [0, 1, 2, 7, 1001, 65535, -1, -333, 2 ** 31 - 1, -2 ** 31]
    c, s = turned(pos, inv)
    rc, rs = exact(pos, inv)
    for got, ref in ((c, rc), (s, rs)):
        lim = VALUE * ref.abs() + torch.tensor(pos).abs().double()[:, None] * 2.0 ** -60
        assert ((got - ref).abs() <= lim).all(), float(((got - ref).abs() / lim).nan_to_num(0).max())
