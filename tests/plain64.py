"""Plain 64-bit forms of the gated recurrence and of the query/key
preparation, written token by token from their definitions, with how far an
fp32 computation may be from each output.

The bounds are running error analyses in units of 2^-24 (half an fp32 step),
carried beside the values:

* A state step h = alpha h' + w x rounds a few times: the gate's alpha = e^z
  is within 4 + 2.5 |z| units of itself (the hardware 2^x 4; the exponent is
  three roundings, of A d, of log2 e and of their product, each at most |z|
  units of e^z, the constant's less than half of one), the polynomial branch
  within 2 of w; the two multiply-adds 2, w x 3, and where tiles are joined
  the decay of a tile adds the roundings of a sum of exponents (at most 16
  units of |z| e^z <= 0.37) and 4 for the 2^x.  GATE = 16 covers all but the
  2.5 |z|, applied to the magnitudes s_t = alpha s' + w |x|; errors of
  earlier tokens decay: E_t = alpha E' + s_t + (2.5 |z| / GATE) alpha s'.
  The hardware 2^x gives 0 below 2^-126, so alpha may be off by that much
  whatever its size (FLUSH, in the same units), and a product below 2^-126
  keeps steps of 2^-149 only.
* A norm's sum of dk squares is within dk/2 units of itself however it is
  ordered (positive terms), its root half of that; products, the weight, the
  rotation (cos and sin within 2) and rsqrt (2) add at most 16: (dk/4 + 16).
* A sum over n terms is within n units of the sum of their magnitudes.

A result rounded to a type adds finfo(type).eps / 2 of itself (bf16 2^-8).
"""
import torch

UNIT = 2.0 ** -24
GATE = 16.0
EXPONENT = 2.5 / GATE
FLUSH = 2.0 ** -126 / (GATE * UNIT)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def spans(offsets, B, T):
    """(state row, batch row, first token, end) of each sequence."""
    if offsets is None:
        return [(b, b, 0, T) for b in range(B)]
    o = [int(v) for v in offsets]
    return [(n, 0, o[n], o[n + 1]) for n in range(len(o) - 1)]


def gated_fwd(x, d, A, h0=None, leak=False, offsets=None):
    """x, d [B,H,T,C], A [H,C], h0 [rows,H,C] or None (any float type).
    Returns (out, final, bound of out, bound of final), fp64; tokens in no
    sequence are NaN in out."""
    x, d, A = x.double(), d.double(), A.double()
    B, H, T, C = x.shape
    sp = spans(offsets, B, T)
    out, err = torch.full_like(x, torch.nan), torch.full_like(x, torch.nan)
    final = torch.zeros(len(sp), H, C, dtype=torch.float64)
    ferr = torch.zeros_like(final)
    for n, b, lo, hi in sp:
        h = torch.zeros(H, C, dtype=torch.float64) if h0 is None else h0[n].double()
        s, e = h.abs(), torch.zeros_like(h)
        for t in range(lo, hi):
            z = -A * d[b, :, t]
            a = torch.exp(z)
            w = -torch.expm1(z) if leak else torch.ones_like(z)
            h = a * h + w * x[b, :, t]
            e = a * e + EXPONENT * z.abs() * a * s + FLUSH * s
            s = a * s + w * x[b, :, t].abs()
            e = e + s
            out[b, :, t], err[b, :, t] = h, GATE * UNIT * e
        final[n], ferr[n] = h, GATE * UNIT * e
    return out, final, err, ferr


def gated_bwd(x, d, A, out, g, h0=None, leak=False, offsets=None, g_final=None):
    """Gradients (dict x, d, A, h0) and their bounds, from the given states."""
    x, d, A, out, g = (t.double() for t in (x, d, A, out, g))
    B, H, T, C = d.shape
    sp = spans(offsets, B, T)
    val = dict(x=torch.full_like(d, torch.nan), d=torch.full_like(d, torch.nan), A=torch.zeros_like(A),
               h0=torch.zeros(len(sp), H, C, dtype=torch.float64))
    err = {k: v.clone() for k, v in val.items()}
    terms = 0
    for n, b, lo, hi in sp:
        u = torch.zeros(H, C, dtype=torch.float64) if g_final is None else g_final[n].double()
        s, e = u.abs(), torch.zeros_like(u)
        for t in range(hi - 1, lo - 1, -1):
            z = -A * d[b, :, t]
            a = torch.exp(z)
            dh, sh, eh = g[b, :, t] + u, g[b, :, t].abs() + s, e
            eh = eh + sh / GATE                     # the addition's rounding
            prev = out[b, :, t - 1] if t > lo else (torch.zeros_like(u) if h0 is None else h0[n].double())
            mag = prev.abs()
            w = torch.ones_like(z)
            if leak:
                w = -torch.expm1(z)
                prev, mag = prev - x[b, :, t], mag + x[b, :, t].abs()
            u, s = a * dh, a * sh
            e = a * eh + s + EXPONENT * z.abs() * s + FLUSH * sh
            val["x"][b, :, t], err["x"][b, :, t] = w * dh, GATE * UNIT * w * (eh + sh)
            val["d"][b, :, t] = -A * u * prev
            err["d"][b, :, t] = GATE * UNIT * A.abs() * (e + s) * mag + A.abs() * 2.0 ** -149
            val["A"] -= d[b, :, t] * u * prev
            err["A"] += UNIT * d[b, :, t].abs() * mag * (GATE * (e + s))
            # the sum's own roundings: below, once the number of terms is known
            err.setdefault("sum", torch.zeros_like(A)).add_(d[b, :, t].abs() * mag * s)
            terms += 1
        val["h0"][n], err["h0"][n] = u, GATE * UNIT * e
    if "sum" in err:
        err["A"] += terms * UNIT * err.pop("sum")
    return val, err


def rotation_angles(pos, inv_freq, axis):
    """[B,T,pairs] fp64 (positions and frequencies are exact in fp64; the
    product is too up to 53 bits)."""
    if len(inv_freq) == 0:
        return torch.zeros(*pos.shape[1:], 0, dtype=torch.float64)
    axis = torch.zeros(len(inv_freq), dtype=torch.long) if axis is None else axis.long()
    return torch.stack([pos[a].double() * f for a, f in zip(axis.tolist(), inv_freq.double())], -1)


def pairs_of(rot, interleaved):
    j = torch.arange(rot)
    return (j[0::2], j[1::2]) if interleaved else (j[:rot // 2], j[rot // 2:])


def norm_scale(x, norm, eps):
    s = x.square().sum(-1, keepdim=True)
    if norm == "none":
        return torch.ones_like(s)
    return 1 / torch.sqrt((s / x.shape[-1] if norm == "rms" else s) + eps)


def qk_fwd(x, w, theta, rot, interleaved, norm, eps):
    """One tensor [B,T,H,dk] -> ([B,H,T,dk], bound)."""
    x = x.double()
    dk = x.shape[-1]
    y = x * norm_scale(x, norm, eps) * (1 if w is None else w.double())
    mag = y.abs()
    if rot:
        i, j = pairs_of(rot, interleaved)
        c, s = torch.cos(theta).unsqueeze(2), torch.sin(theta).unsqueeze(2)
        o, om = y.clone(), mag.clone()
        o[..., i], o[..., j] = y[..., i] * c - y[..., j] * s, y[..., i] * s + y[..., j] * c
        om[..., i] = om[..., j] = mag[..., i] + mag[..., j]
        y, mag = o, om
    return y.transpose(1, 2), ((dk / 4 + 16) * UNIT * mag).transpose(1, 2)


def qk_bwd(x, w, g, theta, rot, interleaved, norm, eps):
    """(grad x, bound, grad w, bound) for one tensor; g [B,H,T,dk]."""
    x, g = x.double(), g.double().transpose(1, 2)
    dk = x.shape[-1]
    wt = torch.ones(dk, dtype=torch.float64) if w is None else w.double()
    gm = g.abs()
    if rot:
        i, j = pairs_of(rot, interleaved)
        c, s = torch.cos(theta).unsqueeze(2), torch.sin(theta).unsqueeze(2)
        o, om = g.clone(), gm.clone()
        o[..., i], o[..., j] = g[..., i] * c + g[..., j] * s, g[..., j] * c - g[..., i] * s
        om[..., i] = om[..., j] = gm[..., i] + gm[..., j]
        g, gm = o, om
    r = norm_scale(x, norm, eps)
    t, tm = g * wt, gm * wt.abs()
    n = dk if norm == "rms" else 1
    gx, gxm = r * t, r * tm
    if norm != "none":
        gx = gx - r ** 3 * x * (t * x).sum(-1, keepdim=True) / n
        gxm = gxm + r ** 3 * x.abs() * (tm * x.abs()).sum(-1, keepdim=True) / n
    k = 3 * (dk / 4 + 16) + dk                       # r cubed, and the sum over the head
    gw, gwm = (r * x * g).sum((0, 1, 2)), (r * x.abs() * gm).sum((0, 1, 2))
    rows = x.shape[0] * x.shape[1] * x.shape[2]
    return gx, k * UNIT * gxm, gw, (dk / 4 + 16 + rows) * UNIT * gwm


def assert_within(got, ref, bound, name=""):
    """|got - ref| <= bound + half a step of got's type, element by element,
    wherever ref is a number."""
    got64 = got.detach().cpu().double()
    assert got64.shape == ref.shape, (name, got64.shape, ref.shape)
    there = ~ref.isnan()
    lim = bound + half_step(got.dtype) * (ref.abs() + bound) + 1e-37
    off = ((got64 - ref).abs() / lim)[there]
    assert off.numel() == 0 or off.isfinite().all(), f"{name}: not finite"
    worst = float(off.max()) if off.numel() else 0.0
    assert worst <= 1.0, f"{name}: {worst:.3g} times the bound"
