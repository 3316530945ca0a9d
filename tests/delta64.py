"""The gated delta rule and its gradients in 64 bits, token by token from the
definition, with how far the library may be from each output.

Norms of rows (over d_k) carry the bounds.  Write e for the relative error of
one product of two operands (a sum of n products in fp32 is within n units of
2^-24 of the sum of their magnitudes; the tensor-core form adds what it cuts
from its operands), z_t = -A d_t for a log decay.

* The transition S -> alpha S (1 - beta k k^T) has norm <= 1 (alpha <= 1, beta
  |k|^2 <= 2), so an error that a token makes is carried on but not enlarged:
      bS_t = alpha bS_{t-1} + beta |k| err(r_t) + gate (alpha |S| + |u| |k|),
  gate = (16 + 2.5 |z|) 2^-24 as for the gated recurrence (plain64.py), plus 4
  units for the update's own roundings.
* err(r_t) = e (|v_t| + alpha |S_{t-1}| |k|) token by token.  In chunks of 64,
  r = z + T (beta z) with z_s = v_s - e^{g_s} S0 k_s: e (|z_t| + sum_s |T_ts|
  beta_s |z_s|), where |z_s| stands for |v_s| + e^{g_s} |S0| |k_s|.
* An output of a chunk is a sum over the chunk's first state and its tokens:
  M_t = e^{g_t} |S0| + sum_{s <= t} e^{g_t - g_s} |u_s| |k_s| is what its terms
  add up to, err(o_t) = bS_t |q| + e M_t |q|.
* The adjoint D walks back with the same transition: bD, N and err(y) alike.
  (Its u is beta y.)
* Gradients are products of r, y, S, D and the inputs; each factor's error times
  the other's magnitude, plus e times the magnitudes.  The gradient of a log
  decay is a sum over the rest of its chunk, and so is its bound.

The tensor-core form (``split`` > 0) has fp16 pairs for operands, scaled by
powers of two to below 2^14: an element is off by 2^-22 of itself, three
products leave out one of 2^-22 (SPLIT covers both, and those of products of
products), or by 2^-25 / 2^13 = 2^-38 of the largest element of its tile or
state row, which is more for what strong decays make small beside the rest of
its chunk.  A sum of up to 128 such products is then off by 2^-31 of the largest
product; for P, which is scaled by a bound of its largest, 2^-5 max|k| max|q| in
place of 2^-13 of that, a sum of 64 by 2^-24 max|k| max|q| max|u|.  A token's bound
is at least e times its own largest product, e > 2^-16, so 2^-8 of the largest
bound among a sequence's tokens covers both (FLOOR).

A result rounded to a type adds half a step of itself.
"""
import torch

UNIT = 2.0 ** -24
CHUNK = 64
SPLIT = 2.0 ** -20
FLOOR = 2.0 ** -8


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def spans(offsets, B, T):
    if offsets is None:
        return [(b, b, 0, T) for b in range(B)]
    o = [int(v) for v in offsets]
    return [(n, 0, o[n], o[n + 1]) for n in range(len(o) - 1)]


def product_error(dk, dv, split=0.0):
    """e: sums over at most max(dk, dv) + 2 x 64 products, 16 roundings more."""
    return (max(dk, dv) + 2 * CHUNK + 16) * UNIT + split


def _norm(x):
    return x.norm(dim=-1)


def _inverse(k, beta, z):
    """|T| of a chunk: T = -G (1 + beta G)^-1, row after row."""
    C = k.shape[-2]
    g = z.cumsum(-1)
    E = torch.exp((g.unsqueeze(-1) - g.unsqueeze(-2)).tril()).tril(-1)
    G = (k @ k.transpose(-1, -2)) * E
    T = torch.zeros_like(G)
    for t in range(C):
        T[..., t, :] = -G[..., t, :] - ((G[..., t, :] * beta).unsqueeze(-2) @ T).squeeze(-2)
    return T.abs()


def delta(q, k, v, beta, d, A, S0=None, offsets=None, grad_out=None, grad_final=None, split=0.0):
    """Inputs of any float type on the CPU.  Returns (values, bounds): dicts of
    fp64 tensors out, final, and with grad_out q, k, v, beta, d, A, S0; NaN for
    tokens in no sequence."""
    q, k, v, beta, d, A = (t.double() for t in (q, k, v, beta, d, A))
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    e = product_error(dk, dv, split)
    sp = spans(offsets, B, T)
    nan = lambda *s: torch.full(s, torch.nan, dtype=torch.float64)  # noqa: E731
    val = dict(out=nan(B, H, T, dv), final=nan(len(sp), H, dv, dk))
    err = dict(out=nan(B, H, T, dv), final=nan(len(sp), H, dv, dk))
    if grad_out is not None:
        go = grad_out.double()
        for x in (val, err):
            x.update(q=nan(B, H, T, dk), k=nan(B, H, T, dk), v=nan(B, H, T, dv), beta=nan(B, H, T), d=nan(B, H, T),
                     A=torch.zeros(H, dtype=torch.float64), S0=nan(len(sp), H, dv, dk))
    for n, b, lo, hi in sp:
        S = torch.zeros(H, dv, dk, dtype=torch.float64) if S0 is None else S0[n].double()
        bS = torch.zeros(H, dv, dtype=torch.float64)
        kept = []
        for t in range(lo, hi):
            kt, qt, vt, bt = k[b, :, t], q[b, :, t], v[b, :, t], beta[b, :, t, None]
            z = -A * d[b, :, t]
            al = torch.exp(z).unsqueeze(-1)
            nk, nq = _norm(kt).unsqueeze(-1), _norm(qt).unsqueeze(-1)
            if (t - lo) % CHUNK == 0:
                c = slice(t, min(hi, t + CHUNK))
                X = _inverse(k[b, :, c], beta[b, :, c], (-A.unsqueeze(-1) * d[b, :, c]))
                g = torch.zeros(H, 1, dtype=torch.float64)
                first, zs, M = _norm(S), [], _norm(S)
            g = g + z.unsqueeze(-1)
            zs.append(vt.abs() + torch.exp(g) * first * nk)
            i = t - lo - (t - lo) // CHUNK * CHUNK
            chunked = zs[i] + sum((X[:, i, s, None] * beta[b, :, c.start + s, None] * zs[s] for s in range(i)),
                                  torch.zeros_like(zs[i]))
            r = vt - al * (S @ kt.unsqueeze(-1)).squeeze(-1)
            er = e * (chunked + vt.abs() + al * _norm(S) * nk)
            u = bt * r
            gate = ((20 + 2.5 * z.abs()) * UNIT).unsqueeze(-1)
            old = al * _norm(S)
            before, b_before = S, bS
            S = al.unsqueeze(-1) * S + u.unsqueeze(-1) * kt.unsqueeze(-2)
            bS = al * bS + bt.abs() * nk * er + gate * (old + u.abs() * nk)
            M = al * M + u.abs() * nk
            val["out"][b, :, t] = (S @ qt.unsqueeze(-1)).squeeze(-1)
            err["out"][b, :, t] = (bS + e * M) * nq
            er = er + al * nk * b_before
            kept.append((before, S, b_before, bS, r, er, M, al, z, gate))
        val["final"][n] = S
        err["final"][n] = bS.unsqueeze(-1).expand_as(S)
        if split and hi > lo:
            err["out"][b, :, lo:hi] += FLOOR * err["out"][b, :, lo:hi].amax((1, 2), keepdim=True)
        if grad_out is None:
            continue
        D = torch.zeros(H, dv, dk, dtype=torch.float64) if grad_final is None else grad_final[n].double()
        bD = torch.zeros(H, dv, dtype=torch.float64)
        for t in range(hi - 1, lo - 1, -1):
            before, S, b_before, bS, r, er, M, al, z, gate = kept[t - lo]
            kt, qt, gt, bt = k[b, :, t], q[b, :, t], go[b, :, t], beta[b, :, t, None]
            nk, nq = _norm(kt).unsqueeze(-1), _norm(qt).unsqueeze(-1)
            at_end = (t - lo) % CHUNK == CHUNK - 1 or t == hi - 1
            if at_end:
                c = slice(lo + (t - lo) // CHUNK * CHUNK, t + 1)
                X = _inverse(k[b, :, c], beta[b, :, c], (-A.unsqueeze(-1) * d[b, :, c]))
                first, zs, N = _norm(D), {}, _norm(D)
                g = torch.zeros(H, 1, dtype=torch.float64)
                # of <D1, S1> and of the tokens behind this one in the chunk
                rest = (first * (bS + e * M) + bD * _norm(S)).sum(-1)
                tail = (D * S).sum((-1, -2))
                gsum = torch.zeros(H, dtype=torch.float64)
            # what du is a sum of: the tokens of the chunk behind this one and the adjoint behind it
            N = N + gt.abs() * nq
            zs[t] = N * nk
            chunked = zs[t] + sum((X[:, s - c.start, t - c.start, None] * beta[b, :, s, None] * zs[s]
                                   for s in range(t + 1, c.stop)), torch.zeros_like(zs[t]))
            D = D + gt.unsqueeze(-1) * qt.unsqueeze(-2)
            y = (D @ kt.unsqueeze(-1)).squeeze(-1)
            ey = e * (chunked + _norm(D) * nk + gt.abs() * nq * nk)
            bD = bD + gate * (_norm(D) + gt.abs() * nq)
            u, lam = bt * r, bt * y
            eyy = ey + nk * bD
            val["q"][b, :, t] = (S.transpose(-1, -2) @ gt.unsqueeze(-1)).squeeze(-1)
            eq = (gt.abs() * (bS + e * M)).sum(-1)
            val["beta"][b, :, t] = (y * r).sum(-1)
            err["beta"][b, :, t] = (y.abs() * er + r.abs() * eyy + er * eyy).sum(-1) + e * (y * r).abs().sum(-1)
            val["v"][b, :, t] = lam
            err["v"][b, :, t] = bt.abs() * eyy + 2 * UNIT * lam.abs()
            a = al.unsqueeze(-1)
            val["k"][b, :, t] = ((D.transpose(-1, -2) @ u.unsqueeze(-1)) - ((a * before).transpose(-1, -2)
                                                                          @ lam.unsqueeze(-1))).squeeze(-1)
            w = bt.abs()
            ek_write = (w * (r.abs() * (bD + e * N) + er * (_norm(D) + bD))).sum(-1)
            ek_read = (w * (y.abs() * (al * b_before + e * M) + eyy * al * (_norm(before) + b_before))).sum(-1)
            err["q"][b, :, t] = eq.unsqueeze(-1)
            err["k"][b, :, t] = (ek_write + ek_read).unsqueeze(-1)
            # the log decay: <G, M> with G the adjoint of alpha S_{t-1}
            G = D - lam.unsqueeze(-1) * kt.unsqueeze(-2)
            ga = (G * (a * before)).sum((-1, -2))
            nq1, nk1 = nq.squeeze(-1), nk.squeeze(-1)
            gsum = gsum + (nq1 * eq + nk1 * (ek_write + ek_read)
                           + e * (nq1 * (gt.abs() * M).sum(-1) + nk1 * (w * (r.abs() * N + y.abs() * M)).sum(-1)))
            eg = rest + gsum
            val["d"][b, :, t] = -A * ga
            err["d"][b, :, t] = A.abs() * (eg + 2 * UNIT * ga.abs())
            val["A"] -= d[b, :, t] * ga
            err["A"] += d[b, :, t].abs() * (eg + (hi - lo + 64 + len(sp)) * UNIT * ga.abs())
            D = a * G
            bD = al * bD + al * bt.abs() * nk * ey + gate * (al * _norm(G) + al * lam.abs() * nk)
            N = al * N + al * lam.abs() * nk
        val["S0"][n] = D
        err["S0"][n] = bD.unsqueeze(-1).expand_as(D)
        if split and hi > lo:
            for name in ("q", "k", "v", "beta", "d"):
                part = err[name][b, :, lo:hi]
                part += FLOOR * part.flatten(1).amax(1).view(-1, *[1] * (part.dim() - 1))
    return val, err


def far(got, val, err, dtype=torch.float32):
    """The largest error over its bound, and whether what is NaN in val is all that is."""
    got = got.detach().cpu().double()
    there = ~val.isnan()
    assert got[there].isfinite().all()
    bound = err[there] + half_step(dtype) * (val[there].abs() + err[there]) + 1e-30
    return float(((got - val)[there].abs() / bound).max()) if there.any() else 0.0
