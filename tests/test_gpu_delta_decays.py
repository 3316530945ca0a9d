"""The gradients of the delta rule's decays, each relative to its own size.

The gradient of token t's log decay is <G, alpha S_{t-1}>, G the adjoint of
alpha S_{t-1}: all that is read from t on of what was written before it, so it
has alpha as a factor, however large the chunk's other terms are, and so has
its bound here:
    alpha sum_rows [(bS + e M) (|G| + bG) + |S| bG + 4 e M N],
with delta64's symbols (bS, bD: what the states' and adjoints' errors have
carried along; M, N: what their terms add up to; e: one product's error) and
bG = bD + e N + |k| err(l).  4 e M N is the direct sum over the pairs (a writer
before t, a reader from t on): two dots of e, one more for the decay between
them (2^-24 of its exponent and two roundings; 272 units and more are e) and
one for sums of 128 terms and less one after another."""
import pytest
import torch

import delta64
from delta64 import CHUNK, UNIT, _inverse, _norm

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def kdn():
    from bayesian_scan_gb300 import kdn as k
    return k


def decays64(q, k, v, beta, d, A, S0, go, gf, split):
    """(value, bound) of one batch of sequences' grad_d and of their share of grad_A."""
    q, k, v, beta, d, A, go = (t.double() for t in (q, k, v, beta, d, A, go))
    B, H, T, dk = q.shape
    e = delta64.product_error(dk, v.shape[-1], split)
    S, bS, kept = S0.double(), torch.zeros(B, H, v.shape[-1], dtype=torch.float64), []
    nk, nq = _norm(k).unsqueeze(-1), _norm(q).unsqueeze(-1)
    for t in range(T):
        i = t % CHUNK
        if i == 0:
            c = slice(t, min(T, t + CHUNK))
            X = _inverse(k[:, :, c], beta[:, :, c], -A.unsqueeze(-1) * d[:, :, c])
            g, first, zs, M = torch.zeros(B, H, 1, dtype=torch.float64), _norm(S), [], _norm(S)
        z = -A * d[:, :, t]
        al, b = torch.exp(z).unsqueeze(-1), beta[:, :, t, None]
        g = g + z.unsqueeze(-1)
        zs.append(v[:, :, t].abs() + torch.exp(g) * first * nk[:, :, t])
        chunked = zs[i] + sum((X[:, :, i, s, None] * beta[:, :, c.start + s, None] * zs[s] for s in range(i)),
                              torch.zeros_like(zs[i]))
        r = v[:, :, t] - al * (S @ k[:, :, t, :, None]).squeeze(-1)
        er = e * (chunked + v[:, :, t].abs() + al * _norm(S) * nk[:, :, t])
        u, gate = b * r, ((20 + 2.5 * z.abs()) * UNIT).unsqueeze(-1)
        kept.append((S, bS, M, al, gate))
        old = al * _norm(S)
        S = al.unsqueeze(-1) * S + u.unsqueeze(-1) * k[:, :, t, None, :]
        bS = al * bS + b.abs() * nk[:, :, t] * er + gate * (old + u.abs() * nk[:, :, t])
        M = al * M + u.abs() * nk[:, :, t]
    D, bD = gf.double(), torch.zeros_like(bS)
    val, err = torch.zeros(B, H, T, dtype=torch.float64), torch.zeros(B, H, T, dtype=torch.float64)
    vA, eA = torch.zeros(H, dtype=torch.float64), torch.zeros(H, dtype=torch.float64)
    for t in range(T - 1, -1, -1):
        before, b_before, M, al, gate = kept[t]
        if t % CHUNK == CHUNK - 1 or t == T - 1:
            c = slice(t // CHUNK * CHUNK, t + 1)
            X = _inverse(k[:, :, c], beta[:, :, c], -A.unsqueeze(-1) * d[:, :, c])
            zs, N = {}, _norm(D)
        gt, b = go[:, :, t], beta[:, :, t, None]
        N = N + gt.abs() * nq[:, :, t]
        zs[t] = N * nk[:, :, t]
        chunked = zs[t] + sum((X[:, :, s - c.start, t - c.start, None] * beta[:, :, s, None] * zs[s]
                               for s in range(t + 1, c.stop)), torch.zeros_like(zs[t]))
        D = D + gt.unsqueeze(-1) * q[:, :, t, None, :]
        y = (D @ k[:, :, t, :, None]).squeeze(-1)
        ey = e * (chunked + _norm(D) * nk[:, :, t] + gt.abs() * nq[:, :, t] * nk[:, :, t])
        bD = bD + gate * (_norm(D) + gt.abs() * nq[:, :, t])
        lam = b * y
        G = D - lam.unsqueeze(-1) * k[:, :, t, None, :]
        N = N + lam.abs() * nk[:, :, t]
        bG = bD + e * N + b.abs() * nk[:, :, t] * (ey + nk[:, :, t] * bD)
        ga = (al.unsqueeze(-1) * G * before).sum((-1, -2))
        ega = (al * ((b_before + e * M) * (_norm(G) + bG) + _norm(before) * bG + 4 * e * M * N)).sum(-1) + 4 * UNIT * ga.abs()
        val[:, :, t], err[:, :, t] = -A * ga, A.abs() * ega
        vA -= (d[:, :, t] * ga).sum(0)
        eA += (d[:, :, t].abs() * (ega + (T + 64 + B) * UNIT * ga.abs())).sum(0)
        D = al.unsqueeze(-1) * G
        bD = al * bD + al * b.abs() * nk[:, :, t] * ey + gate * (al * _norm(G) + al * lam.abs() * nk[:, :, t])
        N = al * N
    return (val, err), (vA, eA)


def draw(B, H, T, dk, dv, dt, kind, seed, rows=None):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    unit = lambda x: torch.nn.functional.normalize(x, dim=-1)  # noqa: E731
    if kind == "strong":                                     # hardly a memory
        d = 5 + 15 * torch.rand(B, H, T, generator=g)
    else:                                                    # long ones, and tokens that wipe them out, at chunks' ends too
        d = 0.02 * torch.rand(B, H, T, generator=g)
        for t in (0, 20, 63, 64, 65, 100, 127, 150, 192) if kind == "resets" else ():
            d[..., t:t + 1] = 12 + 8 * torch.rand(B, H, 1, generator=g)
    x = dict(q=unit(n(B, H, T, dk)).to(dt), k=unit(n(B, H, T, dk)).to(dt), v=n(B, H, T, dv).to(dt),
             beta=torch.sigmoid(n(B, H, T)).to(dt), d=d.to(dt), A=0.7 + 0.6 * torch.rand(H, generator=g))
    return x, n(rows or B, H, dv, dk), n(B, H, T, dv), n(rows or B, H, dv, dk)


FORMS = [(128, 128, BF16, BF16), (64, 64, BF16, BF16), (32, 128, BF16, BF16), (64, 64, BF16, F32), (128, 128, F32, F32),
         (64, 32, F32, F32), (32, 16, F32, F32), (16, 16, F32, BF16)]


@pytest.mark.parametrize("kind", ["strong", "resets", "long"])
@pytest.mark.parametrize("dk,dv,dt,ot", FORMS)
def test_each_decays_gradient(kdn, dk, dv, dt, ot, kind):
    x, S0, go, gf = draw(2, 2, 200, dk, dv, dt, kind, dk + dv)
    go = go.to(ot)
    split = delta64.SPLIT if dt == BF16 else 0.0
    (val, err), (vA, eA) = decays64(**x, S0=S0, go=go, gf=gf, split=split)
    got = kdn.delta_scan_bwd(**{n: t.cuda() for n, t in x.items()}, grad_out=go.cuda(), S0=S0.cuda(), grad_final_state=gf.cuda())
    far = delta64.far(got["d"], val, err, dt), delta64.far(got["A"], vA, eA)
    assert max(far) <= 1, far


@pytest.mark.parametrize("dk,dt", [(128, BF16), (64, F32)])
def test_of_packed_sequences(kdn, dk, dt):
    cuts = [0, 70, 70, 71, 200]
    x, S0, go, gf = draw(1, 2, 203, dk, dk, dt, "resets", 5, len(cuts) - 1)
    go = go.to(dt)
    got = kdn.delta_scan_bwd(**{n: t.cuda() for n, t in x.items()}, grad_out=go.cuda(), S0=S0.cuda(), grad_final_state=gf.cuda(),
                             offsets=torch.tensor(cuts, dtype=torch.int32, device="cuda"))
    A, bound = 0.0, 0.0
    for n, (lo, hi) in enumerate(zip(cuts, cuts[1:])):
        if lo == hi:
            continue
        part = {m: t if m == "A" else t[:, :, lo:hi] for m, t in x.items()}
        (val, err), (vA, eA) = decays64(**part, S0=S0[n:n + 1], go=go[:, :, lo:hi], gf=gf[n:n + 1],
                                        split=delta64.SPLIT if dt == BF16 else 0.0)
        assert delta64.far(got["d"][:, :, lo:hi], val, err, dt) <= 1, n
        A, bound = A + vA, bound + eA
    assert delta64.far(got["A"], A, bound) <= 1


def test_few_heads_of_long_sequences(kdn):
    # cut along the tokens: the parts' first states and adjoints come from folds
    x, S0, go, gf = draw(1, 1, 2200, 128, 128, BF16, "resets", 6)
    x["d"][..., 1000::300] = 15.0
    go = go.to(BF16)
    (val, err), (vA, eA) = decays64(**x, S0=S0, go=go, gf=gf, split=delta64.SPLIT)
    got = kdn.delta_scan_bwd(**{n: t.cuda() for n, t in x.items()}, grad_out=go.cuda(), S0=S0.cuda(), grad_final_state=gf.cuda())
    assert delta64.far(got["d"], val, err, BF16) <= 1 and delta64.far(got["A"], vA, eA) <= 1


@pytest.mark.parametrize("kind", ["strong", "resets", "long"])
def test_the_values_are_delta64s(kind):
    x, S0, go, gf = draw(2, 2, 70, 16, 16, F32, kind, 3)
    want, _ = delta64.delta(**x, S0=S0, grad_out=go, grad_final=gf)
    (val, _), (vA, _) = decays64(**x, S0=S0, go=go, gf=gf, split=0.0)
    assert torch.allclose(val, want["d"], rtol=1e-9, atol=0) and torch.allclose(vA, want["A"], rtol=1e-9, atol=0)
