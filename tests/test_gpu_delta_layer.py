"""The operators of a mixer layer together, as a program runs them: the
residual's addition and its norm, a projection, queries and keys, the gated
delta rule, the way out, and all of it backward; then the same tokens one at a
time from a kept state."""
import pytest
import torch

pytestmark = pytest.mark.gpu

B, T, H, M = 2, 70, 3, 96
G = 4                  # columns of a projection's gates: a row stays a multiple of 16 bytes
INV = (1e4 ** (-torch.arange(16) / 16)).float()
# fp32 operators are within 2e-5 each (tests of their own); five of them follow one another
NEAR = 1e-4


def layer64(x, r, p, dk):
    """The layer from its definitions, in 64 bits; the gradients come from differentiating it."""
    s = x + r
    y = s / torch.sqrt(s.square().mean(-1, keepdim=True) + 1e-6) * p["w1"]
    rows = y @ p["win"]
    q, k, v = (t.unflatten(-1, (H, dk)) for t in rows[..., :3 * H * dk].split(H * dk, -1))
    beta, d = torch.sigmoid(rows[..., 3 * H * dk:3 * H * dk + H]), torch.nn.functional.softplus(rows[..., 3 * H * dk + G:3 * H * dk + G + H])
    turn = torch.arange(x.shape[1], dtype=torch.float64)[:, None] * INV.double()
    c, n = torch.cos(turn)[:, None], torch.sin(turn)[:, None]

    def unit(t):
        t = t / torch.sqrt(t.square().sum(-1, keepdim=True) + 1e-6)
        a, b, rest = t[..., :16], t[..., 16:32], t[..., 32:]
        return torch.cat([a * c - b * n, a * n + b * c, rest], -1)

    q, k = unit(q), unit(k)
    S, outs = torch.zeros(x.shape[0], H, dk, dk, dtype=torch.float64), []
    for t in range(x.shape[1]):
        S = torch.exp(-p["A"] * d[:, t])[..., None, None] * S
        miss = v[:, t].unsqueeze(-1) - S @ k[:, t].unsqueeze(-1)
        S = S + beta[:, t, :, None, None] * miss @ k[:, t].unsqueeze(-2)
        outs.append((S @ q[:, t].unsqueeze(-1)).squeeze(-1))
    o = torch.stack(outs, 1).flatten(-2) @ p["wout"]
    s2 = o + s
    return s2 / torch.sqrt(s2.square().mean(-1, keepdim=True) + 1e-6) * p["w2"], s2


def draw(dk):
    g = torch.Generator().manual_seed(dk)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    p = dict(w1=1 + 0.2 * n(M), w2=1 + 0.2 * n(M), win=n(M, 3 * H * dk + 2 * G) * M ** -0.5,
             wout=n(H * dk, M) * (H * dk) ** -0.5, A=torch.exp(-4 * torch.rand(H, generator=g)))
    return n(B, T, M), n(B, T, M), p, n(B, T, M), n(B, T, M)


def heads_first(t):
    return t.transpose(1, 2).contiguous()


def off(a, b):
    return float((a.detach().cpu().double() - b).norm() / b.norm())


@pytest.mark.parametrize("dk", [32, 64, 128])
def test_layer(dk):
    from bayesian_scan_gb300 import kdn
    x, r, p, gy, gs = draw(dk)
    x64, r64 = x.double().requires_grad_(), r.double().requires_grad_()
    p64 = {k: v.double().requires_grad_() for k, v in p.items()}
    y64, s64 = layer64(x64, r64, p64, dk)
    ((y64 * gy).sum() + (s64 * gs).sum()).backward()

    x, r, gy, gs, inv = x.cuda(), r.cuda(), gy.cuda(), gs.cuda(), INV.cuda()
    p = {k: v.cuda() for k, v in p.items()}
    wide = 3 * H * dk
    y, s, _ = kdn.add_rms_norm_fwd(x, r, weight=p["w1"])
    rows = y @ p["win"]
    q, k, v = (t.unflatten(-1, (H, dk)) for t in rows[..., :wide].split(H * dk, -1))
    qn, kn = kdn.qk_norm_rope_fwd(q, k, inv_freq=inv, norm="l2")
    vn = heads_first(v)
    lb, ld = rows[..., wide:wide + H], rows[..., wide + G:wide + G + H]
    beta, d = heads_first(torch.sigmoid(lb)), heads_first(torch.nn.functional.softplus(ld))
    o, end = kdn.delta_scan_fwd(qn, kn, vn, beta, d, p["A"])
    oo = heads_first(o).flatten(-2)
    y2, s2, _ = kdn.add_rms_norm_fwd(oo @ p["wout"], s, weight=p["w2"])
    assert off(y2, y64.detach()) < NEAR and off(s2, s64.detach()) < NEAR

    g2 = kdn.add_rms_norm_bwd(s2, gy, weight=p["w2"], grad_sum=gs)
    go = heads_first((g2["x"] @ p["wout"].T).unflatten(-1, (H, dk)))
    gd = kdn.delta_scan_bwd(qn, kn, vn, beta, d, p["A"], go)
    grows = torch.zeros_like(rows)
    gq, gk = (t.unflatten(-1, (H, dk)) for t in grows[..., :2 * H * dk].split(H * dk, -1))
    kdn.qk_norm_rope_bwd(q, k, gd["q"], gd["k"], inv_freq=inv, norm="l2", grad_q=gq, grad_k=gk)
    grows[..., 2 * H * dk:wide] = heads_first(gd["v"]).flatten(-2)
    sig = torch.sigmoid(lb)
    grows[..., wide:wide + H] = heads_first(gd["beta"].unsqueeze(-1)).squeeze(-1) * sig * (1 - sig)
    grows[..., wide + G:wide + G + H] = heads_first(gd["d"].unsqueeze(-1)).squeeze(-1) * torch.sigmoid(ld)
    g1 = kdn.add_rms_norm_bwd(s, grows @ p["win"].T, weight=p["w1"], grad_sum=g2["residual"])
    flat = lambda t: t.flatten(0, -2)  # noqa: E731
    got = dict(w1=g1["weight"], w2=g2["weight"], win=flat(y).T @ flat(grows), wout=flat(oo).T @ flat(g2["x"]), A=gd["A"])
    for name, t in got.items():
        assert off(t, p64[name].grad) < NEAR, name
    assert off(g1["x"], x64.grad) < NEAR and off(g1["residual"], r64.grad) < NEAR

    # one token at a time, in a captured step that is replayed with the next token's row and position
    state = torch.zeros(B, H, dk, dk, device="cuda")
    xt, rt, pos = x[:, 0].contiguous(), r[:, 0].contiguous(), torch.zeros(B, 1, dtype=torch.int32, device="cuda")

    def token():
        y, s, _ = kdn.add_rms_norm_fwd(xt, rt, weight=p["w1"])
        row = y @ p["win"]
        q, k, v = (t.unflatten(-1, (H, dk)).unsqueeze(1) for t in row[..., :wide].split(H * dk, -1))
        qn, kn = kdn.qk_norm_rope_fwd(q, k, pos, inv_freq=inv, norm="l2")
        o = kdn.delta_step(qn.squeeze(2), kn.squeeze(2), v.squeeze(1).contiguous(),
                           torch.sigmoid(row[:, wide:wide + H]).contiguous(),
                           torch.nn.functional.softplus(row[:, wide + G:wide + G + H]).contiguous(), p["A"], state)
        return kdn.add_rms_norm_fwd(o.flatten(-2) @ p["wout"], s, weight=p["w2"])[0]

    token()                                                  # (the libraries' first calls are not captured)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = token()
    state.zero_()
    for t in range(T):
        xt.copy_(x[:, t])
        rt.copy_(r[:, t])
        pos.fill_(t)
        graph.replay()
        assert off(out, y64[:, t].detach()) < NEAR, t
    assert off(state, end.cpu().double()) < NEAR
