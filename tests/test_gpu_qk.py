"""Queries and keys for the scans (kdn_qk_norm_rope_fwd, _bwd) against their
64-bit plain form, and the whole mixer they belong to: preparation, scan,
gated recurrence, forward, backward and one token at a time."""
import pytest
import torch

import plain64
from bayesian_scan_gb300 import workloads

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
TYPES = [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)]


def draw(B, T, Hq, Hk, dk, dtype, seed=0, rot=None, axes=1, far=5000, slices=True):
    g = torch.Generator().manual_seed(seed)
    rows = torch.randn(B, T, (Hq + 2 * Hk + 1) * dk, generator=g).to(dtype)
    rows = rows if slices else rows[..., :(Hq + Hk) * dk].contiguous()
    rot = dk if rot is None else rot
    s = dict(rows=rows, wq=1 + 0.3 * torch.randn(dk, generator=g), wk=torch.randn(dk, generator=g),
             inv_freq=(1e4 ** (-torch.arange(rot // 2) / max(1, rot // 2))).float(),
             pos=torch.randint(-far, far, (axes, B, T), generator=g, dtype=torch.int64).to(torch.int32),
             axis=torch.randint(0, axes, (rot // 2,), generator=g, dtype=torch.int64).to(torch.int32),
             gq=torch.randn(B, Hq, T, dk, generator=g), gk=torch.randn(B, Hk, T, dk, generator=g))
    return s


def split(rows, Hq, Hk, dk):
    q = rows[..., :Hq * dk].unflatten(2, (Hq, dk))
    k = rows[..., Hq * dk:(Hq + Hk) * dk].unflatten(2, (Hk, dk))
    return q, k


def check(s, Hq, Hk, dk, out_dtype, norm, interleaved=False, weight=True, eps=1e-6, pos=True, axis=True):
    from bayesian_scan_gb300 import kdn
    q, k = split(s["rows"], Hq, Hk, dk)
    dq, dk_ = split(s["rows"].cuda(), Hq, Hk, dk)
    B, T = q.shape[:2]
    rot = 2 * len(s["inv_freq"])
    p = s["pos"] if pos else torch.arange(T).expand(1, B, T)
    theta = plain64.rotation_angles(p, s["inv_freq"], s["axis"] if axis else None)
    w = {n: s["w" + n] if weight else None for n in "qk"}
    cu = lambda t: None if t is None else t.cuda()
    more = dict(pos=cu(s["pos"]) if pos and rot else None, inv_freq=cu(s["inv_freq"]) if rot else None,
                wq=cu(w["q"]), wk=cu(w["k"]), norm=norm, eps=eps, axis=cu(s["axis"]) if axis and rot else None,
                interleaved=interleaved)
    oq, ok = kdn.qk_norm_rope_fwd(dq, dk_, out_dtype=out_dtype, **more)
    for name, x, o in (("q", q, oq), ("k", k, ok)):
        ref, err = plain64.qk_fwd(x, w[name], theta, rot, interleaved, norm, eps)
        plain64.assert_within(o, ref, err, name)
    gq, gk = s["gq"].to(out_dtype), s["gk"].to(out_dtype)
    got = kdn.qk_norm_rope_bwd(dq, dk_, gq.cuda(), gk.cuda(), grad_w=True, **more)
    for name, x, g in (("q", q, gq), ("k", k, gk)):
        gx, ex, gw, ew = plain64.qk_bwd(x, w[name], g, theta, rot, interleaved, norm, eps)
        plain64.assert_within(got[name], gx, ex, "grad_" + name)
        plain64.assert_within(got["w" + name], gw, ew, "grad_w" + name)


@pytest.mark.parametrize("in_dtype,out_dtype", TYPES)
@pytest.mark.parametrize("norm", ["rms", "l2", "none"])
@pytest.mark.parametrize("dk", [16, 32, 64, 128])
def test_types_and_norms(dk, norm, in_dtype, out_dtype):
    for interleaved in (False, True):
        s = draw(2, 5, 3, 2, dk, in_dtype, seed=dk, axes=3)
        check(s, 3, 2, dk, out_dtype, norm, interleaved)


@pytest.mark.parametrize("dk,rot", [(128, 64), (128, 2), (128, 96), (64, 32), (64, 6), (32, 0), (16, 8), (128, 126),
                                    (16, 14)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_part_of_a_head_rotates(dk, rot, interleaved):
    s = draw(2, 7, 2, 3, dk, F32, seed=rot, rot=rot, axes=2)
    check(s, 2, 3, dk, F32, "rms", interleaved)
    s = draw(1, 3, 1, 1, dk, BF16, seed=rot, rot=rot)
    check(s, 1, 1, dk, BF16, "l2", interleaved, weight=False)


@pytest.mark.parametrize("B,T,Hq,Hk", [(1, 1, 1, 1), (1, 1, 16, 16), (130, 1, 4, 4), (1, 333, 5, 1), (3, 70, 32, 8),
                                       (2, 1027, 1, 1)])
@pytest.mark.parametrize("dk", [64, 128])
def test_sizes(B, T, Hq, Hk, dk):
    s = draw(B, T, Hq, Hk, dk, BF16, seed=T, axes=1)
    check(s, Hq, Hk, dk, BF16, "rms")
    check(s, Hq, Hk, dk, F32, "l2", interleaved=True, weight=False, pos=False, axis=False)
    s = draw(B, T, Hq, Hk, dk, F32, seed=T, axes=4, slices=False)
    check(s, Hq, Hk, dk, F32, "rms")


@pytest.mark.parametrize("dk,Hq,Hk", [(128, 19, 2), (128, 2, 33), (64, 5, 4), (32, 8, 9), (16, 33, 17), (64, 4, 0)])
@pytest.mark.parametrize("in_dtype,out_dtype", [(BF16, F32), (F32, BF16)])
def test_many_tokens(dk, Hq, Hk, in_dtype, out_dtype):
    # tokens enough for the bulk copies; heads that end inside a warp's step and inside a copy
    from bayesian_scan_gb300 import kdn
    B, T = 2, 701
    for interleaved, rot in ((False, dk), (True, dk - 2), (False, dk // 2)):
        s = draw(B, T, Hq, max(Hk, 1), dk, in_dtype, seed=dk + Hq, rot=rot, axes=2)
        q, k = split(s["rows"], Hq, max(Hk, 1), dk)
        dq, dk_ = split(s["rows"].cuda(), Hq, max(Hk, 1), dk)
        theta = plain64.rotation_angles(s["pos"], s["inv_freq"], s["axis"])
        oq, ok = kdn.qk_norm_rope_fwd(dq, dk_ if Hk else None, s["pos"].cuda(), s["inv_freq"].cuda(), s["wq"].cuda(),
                                      s["wk"].cuda(), axis=s["axis"].cuda(), interleaved=interleaved,
                                      out_dtype=out_dtype)
        for x, o, w in ((q, oq, s["wq"]), (k, ok, s["wk"])) if Hk else ((q, oq, s["wq"]),):
            ref, err = plain64.qk_fwd(x, w, theta, rot, interleaved, "rms", 1e-6)
            plain64.assert_within(o, ref, err)
    assert kdn.get_device_error() == kdn.KDN_OK


def test_far_positions():
    # the angle of a far position keeps its accuracy: up to 2^31 - 1, and behind zero
    s = draw(2, 64, 2, 1, 128, F32, seed=1, axes=2)
    s["pos"] = torch.randint(-2**31, 2**31, (2, 2, 64), generator=torch.Generator().manual_seed(2)).to(torch.int32)
    s["pos"][0, 0, :4] = torch.tensor([2**31 - 1, -2**31, 0, -1], dtype=torch.int32)
    q, k = split(s["rows"], 2, 1, 128)
    from bayesian_scan_gb300 import kdn
    dq, dk = split(s["rows"].cuda(), 2, 1, 128)
    oq, ok = kdn.qk_norm_rope_fwd(dq, dk, pos=s["pos"].cuda(), inv_freq=s["inv_freq"].cuda(),
                                  axis=s["axis"].cuda(), norm="l2")
    # the fixed-point frequency f / 2 pi is a double, off by 2^-54 of itself at most (f <= 1: 2^-56.6
    # turns), so the angle by |pos| 2^-56.6 2 pi <= 2^-22.9 at the farthest; the 64-bit reference's
    # product pos * f is off by 2^-53 of itself (2^31: 2^-22).  Both shift (y1, y2) by that much of |y|.
    theta = plain64.rotation_angles(s["pos"], s["inv_freq"], s["axis"])
    for x, o in ((q, oq), (k, ok)):
        ref, err = plain64.qk_fwd(x, None, theta, 128, False, "l2", 1e-6)
        size = x.double().norm(dim=-1).transpose(1, 2).unsqueeze(-1).reciprocal() * x.double().abs().transpose(1, 2)
        i, j = plain64.pairs_of(128, False)
        both = size.clone()
        both[..., i] = both[..., j] = size[..., i] + size[..., j]
        plain64.assert_within(o, ref, err + (2 ** -22.9 + 2 ** -22) * both)


def test_axis_out_of_range_is_clamped_and_zero_rows():
    from bayesian_scan_gb300 import kdn
    s = draw(1, 9, 2, 2, 64, F32, seed=3, axes=2)
    dq, dk = split(s["rows"].cuda(), 2, 2, 64)
    more = dict(pos=s["pos"].cuda(), inv_freq=s["inv_freq"].cuda())
    wild = torch.where(s["axis"] > 0, 1 << 20, -5).to(torch.int32)
    a = kdn.qk_norm_rope_fwd(dq, dk, axis=wild.cuda(), **more)
    b = kdn.qk_norm_rope_fwd(dq, dk, axis=s["axis"].cuda(), **more)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    s["rows"][:, 4] = 0                                   # a token of zeros stays zero, its gradient finite
    for norm in ("rms", "l2"):
        check(s, 2, 2, 64, F32, norm)


def test_no_eps():
    # without eps 1 / sqrt(0) is infinite; it stays with rows of zeros, of which there are none here,
    # and not with the places of a warp that have no row
    for B, T, Hq, Hk in ((1, 3, 3, 1), (1, 1, 1, 1), (1, 5, 7, 2)):
        s = draw(B, T, Hq, Hk, 16, F32, seed=T)
        check(s, Hq, Hk, 16, F32, "rms", eps=0.0)
        s = draw(B, T, Hq, Hk, 128, BF16, seed=T)
        check(s, Hq, Hk, 128, F32, "l2", eps=0.0)


def test_one_tensor_alone_and_slices_written():
    from bayesian_scan_gb300 import kdn
    s = draw(2, 11, 3, 2, 32, BF16, seed=4)
    dq, dk = split(s["rows"].cuda(), 3, 2, 32)
    more = dict(pos=s["pos"].cuda(), inv_freq=s["inv_freq"].cuda())
    oq, ok = kdn.qk_norm_rope_fwd(dq, dk, **more)
    assert torch.equal(kdn.qk_norm_rope_fwd(dq, None, **more)[0], oq)
    assert torch.equal(kdn.qk_norm_rope_fwd(None, dk, **more)[1], ok)
    gq, gk = s["gq"].cuda(), s["gk"].cuda()
    ref = kdn.qk_norm_rope_bwd(dq, dk, gq, gk, grad_w=True, **more)
    alone = kdn.qk_norm_rope_bwd(None, dk, None, gk, **more)
    assert alone["q"] is None and alone["wk"] is None and torch.equal(alone["k"], ref["k"])
    # the fused projection's gradient, written in place; the columns between are left alone
    fused = torch.full_like(s["rows"].cuda(), 5.0)
    fq, fk = split(fused, 3, 2, 32)
    got = kdn.qk_norm_rope_bwd(dq, dk, gq, gk, grad_q=fq, grad_k=fk, grad_w=True, **more)
    assert torch.equal(fq, ref["q"]) and torch.equal(fk, ref["k"]) and (fused[..., 5 * 32:] == 5.0).all()
    assert torch.equal(got["wq"], ref["wq"]) and torch.equal(got["wk"], ref["wk"])


def test_no_tokens():
    from bayesian_scan_gb300 import kdn
    q = torch.empty(2, 0, 3, 64, device="cuda")
    f = torch.ones(32, device="cuda")
    oq, ok = kdn.qk_norm_rope_fwd(q, q, inv_freq=f)
    assert oq.shape == (2, 3, 0, 64)
    g = kdn.qk_norm_rope_bwd(q, q, oq, ok, inv_freq=f, grad_w=True)
    assert (g["wq"] == 0).all() and (g["wk"] == 0).all()


def test_repeats_streams_and_graphs():
    from bayesian_scan_gb300 import kdn
    s = draw(2, 301, 4, 4, 128, BF16, seed=5)
    rows = s["rows"].cuda()
    dq, dk = split(rows, 4, 4, 128)
    gq, gk = s["gq"].cuda(), s["gk"].cuda()
    more = dict(pos=s["pos"].cuda(), inv_freq=s["inv_freq"].cuda(), wq=s["wq"].cuda(), wk=s["wk"].cuda())

    def both():
        g = kdn.qk_norm_rope_bwd(dq, dk, gq, gk, **more)
        return [*kdn.qk_norm_rope_fwd(dq, dk, **more), g["q"], g["k"], g["wq"], g["wk"]]

    first = both()
    assert all(torch.equal(a, b) for a, b in zip(first, both()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = both()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = both()
        graphs.append((graph, held))
    rows.mul_(0.5)
    again = both()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for (graph, _), st in zip(graphs, streams):
        with torch.cuda.stream(st):
            graph.replay()
    torch.cuda.synchronize()
    for _, held in graphs:
        assert all(torch.equal(a, b) for a, b in zip(again, held))


def mixer64(rows, wq, wk, d, beta, A, gx, gA, theta, Hq, dk, dv):
    """The mixer in 64 bits, differentiable: preparation, metaplastic scan,
    readout through the gated recurrence (head layout)."""
    q, k = split(rows, Hq, Hq, dk)
    v = rows[..., 2 * Hq * dk:].unflatten(2, (Hq, dv)).transpose(1, 2)
    c, s = torch.cos(theta).unsqueeze(2), torch.sin(theta).unsqueeze(2)

    def prepare(x, w, norm):
        y = x * plain64.norm_scale(x, norm, 1e-6) * w
        i, j = plain64.pairs_of(dk, False)
        return torch.cat([y[..., i] * c - y[..., j] * s, y[..., i] * s + y[..., j] * c], -1).transpose(1, 2)

    q, k = prepare(q, wq, "l2"), prepare(k, wk, "l2")
    B, H, T, _ = q.shape
    I = torch.ones(B, H, dv, dk, dtype=torch.float64)
    eta = torch.zeros_like(I)
    outs, h = [], torch.zeros(B, H, dv, dtype=torch.float64)
    for t in range(T):
        a = torch.exp(-A[:, None, None] * d[:, :, t, None, None])
        kt, bt = k[:, :, t, None, :], beta[:, :, t, :, None]
        I = a * I + (1 - a) + bt * kt ** 2
        eta = a * eta + bt * v[:, :, t, :, None] * kt
        o = (eta / I * q[:, :, t, None, :]).sum(-1)
        g = torch.exp(-gA * gx[:, :, t])
        h = g * h + (1 - g) * o
        outs.append(h)
    return torch.stack(outs, 2)


def test_mixer_forward_backward_and_decode():
    """Preparation, diagonal scan and gated recurrence as one layer: forward,
    gradients against automatic differentiation of the 64-bit layer, and the
    same tokens one at a time."""
    from bayesian_scan_gb300 import kdn
    B, T, H, dk, dv = 2, 45, 2, 64, 64
    g = torch.Generator().manual_seed(6)
    rows = torch.randn(B, T, 2 * H * dk + H * dv, generator=g)
    _, _, _, beta, d, A = workloads.draw_diag(B, H, T, dk, dv, F32, ("uniform", 0.1, 1.0), gen=g)
    wq, wk = 1 + 0.2 * torch.randn(dk, generator=g), 1 + 0.2 * torch.randn(dk, generator=g)
    gx = torch.nn.functional.softplus(torch.randn(B, H, T, dv, generator=g))
    gA = torch.rand(H, dv, generator=g)
    pos = torch.arange(T, dtype=torch.int32).expand(1, B, T) + 4000
    inv = (1e4 ** (-torch.arange(dk // 2) / (dk // 2))).float()
    leaves = [t.double().requires_grad_() for t in (rows, wq, wk, d, beta, A, gx, gA)]
    ref = mixer64(*leaves, plain64.rotation_angles(pos, inv, None), H, dk, dv)
    go = torch.randn(ref.shape, generator=g)
    ref.backward(go.double())

    rows, wq, wk, d, beta, A, gx, gA, pos, inv, go = (t.cuda() for t in (rows, wq, wk, d, beta, A, gx, gA, pos, inv, go))
    pos = pos.contiguous()
    q_in, k_in = split(rows, H, H, dk)
    v = rows[..., 2 * H * dk:].unflatten(2, (H, dv)).transpose(1, 2).contiguous()
    prep = dict(pos=pos, inv_freq=inv, wq=wq, wk=wk, norm="l2")
    q, k = kdn.qk_norm_rope_fwd(q_in, k_in, **prep)
    o, fs = kdn.diag_scan_fwd(q, k, v, beta, d, A)
    h, hf = kdn.gated_scan_fwd(o, gx, gA, leak=True)
    gs = kdn.gated_scan_bwd(o, gx, gA, h, go, leak=True)
    ds = kdn.diag_scan_bwd(q, k, v, beta, d, A, gs["x"])
    qs = kdn.qk_norm_rope_bwd(q_in, k_in, ds["q"], ds["k"], **prep)
    grad_rows = torch.cat([qs["q"].flatten(2), qs["k"].flatten(2), ds["v"].transpose(1, 2).flatten(2)], -1)
    got = [grad_rows, qs["wq"], qs["wk"], ds["d"], ds["beta"], ds["A"], gs["d"], gs["A"]]

    def rel(a, b):
        return float((a.cpu().double() - b).norm() / b.norm())

    # the scan's backward holds 2e-4; the other operators' steps are far below it
    assert rel(h, ref.detach()) < 2e-5
    for a, leaf in zip(got, leaves):
        assert rel(a, leaf.grad) < 2e-4
    # one token at a time, from the states after 20 tokens
    cut = 20
    o1, fs1 = kdn.diag_scan_fwd(*(t[:, :, :cut].contiguous() for t in (q, k, v, beta, d)), A)
    _, hs = kdn.gated_scan_fwd(o1, gx[:, :, :cut].contiguous(), gA, leak=True)
    for t in range(cut, T):
        q1, k1 = kdn.qk_norm_rope_fwd(q_in[:, t:t + 1], k_in[:, t:t + 1], **dict(prep, pos=pos[:, :, t:t + 1].contiguous()))
        o1 = kdn.diag_step(q1[:, :, 0].contiguous(), k1[:, :, 0].contiguous(), v[:, :, t].contiguous(),
                           beta[:, :, t].contiguous(), d[:, :, t].contiguous(), A, fs1)
        h1 = kdn.gated_step(o1, gx[:, :, t].contiguous(), gA, hs, leak=True)
        assert rel(h1, ref.detach()[:, :, t]) < 2e-5
