"""The gated delta rule on the GPU against its definition in 64 bits, token by
token (delta64.py has the bounds)."""
import pytest
import torch

import delta64

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def kdn():
    from bayesian_scan_gb300 import kdn as k
    return k


def draw(B, H, T, dk, dv, dt, seed, state=False, rows=None, rate=1.0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    unit = lambda x: torch.nn.functional.normalize(x, dim=-1)  # noqa: E731
    x = dict(q=unit(n(B, H, T, dk)).to(dt), k=unit(n(B, H, T, dk)).to(dt), v=n(B, H, T, dv).to(dt),
             beta=torch.sigmoid(n(B, H, T)).to(dt), d=torch.nn.functional.softplus(n(B, H, T)).to(dt),
             A=rate * torch.exp(-6 * torch.rand(H, generator=g)))
    S0 = n(B if rows is None else rows, H, dv, dk) if state else None
    return x, S0, g


def cuda(x):
    return None if x is None else {k: v.cuda() for k, v in x.items()} if isinstance(x, dict) else x.cuda()


# how far a call may be from the 64-bit value beside its bound's fp32 part: what
# the tensor-core form cuts from its operands (see the kernels), 0 for the rest
def split(dk, dv, dt):
    return delta64.SPLIT if dt == BF16 and dk * dv >= 64 * 32 else 0.0


SHAPES = [
    # B, H, T, dk, dv, dtype, out dtype, state
    (1, 1, 1, 16, 16, F32, F32, False), (1, 1, 1, 128, 128, BF16, BF16, True), (2, 3, 2, 32, 64, BF16, F32, True),
    (1, 2, 15, 64, 16, F32, BF16, False), (2, 1, 16, 128, 32, F32, F32, True), (1, 2, 17, 16, 128, BF16, BF16, True),
    (1, 1, 63, 64, 64, F32, F32, True), (2, 2, 64, 128, 128, BF16, F32, False), (1, 3, 65, 128, 128, BF16, F32, True),
    (1, 2, 130, 32, 32, F32, F32, True), (1, 2, 200, 128, 64, BF16, BF16, False), (2, 2, 257, 64, 128, F32, F32, True),
    (3, 1, 129, 128, 128, BF16, BF16, True), (1, 2, 193, 128, 128, F32, F32, False), (1, 1, 640, 128, 128, BF16, F32, True),
    (2, 2, 130, 64, 64, BF16, BF16, True), (1, 3, 65, 64, 64, BF16, F32, True), (2, 33, 29, 64, 128, BF16, BF16, True),
    (1, 2, 100, 32, 128, BF16, BF16, True), (1, 2, 129, 128, 32, BF16, BF16, True), (2, 3, 5, 64, 64, BF16, BF16, True),
    (1, 65, 30, 128, 128, BF16, BF16, True), (3, 2, 1, 128, 128, BF16, BF16, True),
]


@pytest.mark.parametrize("B,H,T,dk,dv,dt,ot,state", SHAPES)
def test_forward(kdn, B, H, T, dk, dv, dt, ot, state):
    x, S0, _ = draw(B, H, T, dk, dv, dt, 7 * T + dk, state)
    val, err = delta64.delta(**x, S0=S0, split=split(dk, dv, dt))
    out, end = kdn.delta_scan_fwd(**cuda(x), S0=cuda(S0), out_dtype=ot)
    assert out.dtype == ot and delta64.far(out, val["out"], err["out"], ot) <= 1
    assert delta64.far(end, val["final"], err["final"]) <= 1


@pytest.mark.parametrize("B,H,T,dk,dv,state", [(1, 2, 2500, 128, 128, True), (1, 1, 2049, 128, 128, False),
                                               (1, 2, 2500, 64, 64, True), (1, 1, 2100, 128, 32, True)])
def test_few_heads_of_long_sequences(kdn, B, H, T, dk, dv, state):
    # cut along the tokens: parts' ends first, then the parts side by side
    x, S0, _ = draw(B, H, T, dk, dv, BF16, T, state, rate=0.05)
    assert kdn.delta_scan_fwd_workspace(B, H, T, dk, dv) > kdn.delta_scan_fwd_workspace(256 * B, H, T, dk, dv) // 256
    val, err = delta64.delta(**x, S0=S0, split=delta64.SPLIT)
    out, end = kdn.delta_scan_fwd(**cuda(x), S0=cuda(S0), out_dtype=F32)
    assert delta64.far(out, val["out"], err["out"]) <= 1 and delta64.far(end, val["final"], err["final"]) <= 1
    for got, want in ((out, val["out"]), (end, val["final"])):
        assert float((got.cpu().double() - want).norm() / want.norm()) < 2e-5


@pytest.mark.parametrize("B,H,T,dk,dv,state", [(1, 2, 2500, 128, 128, True), (1, 1, 2049, 128, 128, False),
                                               (1, 2, 2200, 64, 64, True), (1, 1, 2100, 32, 128, False)])
def test_backward_of_few_heads_of_long_sequences(kdn, B, H, T, dk, dv, state):
    # memories of a few hundred tokens, so that the parts' adjoints count
    x, S0, g = draw(B, H, T, dk, dv, BF16, T, state, rate=0.05)
    assert kdn.delta_scan_bwd_workspace(B, H, T, dk, dv) > kdn.delta_scan_bwd_workspace(256 * B, H, T, dk, dv) // 256
    go = torch.randn(B, H, T, dv, generator=g).to(BF16)
    gf = torch.randn(B, H, dv, dk, generator=g) if state else None
    val, err = delta64.delta(**x, S0=S0, grad_out=go, grad_final=gf, split=delta64.SPLIT)
    got = kdn.delta_scan_bwd(**cuda(x), grad_out=cuda(go), S0=cuda(S0), grad_final_state=cuda(gf))
    for name in ("q", "k", "v", "beta", "d", "A", "S0"):
        dt = BF16 if name in ("q", "k", "v", "beta", "d") else F32
        assert delta64.far(got[name], val[name], err[name], dt) <= 1, name
        # (beside the worst case, as below: roundings of random sign)
        off = float((got[name].cpu().double() - val[name]).norm() / val[name].norm())
        assert off < 2e-5 + (delta64.half_step(BF16) if dt == BF16 else 0.0), (name, off)


@pytest.mark.parametrize("B,H,T,dk,dv,dt,ot,state", SHAPES)
def test_backward(kdn, B, H, T, dk, dv, dt, ot, state):
    x, S0, g = draw(B, H, T, dk, dv, dt, 7 * T + dv, state)
    go = torch.randn(B, H, T, dv, generator=g).to(ot)
    gf = torch.randn(B, H, dv, dk, generator=g) if state else None
    val, err = delta64.delta(**x, S0=S0, grad_out=go, grad_final=gf, split=split(dk, dv, dt))
    got = kdn.delta_scan_bwd(**cuda(x), grad_out=cuda(go), S0=cuda(S0), grad_final_state=cuda(gf))
    for name in ("q", "k", "v", "beta", "d"):
        assert got[name].dtype == dt and delta64.far(got[name], val[name], err[name], dt) <= 1, name
    for name in ("A", "S0"):
        assert got[name].dtype == F32 and delta64.far(got[name], val[name], err[name]) <= 1, name


def test_gradients_are_the_differences():
    # the 64-bit gradients that the others are held to
    x, S0, g = draw(1, 2, 70, 16, 16, torch.float64, 3, True)
    x, S0 = {k: v.double() for k, v in x.items()}, S0.double()
    go, gf = torch.randn(1, 2, 70, 16, generator=g).double(), torch.randn(1, 2, 16, 16, generator=g).double()
    loss = lambda: sum((a * b).sum() for a, b in zip((lambda v: (v["out"], v["final"]))(  # noqa: E731
        delta64.delta(**x, S0=S0)[0]), (go, gf)))
    val, _ = delta64.delta(**x, S0=S0, grad_out=go, grad_final=gf)
    for name, t in (*x.items(), ("S0", S0)):
        way = torch.randn(t.shape, generator=g).double()
        keep, h = t.clone(), 1e-5
        t.copy_(keep + h * way)
        up = loss()
        t.copy_(keep - h * way)
        down = loss()
        t.copy_(keep)
        want = float((val[name] * way).sum())
        # differences: h^2 of the third derivative, and 2^-52 of the loss over h
        assert abs(float(up - down) / (2 * h) - want) < 1e-6 * max(1.0, abs(want)), name


OFFSETS = [[0, 1], [0, 5, 5, 70, 71, 200], [3, 64, 128, 130, 257], [0, 0, 0, 300, 300], [10, 10, 10]]


@pytest.mark.parametrize("offsets", OFFSETS)
@pytest.mark.parametrize("dk,dv,dt", [(64, 32, F32), (128, 128, BF16), (128, 128, F32), (16, 64, BF16), (64, 64, BF16),
                                      (128, 32, BF16)])
def test_packed(kdn, offsets, dk, dv, dt):
    T, H, n = max(offsets[-1], 1) + 7, 2, len(offsets) - 1
    x, S0, g = draw(1, H, T, dk, dv, dt, T, True, n)
    go, gf = torch.randn(1, H, T, dv, generator=g).to(dt), torch.randn(n, H, dv, dk, generator=g)
    for name in ("q", "k", "v", "beta", "d"):                # tokens in no sequence are not read
        x[name][:, :, :offsets[0]] = x[name][:, :, offsets[-1]:] = torch.nan
    go[:, :, :offsets[0]] = go[:, :, offsets[-1]:] = torch.nan
    val, err = delta64.delta(**x, S0=S0, offsets=offsets, grad_out=go, grad_final=gf, split=split(dk, dv, dt))
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    out = torch.full((1, H, T, dv), 7.0, device="cuda")
    y, end = kdn.delta_scan_fwd(**cuda(x), S0=cuda(S0), offsets=off, out=out)
    gone = val["out"].isnan()
    assert y is out and (out.cpu()[gone] == 7).all()         # nor written
    assert delta64.far(out, val["out"], err["out"]) <= 1 and delta64.far(end, val["final"], err["final"]) <= 1
    bufs = {"grad_" + k: torch.full(x[k].shape, 7.0, device="cuda", dtype=dt) for k in ("q", "k", "v", "beta", "d")}
    got = kdn.delta_scan_bwd(**cuda(x), grad_out=cuda(go), S0=cuda(S0), offsets=off, grad_final_state=cuda(gf), **bufs)
    for name in ("q", "k", "v", "beta", "d"):
        assert (got[name].cpu()[val[name].isnan()] == 7).all(), name
        assert delta64.far(got[name], val[name], err[name], dt) <= 1, name
    for name in ("A", "S0"):
        assert delta64.far(got[name], val[name], err[name]) <= 1, name


@pytest.mark.parametrize("dk,dt", [(64, F32), (64, BF16), (128, BF16)])
def test_offsets_out_of_order_stay_in_bounds(kdn, dk, dt):
    # which tokens are whose is unspecified; nothing outside the tensors is touched, and the call returns
    x, _, g = draw(1, 2, 150, dk, dk, dt, 5)
    for offsets in ([-9, 80, 40, 400, 20], [149, 0, 149, 0], [500, 600], [-5, -3, -1]):
        off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        kdn.delta_scan_fwd(**cuda(x), offsets=off)
        kdn.delta_scan_bwd(**cuda(x), grad_out=torch.ones(1, 2, 150, dk, device="cuda", dtype=dt), offsets=off)
    torch.cuda.synchronize()


def test_no_tokens(kdn):
    x, S0, _ = draw(2, 3, 0, 64, 32, BF16, 1, True)
    out, end = kdn.delta_scan_fwd(**cuda(x), S0=S0.cuda())
    assert out.shape == (2, 3, 0, 32) and torch.equal(end.cpu(), S0)
    assert (kdn.delta_scan_fwd(**cuda(x))[1] == 0).all()
    got = kdn.delta_scan_bwd(**cuda(x), grad_out=cuda(x)["v"], S0=S0.cuda(), grad_final_state=2 * S0.cuda())
    assert torch.equal(got["S0"].cpu(), 2 * S0) and (got["A"] == 0).all()
    assert (kdn.delta_scan_bwd(**cuda(x), grad_out=cuda(x)["v"])["S0"] == 0).all()


@pytest.mark.parametrize("dk,dv,dt", [(128, 128, BF16), (64, 128, BF16), (64, 32, F32)])
def test_a_state_handed_on(kdn, dk, dv, dt):
    # prefill, more prefill, single tokens: what one call gives
    x, S0, _ = draw(2, 3, 150, dk, dv, dt, 9, True)
    val, err = delta64.delta(**x, S0=S0, split=split(dk, dv, dt))
    x = cuda(x)
    part = lambda a, b: {k: t if k == "A" else t[:, :, a:b].contiguous() for k, t in x.items()}  # noqa: E731
    outs, S = [], S0.cuda()
    for a, b in ((0, 70), (70, 71), (71, 147)):
        o, S = kdn.delta_scan_fwd(**part(a, b), S0=S, out_dtype=F32)
        outs.append(o)
    for t in range(147, 150):
        one = {k: v if k == "A" else v[:, :, t].contiguous() for k, v in x.items()}
        outs.append(kdn.delta_step(**one, state=S, out_dtype=F32).unsqueeze(2))
    assert delta64.far(torch.cat(outs, 2), val["out"], err["out"]) <= 1
    assert delta64.far(S, val["final"], err["final"]) <= 1


@pytest.mark.parametrize("B,H,dk,dv,dt,ot", [(1, 1, 16, 16, F32, F32), (3, 5, 128, 128, BF16, BF16), (40, 16, 128, 128, BF16, F32),
                                             (2, 3, 64, 16, F32, BF16), (65, 2, 32, 64, BF16, BF16)])
def test_step(kdn, B, H, dk, dv, dt, ot):
    x, S0, _ = draw(B, H, 1, dk, dv, dt, B, True)
    val, err = delta64.delta(**x, S0=S0)
    one = {k: v.cuda() if k == "A" else v[:, :, 0].contiguous().cuda() for k, v in x.items()}
    state, new = S0.cuda(), torch.full_like(S0, 7.0).cuda()
    o = kdn.delta_step(**one, state=state, new_state=new, out_dtype=ot)
    assert torch.equal(state.cpu(), S0)
    assert delta64.far(o.unsqueeze(2), val["out"], err["out"], ot) <= 1 and delta64.far(new, val["final"], err["final"]) <= 1
    assert torch.equal(kdn.delta_step(**one, state=state, out_dtype=ot), o) and torch.equal(state, new)   # in place


@pytest.mark.parametrize("dk,dt", [(128, BF16), (64, BF16), (64, F32)])
def test_gates_at_their_ends(kdn, dk, dt):
    # decays of nothing, of everything and of infinity; betas of 0, 1 and 2
    x, S0, g = draw(1, 2, 200, dk, dk, dt, 11, True)
    d = x["d"].float()
    d[..., ::7], d[..., 3::11], d[..., 100:120] = 0.0, 1e4, 30.0
    x["d"] = d.to(dt)
    x["A"] = torch.tensor([1.0, 0.01])
    x["beta"][..., ::5], x["beta"][..., 1::5], x["beta"][..., 2::13] = 0.0, 1.0, 2.0
    go = torch.randn(1, 2, 200, dk, generator=g).to(dt)
    val, err = delta64.delta(**x, S0=S0, grad_out=go, split=split(dk, dk, dt))
    out, end = kdn.delta_scan_fwd(**cuda(x), S0=S0.cuda(), out_dtype=F32)
    assert delta64.far(out, val["out"], err["out"]) <= 1 and delta64.far(end, val["final"], err["final"]) <= 1
    got = kdn.delta_scan_bwd(**cuda(x), grad_out=go.cuda(), S0=S0.cuda())
    for name in ("q", "k", "v", "beta", "d"):
        assert delta64.far(got[name], val[name], err[name], dt) <= 1, name
    x["d"][..., 50] = torch.inf                              # the state before is gone, and that is all
    cut, _ = delta64.delta(**{k: v if k == "A" else v[:, :, 50:] for k, v in dict(x, d=x["d"].clone().nan_to_num(posinf=1e4)).items()})
    out, end = kdn.delta_scan_fwd(**cuda(x), S0=S0.cuda(), out_dtype=F32)
    assert out.isfinite().all() and delta64.far(out[:, :, 50:], cut["out"], err["out"][:, :, 50:]) <= 1


@pytest.mark.parametrize("at", [0, 37, 63, 64, 150])
@pytest.mark.parametrize("name,value", [("q", torch.nan), ("k", torch.nan), ("k", torch.inf), ("v", torch.nan), ("v", -torch.inf),
                                        ("beta", torch.nan), ("beta", torch.inf), ("d", torch.nan), ("d", -torch.inf)])
@pytest.mark.parametrize("dk,dt", [(128, BF16), (64, BF16), (128, F32)])
def test_what_is_not_finite_spoils_nothing_before_it(kdn, dk, dt, name, value, at):
    # (padding behind a sequence's tokens may hold anything)
    x, S0, _ = draw(1, 2, 200, dk, dk, dt, 23, True)
    val, err = delta64.delta(**x, S0=S0, split=split(dk, dk, dt))
    where = (0, 1, at, 5) if name in "qkv" else (0, 1, at)
    x[name] = x[name].clone()
    x[name][where] = value
    out, end = kdn.delta_scan_fwd(**cuda(x), S0=S0.cuda(), out_dtype=F32)
    clean = torch.ones(1, 2, 200, dk, dtype=torch.bool)
    if name == "q":
        clean[0, 1, at] = False                              # its own outputs
    elif name == "v":
        clean[0, 1, at:, 5] = False                          # its channel from there on
    else:
        clean[0, 1, at:] = False
    fine = torch.where(clean, val["out"], torch.nan)
    assert delta64.far(out, fine, err["out"]) <= 1
    assert not out.cpu()[0, 1, at][..., 5].isfinite() and delta64.far(end[:, :1], val["final"][:, :1], err["final"][:, :1]) <= 1
    if name == "q":
        assert delta64.far(end, val["final"], err["final"]) <= 1
    elif name == "v":
        rest = torch.arange(dk) != 5
        assert delta64.far(end[:, :, rest], val["final"][:, :, rest], err["final"][:, :, rest]) <= 1
        assert not end[0, 1, 5].isfinite().any()
    else:
        assert not end[0, 1].isfinite().any()


@pytest.mark.parametrize("dk,dt", [(128, BF16), (64, BF16), (64, F32)])
def test_same_keys(kdn, dk, dt):
    # one key over and over, beta 1: each write replaces the last one's answer
    x, _, g = draw(1, 1, 150, dk, dk, dt, 13)
    x["k"] = x["k"][:, :, :1].expand_as(x["k"]).contiguous()
    x["beta"] = torch.ones_like(x["beta"])
    go = torch.randn(1, 1, 150, dk, generator=g).to(dt)
    val, err = delta64.delta(**x, grad_out=go, split=split(dk, dk, dt))
    out, _ = kdn.delta_scan_fwd(**cuda(x), out_dtype=F32)
    assert delta64.far(out, val["out"], err["out"]) <= 1
    got = kdn.delta_scan_bwd(**cuda(x), grad_out=go.cuda())
    for name in ("q", "k", "v", "beta", "d"):
        assert delta64.far(got[name], val[name], err[name], dt) <= 1, name


@pytest.mark.parametrize("dk,dt", [(128, BF16), (64, BF16), (64, F32), (128, F32)])
def test_as_exact_as_its_types(kdn, dk, dt):
    # beside the worst case: roundings of random sign.  The fp32 outputs of 700 tokens with memories of up to
    # 400: sums of roots, (272 products)^1/2 x (400 tokens)^1/2 half steps of 2^-24 -> 2e-5
    x, S0, g = draw(1, 4, 700, dk, dk, dt, 17, True)
    go, gf = torch.randn(1, 4, 700, dk, generator=g).to(dt), torch.randn(1, 4, dk, dk, generator=g)
    val, _ = delta64.delta(**x, S0=S0, grad_out=go, grad_final=gf)
    out, end = kdn.delta_scan_fwd(**cuda(x), S0=S0.cuda(), out_dtype=F32)
    got = kdn.delta_scan_bwd(**cuda(x), grad_out=go.cuda(), S0=S0.cuda(), grad_final_state=gf.cuda())
    for name, t in dict(out=out, final=end, **got).items():
        more = delta64.half_step(t.dtype) if t.dtype != F32 else 0.0
        off = float((t.cpu().double() - val[name]).norm() / val[name].norm())
        assert off <= 2e-5 + more, (name, off)


@pytest.mark.parametrize("dk,dv,dt", [(128, 128, BF16), (64, 64, BF16), (64, 32, F32)])
def test_streams_graphs_and_the_same_again(kdn, dk, dv, dt):
    x, S0, g = draw(2, 3, 150, dk, dv, dt, 19, True)
    x, S0 = cuda(x), S0.cuda()
    go = torch.randn(2, 3, 150, dv, generator=g).cuda()
    want, end = kdn.delta_scan_fwd(**x, S0=S0)
    grads = kdn.delta_scan_bwd(**x, grad_out=go.to(dt), S0=S0)
    again, _ = kdn.delta_scan_fwd(**x, S0=S0)
    assert torch.equal(want, again)
    for n, t in kdn.delta_scan_bwd(**x, grad_out=go.to(dt), S0=S0).items():
        assert torch.equal(t, grads[n]), n
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, _ = kdn.delta_scan_fwd(**x, S0=S0, stream=side)
    more = kdn.delta_scan_bwd(**x, grad_out=go.to(dt), S0=S0, stream=side)
    side.synchronize()
    assert torch.equal(out, want) and all(torch.equal(more[n], grads[n]) for n in grads)
    # a step of training captured and replayed on other values
    static = {k: t.clone() for k, t in x.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, e = kdn.delta_scan_fwd(**static, S0=S0)
        gr = kdn.delta_scan_bwd(**static, grad_out=go.to(dt), S0=S0)
    static["v"].mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    other = dict(x, v=2 * x["v"])
    assert torch.equal(o, kdn.delta_scan_fwd(**other, S0=S0)[0])
    for n, t in kdn.delta_scan_bwd(**other, grad_out=go.to(dt), S0=S0).items():
        assert torch.equal(t, gr[n]), n
    # without a workspace the C call takes its own
    import ctypes
    B, H, T = 2, 3, 150
    mine = {n: torch.empty_like(t) for n, t in grads.items()}
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    st = kdn.lib.kdn_delta_scan_bwd(*[p(x[n]) for n in ("q", "k", "v", "beta", "d", "A")], p(S0), None, 0, p(go.to(dt)), None,
                                    *[p(mine[n]) for n in ("q", "k", "v", "beta", "d", "A", "S0")], B, H, T, dk, dv,
                                    int(dt == BF16), int(dt == BF16), None, 0,
                                    ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert st == 0 and all(torch.equal(mine[n], grads[n]) for n in grads)
    assert kdn.get_device_error() == 0
