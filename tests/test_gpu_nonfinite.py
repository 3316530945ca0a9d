"""Infinities and NaN in the gated recurrence and in queries and keys: they
propagate as the definition in IEEE arithmetic has it, and nowhere else."""
import math

import pytest
import torch

import plain64

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
INF, NAN = math.inf, math.nan


def assert_same(got, ref, err, name):
    """Equal where ref is not finite (NaN for NaN, the infinity's sign), else
    within the bound and half a step of got's type."""
    got = got.detach().cpu().double()
    assert torch.equal(got.isnan(), ref.isnan()), f"{name}: NaN in other places"
    odd = ref.isinf()
    assert torch.equal(got.isinf(), odd) and torch.equal(got[odd], ref[odd]), f"{name}: infinities in other places"
    ok = ref.isfinite()
    return got[ok], ref[ok], err[ok]


def assert_within(got, ref, err, name):
    g, r, e = assert_same(got, ref, err, name)
    plain64.assert_within(g.to(got.dtype), r, e, name)


def draw(B, T, C, dtype, rows, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, 1, T, C, generator=g).to(dtype)
    d = torch.nn.functional.softplus(torch.randn(B, 1, T, C, generator=g)).to(dtype)
    # no token's decay underflows (A d < 6), the decay of a warp's, tile's or part's tokens does
    A = torch.exp(torch.empty(1, C).uniform_(math.log(1e-3), 0.0, generator=g))
    h0 = torch.randn(rows, 1, C, generator=g)
    go = torch.randn(B, 1, T, C, generator=g).to(dtype)
    gf = torch.randn(rows, 1, C, generator=g)
    return x, d, A, h0, go, gf


# tiles alone, clusters, parts, packed sequences; every alignment
CASES = [(2, 77, 64, F32, None), (1, 1300, 200, BF16, None), (1, 1300, 201, BF16, None), (1, 9001, 64, F32, None),
         (2, 300, 66, BF16, None), (1, 1500, 40, F32, [0, 1, 1, 40, 700, 1500]), (160, 130, 64, F32, None)]


@pytest.mark.parametrize("B,T,C,dtype,offsets", CASES)
@pytest.mark.parametrize("leak", [False, True])
def test_infinite_states_and_inputs(B, T, C, dtype, offsets, leak):
    from bayesian_scan_gb300 import kdn
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32)
    rows = B if offsets is None else len(offsets) - 1
    x, d, A, h0, _, _ = draw(B, T, C, dtype, rows, T + C)
    h0[:, 0, 3], h0[:, 0, 4], h0[:, 0, 5], h0[0, 0, 6] = INF, -INF, NAN, INF
    x[:, 0, T // 3, 7], x[:, 0, 0, 8] = INF, -INF
    x[:, 0, T // 3, 9], x[:, 0, T // 2, 9] = INF, -INF       # their sum is NaN
    x[:, 0, T // 2, 10] = NAN
    d[:, 0, T // 3, 11] = NAN
    # an infinite gate forgets the state, and makes NaN of an infinite one (to the reference a gate of
    # 2000, whose decay is 0 in 64 bits too)
    A[0, 12:14], h0[:, 0, 13] = 1.0, INF
    gate = d.clone()
    d[:, 0, T // 2, 12:14], gate[:, 0, T // 2, 12:14] = 2000.0, INF
    o, f = kdn.gated_scan_fwd(x.cuda(), gate.cuda(), A.cuda(), h0=h0.cuda(), leak=leak,
                              offsets=None if off is None else off.cuda())
    ro, rf, eo, ef = plain64.gated_fwd(x, d, A, h0, leak, off)
    assert_within(o, ro, eo, "out")
    assert_within(f, rf, ef, "final_state")


@pytest.mark.parametrize("leak", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_step_on_infinite_states(leak, dtype):
    from bayesian_scan_gb300 import kdn
    g = torch.Generator().manual_seed(5)
    B, C = 3, 70
    x, A, state = torch.randn(B, C, generator=g).to(dtype), torch.rand(C, generator=g), torch.randn(B, C, generator=g)
    d = (torch.rand(B, C, generator=g) * 3).to(dtype)        # gates on both sides of 1/2
    state[0, ::2], state[1, ::3], state[2, ::5] = INF, -INF, NAN
    x[0, :8], x[1, :9], d[:, 20] = -INF, -INF, NAN
    ro, rf, eo, ef = plain64.gated_fwd(x[:, None, None], d[:, None, None], A[None], state[:, None], leak)
    s = state.cuda()
    o = kdn.gated_step(x.cuda(), d.cuda(), A.cuda(), s, leak=leak)
    assert_within(o, ro[:, 0, 0], eo[:, 0, 0], "out")
    assert_within(s, rf[:, 0], ef[:, 0], "state")


@pytest.mark.parametrize("B,T,C,dtype,offsets", CASES)
@pytest.mark.parametrize("leak", [False, True])
def test_infinite_gradients(B, T, C, dtype, offsets, leak):
    from bayesian_scan_gb300 import kdn
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32)
    rows = B if offsets is None else len(offsets) - 1
    x, d, A, h0, go, gf = draw(B, T, C, dtype, rows, T + C)
    x, h0 = x.abs() + 0.5, h0.abs() + 0.5                    # without leak, the terms of grad A have one sign
    out = plain64.gated_fwd(x, d, A, h0, leak, off)[0].to(dtype)
    gf[:, 0, 3], gf[:, 0, 4], gf[:, 0, 5] = INF, -INF, NAN
    go[:, 0, T // 3, 7], go[:, 0, T - 1, 8] = INF, -INF
    go[:, 0, T // 3, 9], go[:, 0, T // 2, 9] = INF, -INF
    go[:, 0, T // 2, 10] = NAN
    d[:, 0, T // 3, 11] = NAN
    cu = lambda t: None if t is None else t.cuda()
    got = kdn.gated_scan_bwd(*(t.cuda() for t in (x, d, A, out, go)), h0=h0.cuda(), leak=leak, offsets=cu(off),
                             grad_final_state=gf.cuda())
    val, err = plain64.gated_bwd(x, d, A, out, go, h0, leak, off, gf)
    for n in ("x", "d", "h0", "A"):
        assert_within(got[n], val[n], err[n], "grad_" + n)


@pytest.mark.parametrize("T", [1, 77, 1300, 9001])
@pytest.mark.parametrize("leak", [False, True])
def test_rates_at_the_end_of_the_range(T, leak):
    # such a channel forgets at once, also in its final state and in the gradient of its initial one,
    # whatever lies behind the sequence's end in a tile
    from bayesian_scan_gb300 import kdn
    C = 40
    x, d, A, h0, go, gf = draw(1, T, C, F32, 1, T)
    d = d + 0.01
    A[0, :3] = torch.tensor([2.0 ** 127, 1e38, 3e37])
    o, f = kdn.gated_scan_fwd(x.cuda(), d.cuda(), A.cuda(), h0=h0.cuda(), leak=leak)
    ro, rf, eo, ef = plain64.gated_fwd(x, d, A, h0, leak)
    plain64.assert_within(o, ro, eo, "out")
    plain64.assert_within(f, rf, ef, "final_state")
    got = kdn.gated_scan_bwd(x.cuda(), d.cuda(), A.cuda(), ro.float().cuda(), go.cuda(), h0=h0.cuda(), leak=leak,
                             grad_final_state=gf.cuda())
    val, err = plain64.gated_bwd(x, d, A, ro.float(), go, h0, leak, None, gf)
    for n in ("x", "d", "h0", "A"):
        plain64.assert_within(got[n], val[n], err[n], "grad_" + n)
    s = h0[:, 0].cuda()
    y = kdn.gated_step(x[:, 0, 0].cuda(), d[:, 0, 0].cuda(), A[0].cuda(), s, leak=leak)
    plain64.assert_within(y, ro[:, 0, 0], eo[:, 0, 0], "step")


@pytest.mark.parametrize("dk,rot", [(128, 64), (128, 0), (64, 6), (16, 8), (128, 126), (32, 16)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,T,H", [(1, 5, 3), (2, 701, 32)])
def test_elements_that_do_not_rotate_are_copied(dk, rot, interleaved, B, T, H):
    from bayesian_scan_gb300 import kdn
    g = torch.Generator().manual_seed(dk + rot)
    x, go = torch.randn(B, T, H, dk, generator=g), torch.randn(B, H, T, dk, generator=g)
    w = 1 + torch.rand(dk, generator=g)
    for t in (x, go):
        for i, v in enumerate((INF, NAN, -INF)):
            t.view(-1, dk)[i::7, rot + i % (dk - rot)] = v
    inv = (1e4 ** (-torch.arange(rot // 2) / max(1, rot // 2))).float()
    more = dict(inv_freq=inv.cuda() if rot else None, wq=w.cuda(), norm="none", interleaved=interleaved)
    theta = plain64.rotation_angles(torch.arange(T).expand(1, B, T), inv, None)
    o = kdn.qk_norm_rope_fwd(x.cuda(), None, **more)[0].cpu()
    want = (x * w).transpose(1, 2)                           # one fp32 product: exact
    assert torch.equal(o[..., rot:].isnan(), want[..., rot:].isnan())
    assert torch.equal(o[..., rot:].nan_to_num(0.25, 1e38, -1e38), want[..., rot:].nan_to_num(0.25, 1e38, -1e38))
    ref, err = plain64.qk_fwd(x[..., :rot], w[:rot], theta, rot, interleaved, "none", 0.0)
    plain64.assert_within(o[..., :rot], ref, err)
    got = kdn.qk_norm_rope_bwd(x.cuda(), None, go.cuda(), None, grad_w=True, **more)
    gx, want = got["q"].cpu(), go.transpose(1, 2) * w
    assert torch.equal(gx[..., rot:].isnan(), want[..., rot:].isnan())
    assert torch.equal(gx[..., rot:].nan_to_num(0.25, 1e38, -1e38), want[..., rot:].nan_to_num(0.25, 1e38, -1e38))
    if rot:
        gx64, ex, gw, ew = plain64.qk_bwd(x[..., :rot], w[:rot], go[..., :rot], theta, rot, interleaved, "none", 0.0)
        plain64.assert_within(gx[..., :rot], gx64, ex)
        plain64.assert_within(got["wq"][:rot], gw, ew)
