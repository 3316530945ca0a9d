"""What the gated recurrence and the query/key preparation refuse, before any
CUDA call: the C ABI with addresses that only host checks see, and the
binding's own checks."""
import ctypes

import pytest
import torch

FAKE = 0x10000


@pytest.fixture(scope="module")
def kdn():
    from bayesian_scan_gb300 import build
    build.build()
    from bayesian_scan_gb300 import kdn as k
    return k


def vp(x):
    return None if x is None else ctypes.c_void_p(x)


def fwd(kdn, x=FAKE, x_ld=64, d=FAKE, d_ld=64, A=FAKE, h0=None, off=None, nseq=0, leak=0, out=FAKE, fs=None,
        B=1, H=1, T=8, C=64, it=1, ot=1):
    return kdn.lib.kdn_gated_scan_fwd(vp(x), x_ld, vp(d), d_ld, vp(A), vp(h0), vp(off), nseq, leak, vp(out),
                                      vp(fs), B, H, T, C, it, ot, None)


def bwd(kdn, x=FAKE, x_ld=64, d=FAKE, d_ld=64, A=FAKE, h0=None, off=None, nseq=0, leak=1, out=FAKE, go=FAKE,
        gf=None, gx=FAKE, gd=FAKE, gA=FAKE, gh0=None, B=1, H=1, T=8, C=64, it=1, ot=1, ws=None, n=0):
    return kdn.lib.kdn_gated_scan_bwd(vp(x), x_ld, vp(d), d_ld, vp(A), vp(h0), vp(off), nseq, leak, vp(out),
                                      vp(go), vp(gf), vp(gx), vp(gd), vp(gA), vp(gh0), B, H, T, C, it, ot,
                                      vp(ws), n, None)


SIZES = [
    (dict(B=0), -1), (dict(H=0), -1), (dict(T=-1), -1), (dict(C=0), -1), (dict(A=None), -1),
    (dict(it=2), -2), (dict(ot=-1), -2), (dict(x_ld=63), -1), (dict(d_ld=63), -1), (dict(x_ld=-64), -1),
    (dict(off=FAKE), -1), (dict(off=FAKE, nseq=-1), -1), (dict(nseq=3), -1), (dict(off=FAKE, nseq=3, B=2), -1),
    (dict(off=FAKE + 2, nseq=3), -1), (dict(x=FAKE + 1), -1), (dict(d=FAKE + 2, it=0), -1), (dict(A=FAKE + 2), -1),
    (dict(h0=FAKE + 1), -1), (dict(out=FAKE + 2, ot=0), -1),
    (dict(T=0x7fffffff), -1), (dict(C=(1 << 28) + 1, x_ld=1 << 29, d_ld=1 << 29), -1),
    (dict(B=1 << 30, H=1 << 30), -1), (dict(x_ld=1 << 60, T=1 << 20), -1), (dict(B=1 << 15, H=1 << 15, T=1 << 30, C=64), -1),
]


@pytest.mark.parametrize("field", ["x", "d", "A", "out"])
def test_fwd_null(kdn, field):
    assert fwd(kdn, **{field: None}) == -1


@pytest.mark.parametrize("field", ["x", "d", "A", "out", "go", "gx", "gd"])
def test_bwd_null(kdn, field):
    assert bwd(kdn, **{field: None}) == -1


@pytest.mark.parametrize("kw,status", SIZES)
def test_scan_rejects(kdn, kw, status):
    assert fwd(kdn, **kw) == status
    assert bwd(kdn, **kw) == status


def test_bwd_rejects_more(kdn):
    for f in ("gf", "gA", "gh0"):
        assert bwd(kdn, **{f: FAKE + 2}) == -1
    assert bwd(kdn, gx=FAKE + 1) == -1 and bwd(kdn, go=FAKE + 1) == -1
    assert bwd(kdn, ws=FAKE + 16, n=1 << 30) == -1 and bwd(kdn, B=2, ws=FAKE, n=8) == -1


def test_workspaces(kdn):
    n = ctypes.c_longlong(-1)
    f = kdn.lib.kdn_gated_scan_bwd_workspace
    assert f(2, 3, 100, 64, 0, ctypes.byref(n)) == 0 and n.value >= 2 * 3 * 64 * 4
    assert f(1, 3, 100, 64, 5, ctypes.byref(n)) == 0 and n.value >= 5 * 3 * 64 * 4
    for bad in ((1, 1, 0x7fffffff, 1, 0), (1, 1, 1, 1 << 29, 0), (0, 1, 1, 1, 0), (1, 0, 1, 1, 0), (1, 1, -1, 1, 0), (1, 1, 1, 0, 0), (2, 1, 1, 1, 3), (1, 1, 1, 1, -1)):
        assert f(*bad, ctypes.byref(n)) == -1
    assert f(1, 1, 1, 1, 0, None) == -1
    f = kdn.lib.kdn_qk_norm_rope_bwd_workspace
    assert f(2, 100, 4, 4, 64, ctypes.byref(n)) == 0 and n.value >= 2 * 64 * 4
    assert f(2, 100, 4, 4, 65, ctypes.byref(n)) == -2
    for bad in ((1, 1, 1 << 25, 1, 64), (0, 1, 1, 1, 64), (1, -1, 1, 1, 64), (1, 1, 0, 0, 64), (1, 1, -1, 2, 64)):
        assert f(*bad, ctypes.byref(n)) == -1
    with pytest.raises(kdn.KdnError):
        kdn.gated_scan_bwd_workspace(0, 1, 1, 1)
    with pytest.raises(kdn.KdnError):
        kdn.qk_norm_rope_bwd_workspace(1, 1, 1, 1, 24)


def step(kdn, x=FAKE, d=FAKE, A=FAKE, s=FAKE, n=FAKE, out=FAKE, B=1, H=1, C=8, it=1, ot=1):
    return kdn.lib.kdn_gated_step(vp(x), vp(d), vp(A), 0, vp(s), vp(n), vp(out), B, H, C, it, ot, None)


@pytest.mark.parametrize("kw,status", [
    *((({f: None}), -1) for f in ("x", "d", "A", "s", "n", "out")),
    (dict(B=0), -1), (dict(H=0), -1), (dict(C=-1), -1), (dict(it=7), -2), (dict(ot=2), -2), (dict(x=FAKE + 1), -1),
    (dict(s=FAKE + 2), -1), (dict(n=FAKE + 1), -1), (dict(out=FAKE + 2, ot=0), -1),
    (dict(B=1 << 30, H=1 << 30, C=1 << 30), -1),
])
def test_step_rejects(kdn, kw, status):
    assert step(kdn, **kw) == status


def qk(kdn, q=FAKE, q_ld=128, k=FAKE, k_ld=64, wq=None, wk=None, norm=1, eps=1e-6, pos=FAKE, axes=1, inv=FAKE,
       axis=None, rot=64, inter=0, qo=FAKE, ko=FAKE, B=1, T=4, Hq=2, Hk=1, dk=64, it=1, ot=1):
    return kdn.lib.kdn_qk_norm_rope_fwd(vp(q), q_ld, vp(k), k_ld, vp(wq), vp(wk), norm, eps, vp(pos), axes, vp(inv),
                                        vp(axis), rot, inter, vp(qo), vp(ko), B, T, Hq, Hk, dk, it, ot, None)


def qk_back(kdn, q=FAKE, q_ld=128, k=FAKE, k_ld=64, wq=None, wk=None, norm=1, eps=1e-6, pos=FAKE, axes=1, inv=FAKE,
            axis=None, rot=64, inter=0, qo=FAKE, ko=FAKE, gq=FAKE, gq_ld=128, gk=FAKE, gk_ld=64, gwq=FAKE, gwk=None,
            B=1, T=4, Hq=2, Hk=1, dk=64, it=1, ot=1, ws=None, n=0):
    return kdn.lib.kdn_qk_norm_rope_bwd(vp(q), q_ld, vp(k), k_ld, vp(wq), vp(wk), norm, eps, vp(pos), axes, vp(inv),
                                        vp(axis), rot, inter, vp(qo), vp(ko), vp(gq), gq_ld, vp(gk), gk_ld, vp(gwq),
                                        vp(gwk), B, T, Hq, Hk, dk, it, ot, vp(ws), n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), -1), (dict(k=None), -1), (dict(qo=None), -1), (dict(ko=None), -1), (dict(B=0), -1), (dict(T=-1), -1),
    (dict(Hq=0, Hk=0), -1), (dict(Hq=-1), -1), (dict(dk=48), -2), (dict(dk=256), -2), (dict(it=2), -2), (dict(ot=3), -2),
    (dict(norm=3), -2), (dict(norm=-1), -2), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1), (dict(rot=63), -1),
    (dict(rot=66), -1), (dict(rot=-2), -1), (dict(inv=None), -1), (dict(axes=0), -1), (dict(axes=5), -1),
    (dict(q_ld=127), -1), (dict(q_ld=132), -1), (dict(k_ld=56), -1), (dict(q=FAKE + 8), -1), (dict(ko=FAKE + 4), -1),
    (dict(wq=FAKE + 4), -1), (dict(pos=FAKE + 2), -1), (dict(axis=FAKE + 1), -1), (dict(inv=FAKE + 2), -1),
    (dict(q_ld=1 << 59, T=1 << 20), -1), (dict(Hq=1 << 25, q_ld=1 << 31), -1),
])
def test_qk_rejects(kdn, kw, status):
    assert qk(kdn, **kw) == status
    assert qk_back(kdn, **kw) == status


def test_qk_back_rejects_more(kdn):
    for kw in (dict(gq=None), dict(gk=None), dict(gq_ld=120), dict(gk_ld=68), dict(gq=FAKE + 2), dict(gwq=FAKE + 2),
               dict(ws=FAKE + 8, n=1 << 30), dict(ws=FAKE, n=4)):
        assert qk_back(kdn, **kw) == -1
    # nothing to do: no tokens
    assert qk(kdn, T=0, q=None, k=None, qo=None, ko=None) == 0
    assert qk_back(kdn, T=0, q=None, k=None, qo=None, ko=None, gq=None, gk=None, gwq=None) == 0


def test_binding_rejects_scan(kdn):
    x, A = torch.zeros(2, 5, 8), torch.zeros(8)
    f = kdn.gated_scan_fwd
    for args, kw, match in [
        ((x.half(), x.half(), A), {}, "bf16 or fp32"),
        ((x, x.bfloat16(), A), {}, "d must be"),
        ((x, x[:, :4], A), {}, "d must have shape"),
        ((x, x, torch.zeros(7)), {}, "A must have shape"),
        ((x, x, A.double()), {}, "A must be"),
        ((x[0], x[0], A), {}, "x must be"),
        ((x.transpose(1, 2), x.transpose(1, 2), torch.zeros(5)), {}, "adjacent"),
        ((x.transpose(0, 1), x.transpose(0, 1), A), {}, "rows must follow|adjacent"),
        ((x, x, A), dict(h0=torch.zeros(2, 7)), "h0 must have shape"),
        ((x, x, A), dict(offsets=torch.zeros(3, dtype=torch.int32)), "B = 1"),
        ((x[:1], x[:1], A), dict(offsets=torch.zeros(3)), "offsets must be"),
        ((x[:1], x[:1], A), dict(offsets=torch.zeros(1, dtype=torch.int32)), "offsets must be"),
        ((x, x, A), dict(out=torch.zeros(2, 5, 9)), "out must have shape"),
        ((x, x, A), dict(out=x.double()), "out must be"),
        ((x, x, A), dict(out=x.clone(), out_dtype=torch.bfloat16), "out must be"),
        ((x, x, A), dict(final_state=torch.zeros(8)), "final_state must have shape"),
        ((x, x, A), {}, "must be a CUDA tensor"),
    ]:
        with pytest.raises(ValueError, match=match):
            f(*args, **kw)
    b = kdn.gated_scan_bwd
    for args, kw, match in [
        ((x, x, A, x, x.bfloat16()), {}, "grad_out must be"),
        ((x, x, A, x[:, :4].contiguous(), x), {}, "out must have shape"),
        ((x, x, A, x, x), dict(grad_final_state=torch.zeros(2, 9)), "grad_final_state must have shape"),
        ((x, x, A, x, x), dict(grad_x=x.bfloat16()), "grad_x must be"),
        ((x, x, A, x, x), dict(grad_A=torch.zeros(9)), "grad_A must have shape"),
        ((x, x, A, x, x), dict(workspace=torch.zeros(1, dtype=torch.uint8)), "workspace must hold"),
        ((x, x, A, x, x), {}, "must be a CUDA tensor"),
    ]:
        with pytest.raises(ValueError, match=match):
            b(*args, **kw)
    y, s = torch.zeros(3, 8), torch.zeros(3, 8)
    for args, kw, match in [
        ((y[0], y[0], A, s), {}, "x must be"),
        ((y, y.bfloat16(), A, s), {}, "d must be"),
        ((y, y, A, s.double()), {}, "state must be"),
        ((y, y, A, s), dict(new_state=torch.zeros(3, 7)), "new_state must have shape"),
        ((y, y, A, s), {}, "must be a CUDA tensor"),
    ]:
        with pytest.raises(ValueError, match=match):
            kdn.gated_step(*args, **kw)


def test_binding_rejects_qk(kdn):
    q, f = torch.zeros(2, 5, 3, 32), torch.ones(16)
    pos = torch.zeros(2, 5, dtype=torch.int32)
    for args, kw, match in [
        ((None, None), {}, "q or k"),
        ((q[0], q), {}, r"\[B,T,H,dk\]"),
        ((q, q[:, :4]), {}, "k must be"),
        ((q, q.bfloat16()), {}, "k must be"),
        ((q.half(), q.half()), {}, "bf16 or fp32"),
        ((q.transpose(1, 2).contiguous().transpose(1, 2), q), {}, "side by side"),
        ((q, q), dict(norm="max"), "norm must be"),
        ((q, q), dict(wq=torch.ones(31)), "wq must have shape"),
        ((q, q), dict(inv_freq=torch.ones(17)), "inv_freq must be"),
        ((q, q), dict(pos=pos), "need inv_freq"),
        ((q, q), dict(pos=pos.long(), inv_freq=f), "pos must be"),
        ((q, q), dict(pos=pos[:, :4], inv_freq=f), "pos must"),
        ((q, q), dict(pos=pos.expand(5, 2, 5), inv_freq=f), "1 to 4 axes"),
        ((q, q), dict(pos=pos, inv_freq=f, axis=torch.zeros(15, dtype=torch.int32)), "axis must have shape"),
        ((q, q), dict(q_out=torch.zeros(2, 5, 3, 32)), "q_out must have shape"),
        ((q, q), dict(q_out=torch.zeros(2, 3, 5, 32), k_out=torch.zeros(2, 3, 5, 32).bfloat16()), "one type"),
        ((q, q), {}, "must be a CUDA tensor"),
    ]:
        with pytest.raises(ValueError, match=match):
            kdn.qk_norm_rope_fwd(*args, **kw)
    g = torch.zeros(2, 3, 5, 32)
    for args, kw, match in [
        ((q, q, g, None), {}, "grad_k_out must be given"),
        ((q, q, g[:, :2].contiguous(), g), {}, "grad_q_out must have shape"),
        ((q, q, g, g.bfloat16()), {}, "one type"),
        ((q, q, g.half(), g.half()), {}, "bf16 or fp32"),
        ((q, q, g, g), dict(grad_q=q[:, :, :2]), "heads"),
        ((q, q, g, g), dict(grad_q=q.bfloat16()), "grad_q must be"),
        ((q, q, g, g), dict(grad_w=True, workspace=torch.zeros(1, dtype=torch.uint8)), "workspace must hold"),
        ((q, q, g, g), {}, "must be a CUDA tensor"),
    ]:
        with pytest.raises(ValueError, match=match):
            kdn.qk_norm_rope_bwd(*args, **kw)


def test_workspace_sizes_are_the_current_device_s(kdn, monkeypatch):
    # a call on another device's tensors is refused, and leaves no size of the current device under the other's name
    class On:
        is_cuda = True

        def get_device(self):
            return 1

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    assert kdn._ws_device(On()) == 0
    assert kdn._ws_device(torch.zeros(1)) == -1
