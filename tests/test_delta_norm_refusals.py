"""What the gated delta rule and the residual's addition with its norm refuse,
before any CUDA call: the C ABI with addresses that only host checks see, and
the binding's own checks."""
import ctypes

import pytest
import torch

FAKE = 0x10000
BIG = 2 ** 32 + 5      # cut to 32 bits: 5


@pytest.fixture(scope="module")
def kdn():
    from bayesian_scan_gb300 import build
    build.build()
    from bayesian_scan_gb300 import kdn as k
    return k


def vp(x):
    return None if x is None else ctypes.c_void_p(x)


def fwd(kdn, q=FAKE, k=FAKE, v=FAKE, beta=FAKE, d=FAKE, A=FAKE, S0=None, off=None, nseq=0, out=FAKE, fs=None, B=1, H=2,
        T=8, dk=64, dv=32, it=1, ot=1, ws=None, n=0):
    return kdn.lib.kdn_delta_scan_fwd(vp(q), vp(k), vp(v), vp(beta), vp(d), vp(A), vp(S0), vp(off), nseq, vp(out), vp(fs),
                                      B, H, T, dk, dv, it, ot, vp(ws), n, None)


def bwd(kdn, q=FAKE, k=FAKE, v=FAKE, beta=FAKE, d=FAKE, A=FAKE, S0=None, off=None, nseq=0, out=FAKE, fs=None, gq=FAKE,
        gk=FAKE, gv=FAKE, gb=FAKE, gd=FAKE, gA=FAKE, gS=None, B=1, H=2, T=8, dk=64, dv=32, it=1, ot=1, ws=None, n=0):
    return kdn.lib.kdn_delta_scan_bwd(vp(q), vp(k), vp(v), vp(beta), vp(d), vp(A), vp(S0), vp(off), nseq, vp(out), vp(fs),
                                      vp(gq), vp(gk), vp(gv), vp(gb), vp(gd), vp(gA), vp(gS), B, H, T, dk, dv, it, ot,
                                      vp(ws), n, None)


def step(kdn, q=FAKE, k=FAKE, v=FAKE, beta=FAKE, d=FAKE, A=FAKE, S0=FAKE, fs=FAKE, out=FAKE, B=1, H=2, dk=64, dv=32, it=1,
         ot=1):
    return kdn.lib.kdn_delta_step(vp(q), vp(k), vp(v), vp(beta), vp(d), vp(A), vp(S0), vp(fs), vp(out), B, H, dk, dv, it,
                                  ot, None)


ROWS = [
    (dict(B=0), -1), (dict(H=0), -1), (dict(it=2), -2), (dict(ot=-1), -2), (dict(dk=48), -2), (dict(dv=256), -2),
    (dict(q=FAKE + 8), -1), (dict(k=FAKE + 4), -1), (dict(beta=FAKE + 1), -1), (dict(d=FAKE + 2, it=0), -1),
    (dict(A=FAKE + 2), -1), (dict(S0=FAKE + 8), -1), (dict(fs=FAKE + 4), -1), (dict(out=FAKE + 1), -1),
    (dict(B=1 << 30, H=1 << 30), -1),
]
SCAN = [
    (dict(T=-1), -1), (dict(T=0x7fffffff), -1), (dict(v=FAKE + 8), -1), (dict(out=FAKE + 8), -1), (dict(off=FAKE), -1),
    (dict(off=FAKE, nseq=-1), -1), (dict(nseq=3), -1), (dict(off=FAKE, nseq=3, B=2), -1), (dict(off=FAKE + 2, nseq=3), -1),
    (dict(B=1 << 15, H=1 << 15, T=1 << 30), -1),
]


@pytest.mark.parametrize("kw,status", ROWS + SCAN)
def test_scan_rejects(kdn, kw, status):
    assert fwd(kdn, **kw) == status
    assert bwd(kdn, **kw) == status


@pytest.mark.parametrize("kw,status", ROWS)
def test_step_rejects(kdn, kw, status):
    assert step(kdn, **kw) == status


@pytest.mark.parametrize("field", ["q", "k", "v", "beta", "d", "A", "out"])
def test_null(kdn, field):
    assert fwd(kdn, **{field: None}) == -1
    assert bwd(kdn, **{field: None}) == -1
    assert step(kdn, **{field: None}) == -1


def test_more(kdn):
    for f in ("gq", "gk", "gv", "gb", "gd"):
        assert bwd(kdn, **{f: None}) == -1
    for f in ("gq", "gk", "gv", "gS"):
        assert bwd(kdn, **{f: FAKE + 8}) == -1
    assert bwd(kdn, gb=FAKE + 1) == -1 and bwd(kdn, gA=FAKE + 2) == -1
    assert step(kdn, S0=None) == -1 and step(kdn, fs=None) == -1 and step(kdn, v=FAKE + 1) == -1
    assert bwd(kdn, ws=FAKE + 16, n=1 << 30) == -1 and bwd(kdn, ws=FAKE, n=8) == -1
    assert fwd(kdn, ws=FAKE + 16, n=1 << 30) == -1


def test_workspaces(kdn):
    for f in (kdn.lib.kdn_delta_scan_fwd_workspace, kdn.lib.kdn_delta_scan_bwd_workspace):
        n = ctypes.c_longlong(-1)
        assert f(2, 3, 100, 64, 32, 0, 1, ctypes.byref(n)) == 0 and n.value >= 0
        assert f(1, 3, 100, 64, 32, 4, 0, ctypes.byref(n)) == 0
        for bad, status in (((0, 1, 1, 16, 16, 0, 0), -1), ((1, 0, 1, 16, 16, 0, 0), -1), ((1, 1, -1, 16, 16, 0, 0), -1),
                            ((1, 1, 1, 24, 16, 0, 0), -2), ((1, 1, 1, 16, 8, 0, 0), -2), ((1, 1, 1, 16, 16, -1, 0), -1),
                            ((2, 1, 1, 16, 16, 3, 0), -1), ((1, 1, 1, 16, 16, 0, 2), -2)):
            assert f(*bad, ctypes.byref(n)) == status
        assert f(1, 1, 1, 16, 16, 0, 0, None) == -1
    assert kdn.delta_scan_bwd_workspace(2, 3, 0, 64, 64) == 0
    # the states and adjoints of chunks of 64 tokens and two rows a token
    assert kdn.delta_scan_bwd_workspace(2, 3, 128, 64, 32, dtype=torch.float32) >= 2 * 6 * 2 * 64 * 32 * 4 + 2 * 6 * 128 * 32 * 4
    n = ctypes.c_longlong(-1)
    f = kdn.lib.kdn_add_rms_norm_bwd_workspace
    assert f(100, 64, ctypes.byref(n)) == 0 and n.value >= 64 * 4
    assert f(0, 64, ctypes.byref(n)) == 0
    for bad in ((-1, 64), (4, 0), (4, (1 << 28) + 1), (1 << 31, 64)):
        assert f(*bad, ctypes.byref(n)) == -1
    assert f(4, 64, None) == -1


def norm(kdn, x=FAKE, ld=64, r=FAKE, w=FAKE, eps=1e-6, s=FAKE, y=FAKE, scale=None, rows=4, C=64, xt=1, rt=1, yt=1):
    return kdn.lib.kdn_add_rms_norm_fwd(vp(x), ld, vp(r), vp(w), eps, vp(s), vp(y), vp(scale), rows, C, xt, rt, yt, None)


def norm_back(kdn, s=FAKE, w=FAKE, eps=1e-6, gy=FAKE, gs=None, gr=FAKE, gx=None, gw=FAKE, rows=4, C=64, xt=1, rt=1, yt=1,
              ws=None, n=0):
    return kdn.lib.kdn_add_rms_norm_bwd(vp(s), vp(w), eps, vp(gy), vp(gs), vp(gr), vp(gx), vp(gw), rows, C, xt, rt, yt, vp(ws),
                                        n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), -1), (dict(y=None), -1), (dict(s=None), -1), (dict(r=None), -1), (dict(r=None, s=None, rt=0), -1),
    (dict(rows=-1), -1), (dict(rows=1 << 31), -1), (dict(C=0), -1), (dict(C=1 << 29, ld=1 << 29), -1), (dict(ld=63), -1), (dict(ld=1 << 59), -1),
    (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1), (dict(xt=2), -2), (dict(rt=2), -2), (dict(yt=3), -2),
    (dict(yt=2), -1), (dict(scale=FAKE), -1), (dict(yt=2, scale=FAKE + 2), -1), (dict(x=FAKE + 1), -1),
    (dict(r=FAKE + 2, rt=0), -1), (dict(s=FAKE + 1), -1), (dict(y=FAKE + 1), -1), (dict(w=FAKE + 2), -1),
])
def test_norm_rejects(kdn, kw, status):
    assert norm(kdn, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(s=None), -1), (dict(gy=None), -1), (dict(gr=None, gw=None), -1), (dict(rows=-1), -1), (dict(C=0), -1),
    (dict(eps=-1.0), -1), (dict(xt=2), -2), (dict(rt=2), -2), (dict(yt=2), -2), (dict(s=FAKE + 1), -1),
    (dict(gy=FAKE + 1), -1), (dict(gs=FAKE + 1), -1), (dict(gr=FAKE + 1), -1), (dict(gx=FAKE + 1), -1),
    (dict(gw=FAKE + 2), -1), (dict(w=FAKE + 1), -1), (dict(ws=FAKE + 8, n=1 << 20), -1), (dict(ws=FAKE, n=4), -1),
])
def test_norm_backward_rejects(kdn, kw, status):
    assert norm_back(kdn, **kw) == status


def meta(*shape, dtype=torch.float32):
    return torch.empty(shape, device="meta", dtype=dtype)


def scan(kdn, B=1, H=1, T=1, dk=16, dv=16, **kw):
    return kdn.delta_scan_fwd(meta(B, H, T, dk), meta(B, H, T, dk), meta(B, H, T, dv), meta(B, H, T), meta(B, H, T), meta(H),
                              **kw)


@pytest.mark.parametrize("call", [
    lambda k: scan(k, B=BIG), lambda k: scan(k, H=BIG), lambda k: scan(k, T=BIG), lambda k: scan(k, dk=BIG),
    lambda k: scan(k, offsets=meta(BIG + 1, dtype=torch.int32)),
    lambda k: k.delta_scan_bwd(meta(1, BIG, 1, 16), meta(1, BIG, 1, 16), meta(1, BIG, 1, 16), meta(1, BIG, 1), meta(1, BIG, 1),
                               meta(BIG), meta(1, BIG, 1, 16)),
    lambda k: k.delta_step(meta(BIG, 1, 16), meta(BIG, 1, 16), meta(BIG, 1, 16), meta(BIG, 1), meta(BIG, 1), meta(1),
                           meta(BIG, 1, 16, 16)),
    lambda k: k.delta_scan_fwd_workspace(1, 1, BIG, 16, 16), lambda k: k.delta_scan_bwd_workspace(1, 1, 1, 16, 16, nseq=BIG),
    lambda k: k.add_rms_norm_fwd(meta(1, BIG)), lambda k: k.add_rms_norm_bwd_workspace(1, BIG),
])
def test_sizes_that_32_bits_do_not_hold_are_refused(kdn, call):
    with pytest.raises(ValueError, match=r"below 2\*\*31"):
        call(kdn)


def cpu(B=2, H=3, T=5, dk=16, dv=32, dt=torch.float32):
    z = lambda *s: torch.zeros(s, dtype=dt)  # noqa: E731
    return dict(q=z(B, H, T, dk), k=z(B, H, T, dk), v=z(B, H, T, dv), beta=z(B, H, T), d=z(B, H, T), A=torch.zeros(H))


@pytest.mark.parametrize("name,bad,match", [
    ("k", torch.zeros(2, 3, 5, 32), "k must have shape"), ("k", torch.zeros(2, 3, 5, 16).bfloat16(), "k must be"),
    ("v", torch.zeros(2, 3, 4, 32), "v must have shape"), ("v", torch.zeros(2, 3, 5, 64)[..., ::2], "v must be contiguous"),
    ("beta", torch.zeros(2, 3, 5, 1), "beta must have shape"), ("d", torch.zeros(2, 3, 6), "d must have shape"),
    ("A", torch.zeros(2), "A must have shape"), ("A", torch.zeros(3).double(), "A must be"),
    ("q", torch.zeros(2, 3, 5, 16).half(), "must be bf16 or fp32"), ("q", torch.zeros(3, 5, 16), "q must be"),
    ("S0", torch.zeros(2, 3, 16, 32), "S0 must have shape"), ("out", torch.zeros(2, 3, 5, 16), "out must have shape"),
    ("out_dtype", torch.half, "out must be bf16 or fp32"), ("final_state", torch.zeros(2, 3, 32), "final_state must have"),
    ("offsets", torch.zeros(3, dtype=torch.int32), "B = 1"), ("offsets", torch.zeros(3), "offsets must be"),
])
def test_binding_refuses(kdn, name, bad, match):
    with pytest.raises(ValueError, match=match):
        kdn.delta_scan_fwd(**dict(cpu(), **{name: bad}))


def test_host_tensors_are_refused(kdn):
    x = cpu()
    with pytest.raises(ValueError, match="CUDA tensor"):
        kdn.delta_scan_fwd(**x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        kdn.delta_scan_bwd(**x, grad_out=x["v"])
    one = {k: t if k == "A" else t[:, :, 0].contiguous() for k, t in x.items()}
    with pytest.raises(ValueError, match="CUDA tensor"):
        kdn.delta_step(**one, state=torch.zeros(2, 3, 32, 16))
    with pytest.raises(ValueError, match="state must have shape"):
        kdn.delta_step(**one, state=torch.zeros(2, 3, 16, 32))
    with pytest.raises(ValueError, match="CUDA tensor"):
        kdn.add_rms_norm_fwd(torch.zeros(2, 8))
    with pytest.raises(ValueError, match="CUDA tensor"):
        kdn.add_rms_norm_bwd(torch.zeros(2, 8), torch.zeros(2, 8))
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(1 << 24), torch.zeros(1 << 24, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace must be contiguous"):
            kdn.delta_scan_bwd(**x, grad_out=x["v"], workspace=ws)
        with pytest.raises(ValueError, match="workspace must be contiguous"):
            kdn.add_rms_norm_bwd(torch.zeros(2, 8), torch.zeros(2, 8), grad_weight=True, workspace=ws)
    with pytest.raises(ValueError, match="workspace must hold"):
        kdn.delta_scan_bwd(**x, grad_out=x["v"], workspace=torch.zeros(8, dtype=torch.uint8))


@pytest.mark.parametrize("kw,match", [
    (dict(residual=torch.zeros(2, 9)), "residual must have shape"), (dict(residual=torch.zeros(2, 8).half()), "bf16 or fp32"),
    (dict(weight=torch.zeros(9)), "weight must have shape"), (dict(weight=torch.zeros(8).bfloat16()), "weight must be"),
    (dict(sum_out=torch.zeros(2, 8)), "needs a residual"), (dict(out_dtype=torch.half), "float8_e4m3fn"),
    (dict(scale=torch.zeros(2, 1)), "scale needs"), (dict(out_dtype=torch.float8_e4m3fn, scale=torch.zeros(2, 2)), "scale must"),
    (dict(residual=torch.zeros(2, 8), sum_out=torch.zeros(2, 8).bfloat16()), "sum_out must be"),
    (dict(x=torch.zeros(2, 3, 16)[:, :, ::2]), "adjacent channels"), (dict(x=torch.zeros(4, 3, 8)[::2]), "evenly apart"),
    (dict(x=torch.zeros(1, 8).expand(3, 8)), "apart by at least"), (dict(x=torch.zeros(())), "x must be"),
    (dict(x=torch.zeros(3, 0)), "C > 0"),
])
def test_norm_binding_refuses(kdn, kw, match):
    with pytest.raises(ValueError, match=match):
        kdn.add_rms_norm_fwd(**dict(dict(x=torch.zeros(2, 8)), **kw))
