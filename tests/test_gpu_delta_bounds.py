"""What the delta rule and the residual's norm write lies inside what they are
given, whatever the offsets say, and calls on two streams at once keep out of
one another's way."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
MARGIN, FILL = 1 << 16, 0x5A


@pytest.fixture(scope="module")
def kdn():
    from bayesian_scan_gb300 import kdn as k
    return k


class Fences:
    """Tensors that lie 64 KB inside buffers of one value, and whether what is around them still has it."""

    def __init__(self):
        self.kept = []

    def __call__(self, *shape, dtype=F32):
        size = torch.empty(0, dtype=dtype).element_size()
        for n in shape:
            size *= n
        whole = torch.full((2 * MARGIN + size,), FILL, device="cuda", dtype=torch.uint8)
        self.kept.append((whole, size))
        return whole[MARGIN:MARGIN + size].view(dtype).view(shape)

    def hold(self):
        return all((w[:MARGIN] == FILL).all() and (w[MARGIN + n:] == FILL).all() for w, n in self.kept)


def draw(B, H, T, dk, dv, dt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    unit = lambda x: torch.nn.functional.normalize(x, dim=-1)  # noqa: E731
    x = dict(q=unit(n(B, H, T, dk)), k=unit(n(B, H, T, dk)), v=n(B, H, T, dv), beta=torch.sigmoid(n(B, H, T)),
             d=torch.nn.functional.softplus(n(B, H, T)))
    return dict({name: t.to(dt) for name, t in x.items()}, A=0.1 * torch.rand(H, device="cuda", generator=g)), n


OFFSETS = [None, [0, 5, 5, 70, 71, 140], [3, 64, 128, 130], [-9, 80, 40, 400, 20], [149, 0, 149, 0], [500, 600], [-5, -3, -1],
           [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1], [0, 150, 0, 150, 0, 150]]


@pytest.mark.parametrize("offsets", OFFSETS)
@pytest.mark.parametrize("dk,dv,dt,ot", [(64, 64, F32, F32), (16, 32, F32, BF16), (64, 64, BF16, BF16), (128, 128, BF16, BF16),
                                         (128, 32, BF16, F32)])
def test_scan(kdn, dk, dv, dt, ot, offsets):
    B, H, T, rows = (2, 2, 150, 2) if offsets is None else (1, 2, 150, len(offsets) - 1)
    x, n = draw(B, H, T, dk, dv, dt, 5)
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    S0, gf, go = n(rows, H, dv, dk), n(rows, H, dv, dk), n(B, H, T, dv).to(ot)
    new, nseq = Fences(), 0 if offsets is None else rows
    out, end = new(B, H, T, dv, dtype=ot), new(rows, H, dv, dk)
    ws = kdn.delta_scan_fwd_workspace(B, H, T, dk, dv, nseq, dt)
    kdn.delta_scan_fwd(**x, S0=S0, offsets=off, out=out, final_state=end, workspace=new(ws, dtype=torch.uint8))
    torch.cuda.synchronize()
    assert new.hold()
    grads = {"grad_" + m: new(*x[m].shape, dtype=dt) for m in ("q", "k", "v", "beta", "d")}
    ws = kdn.delta_scan_bwd_workspace(B, H, T, dk, dv, nseq, dt)
    kdn.delta_scan_bwd(**x, grad_out=go, S0=S0, offsets=off, grad_final_state=gf, grad_A=new(H), grad_S0=new(rows, H, dv, dk),
                       workspace=new(ws, dtype=torch.uint8), **grads)
    torch.cuda.synchronize()
    assert new.hold() and kdn.get_device_error() == kdn.KDN_OK


@pytest.mark.parametrize("B,H,T,dk,dv", [(1, 2, 2501, 128, 128), (1, 1, 2100, 64, 64)])
def test_parts(kdn, B, H, T, dk, dv):
    x, n = draw(B, H, T, dk, dv, BF16, 6)
    new = Fences()
    kdn.delta_scan_fwd(**x, out=new(B, H, T, dv, dtype=F32), final_state=new(B, H, dv, dk),
                       workspace=new(kdn.delta_scan_fwd_workspace(B, H, T, dk, dv), dtype=torch.uint8))
    kdn.delta_scan_bwd(**x, grad_out=n(B, H, T, dv).to(BF16), grad_A=new(H), grad_S0=new(B, H, dv, dk),
                       workspace=new(kdn.delta_scan_bwd_workspace(B, H, T, dk, dv), dtype=torch.uint8),
                       **{"grad_" + m: new(*x[m].shape, dtype=BF16) for m in ("q", "k", "v", "beta", "d")})
    torch.cuda.synchronize()
    assert new.hold()


@pytest.mark.parametrize("B,H,dk,dv", [(1, 1, 16, 16), (3, 5, 128, 64), (65, 16, 64, 128)])
@pytest.mark.parametrize("dt,ot", [(BF16, F32), (F32, BF16)])
def test_step(kdn, B, H, dk, dv, dt, ot):
    x, n = draw(B, H, 1, dk, dv, dt, 7)
    one = {m: t if m == "A" else t[:, :, 0].contiguous() for m, t in x.items()}
    new = Fences()
    kdn.delta_step(**one, state=n(B, H, dv, dk), new_state=new(B, H, dv, dk), out=new(B, H, dv, dtype=ot))
    torch.cuda.synchronize()
    assert new.hold()


@pytest.mark.parametrize("rows,C", [(1, 1), (3, 7), (5, 136), (9, 2048), (2, 20001), (1300, 512), (1501, 129)])
@pytest.mark.parametrize("dt,rt", [(BF16, BF16), (BF16, F32), (F32, F32)])
def test_norm(kdn, rows, C, dt, rt):
    g = torch.Generator(device="cuda").manual_seed(C)
    n = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    x, r, w = n(rows, C).to(dt), n(rows, C).to(rt), n(C)
    new = Fences()
    _, s, _ = kdn.add_rms_norm_fwd(x, r, weight=w, sum_out=new(rows, C, dtype=rt), out=new(rows, C, dtype=E4M3),
                                   scale=new(rows, -(-C // 128)))
    kdn.add_rms_norm_fwd(x, r, weight=w, sum_out=new(rows, C, dtype=rt), out=new(rows, C, dtype=dt))
    kdn.add_rms_norm_bwd(s, x, weight=w, grad_sum=r, grad_residual=new(rows, C, dtype=rt), grad_x=new(rows, C, dtype=dt),
                         workspace=new(kdn.add_rms_norm_bwd_workspace(rows, C), dtype=torch.uint8))
    torch.cuda.synchronize()
    assert new.hold()


@pytest.mark.parametrize("dk,dt", [(128, BF16), (64, BF16), (64, F32)])
def test_two_streams_at_once(kdn, dk, dt):
    # sizes that leave SMs free, so that the calls do run beside one another
    work = []
    for i in range(2):
        x, n = draw(2, 8, 700 + 65 * i, dk, dk, dt, 8 + i)
        go, rows = n(*x["v"].shape).to(dt), n(300, 1000).to(dt)
        work.append((x, go, rows))

    def run(x, go, rows, stream=None):
        o, end = kdn.delta_scan_fwd(**x, stream=stream)
        g = kdn.delta_scan_bwd(**x, grad_out=go, stream=stream)
        y, s, _ = kdn.add_rms_norm_fwd(rows, rows, stream=stream)
        b = kdn.add_rms_norm_bwd(s, y, grad_weight=True, stream=stream)
        return [o, end, *g.values(), y, s, b["x"], b["weight"]]

    want = [run(*w) for w in work]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in work]
    for _ in range(3):
        got = [None, None]
        for _ in range(4):
            for i, w in enumerate(work):
                got[i] = run(*w, stream=side[i])
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(s, t) for s, t in zip(a, b))
    assert kdn.get_device_error() == kdn.KDN_OK
