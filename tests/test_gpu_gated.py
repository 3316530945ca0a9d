"""The gated recurrence (kdn_gated_scan_fwd, kdn_gated_scan_bwd,
kdn_gated_step) against its 64-bit plain form: types, layouts, lengths from
none to many tiles, odd channel counts, packed sequences, and the calls around
them (streams, graphs, resume, buffers of the caller)."""
import math

import pytest
import torch

import plain64

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def draw(B, H, T, C, dtype=F32, seed=0, rows=None, A_lo=1e-3, A_hi=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, H, T, C, generator=g).to(dtype)
    d = torch.nn.functional.softplus(torch.randn(B, H, T, C, generator=g)).to(dtype)
    A = torch.exp(torch.empty(H, C).uniform_(math.log(A_lo), math.log(A_hi), generator=g))
    h0 = torch.randn(rows or B, H, C, generator=g)
    go = torch.randn(B, H, T, C, generator=g)
    gf = torch.randn(rows or B, H, C, generator=g)
    return x, d, A, h0, go, gf


def check_fwd(x, d, A, h0, leak, out_dtype, offsets=None):
    from bayesian_scan_gb300 import kdn
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32)
    out = torch.full(x.shape, 7.0, dtype=out_dtype, device="cuda")
    o, f = kdn.gated_scan_fwd(x.cuda(), d.cuda(), A.cuda(), h0=None if h0 is None else h0.cuda(), leak=leak,
                              offsets=None if off is None else off.cuda(), out=out)
    ro, rf, eo, ef = plain64.gated_fwd(x, d, A, h0, leak, off)
    plain64.assert_within(o, ro, eo, "out")
    plain64.assert_within(f, rf, ef, "final_state")
    assert (o.cpu()[ro.isnan()] == 7.0).all(), "a token in no sequence was written"
    return o, f


def check_bwd(x, d, A, h0, go, gf, leak, out_dtype, offsets=None):
    from bayesian_scan_gb300 import kdn
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32)
    out = plain64.gated_fwd(x, d, A, h0, leak, off)[0].nan_to_num(3.0).to(out_dtype)
    go = go.to(out_dtype)
    gx, gd = (torch.full(x.shape, 7.0, dtype=x.dtype, device="cuda") for _ in range(2))
    cu = lambda t: None if t is None else t.cuda()
    got = kdn.gated_scan_bwd(x.cuda(), d.cuda(), A.cuda(), out.cuda(), go.cuda(), h0=cu(h0), leak=leak,
                             offsets=cu(off), grad_final_state=cu(gf), grad_x=gx, grad_d=gd)
    val, err = plain64.gated_bwd(x, d, A, out, go, h0, leak, off, gf)
    for n in ("x", "d", "A", "h0"):
        plain64.assert_within(got[n], val[n], err[n], "grad_" + n)
    for n in ("x", "d"):
        assert (got[n].cpu()[val[n].isnan()] == 7.0).all(), "a token in no sequence was written"
    return got


TYPES = [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)]


@pytest.mark.parametrize("in_dtype,out_dtype", TYPES)
@pytest.mark.parametrize("leak", [False, True])
@pytest.mark.parametrize("B,H,T,C", [(2, 1, 77, 64), (1, 3, 130, 250), (2, 2, 33, 7)])
def test_types_and_layouts(B, H, T, C, in_dtype, out_dtype, leak):
    x, d, A, h0, go, gf = draw(B, H, T, C, in_dtype, seed=T + C)
    check_fwd(x, d, A, h0, leak, out_dtype)
    check_bwd(x, d, A, h0, go, gf, leak, out_dtype)


@pytest.mark.parametrize("T", [0, 1, 2, 15, 16, 17, 31, 64, 127, 128, 129, 255, 1023, 1024, 1025, 2049])
@pytest.mark.parametrize("C,dtype", [(64, BF16), (33, F32)])
def test_lengths(T, C, dtype):
    x, d, A, h0, go, gf = draw(1, 1, T, C, dtype, seed=T)
    check_fwd(x, d, A, h0, True, dtype)
    check_bwd(x, d, A, h0, go, gf, True, dtype)
    check_fwd(x, d, A, None, False, F32)
    check_bwd(x, d, A, None, go, None, False, F32)


@pytest.mark.parametrize("C", [1, 2, 3, 8, 31, 32, 63, 65, 96, 128, 130, 257, 1000])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_channel_counts(C, dtype):
    x, d, A, h0, go, gf = draw(2, 1, 150, C, dtype, seed=C)
    check_fwd(x, d, A, h0, False, dtype)
    check_bwd(x, d, A, h0, go, gf, False, dtype)


@pytest.mark.parametrize("C,T,H", [(16, 20000, 1), (64, 9001, 2), (5, 6000, 1), (200, 5000, 1)])
@pytest.mark.parametrize("leak", [False, True])
def test_long_sequences_of_few_channels(C, T, H, leak):
    x, d, A, h0, go, gf = draw(1, H, T, C, F32, seed=T)
    check_fwd(x, d, A, h0, leak, F32)
    check_bwd(x, d, A, h0, go, gf, leak, F32)


@pytest.mark.parametrize("A_lo,A_hi", [(0.0, 1e-30), (1e-6, 1e-5), (5.0, 50.0), (100.0, 1e4)])
@pytest.mark.parametrize("leak", [False, True])
def test_gate_extremes(A_lo, A_hi, leak):
    # alpha = 1 (a plain sum), memories longer than the sequence, and gates that forget everything
    x, d, A, h0, go, gf = draw(2, 1, 300, 40, F32, seed=3)
    A = torch.zeros_like(A) if A_lo == 0 else torch.exp(torch.empty_like(A).uniform_(
        math.log(A_lo), math.log(A_hi), generator=torch.Generator().manual_seed(1)))
    check_fwd(x, d, A, h0, leak, F32)
    check_bwd(x, d, A, h0, go, gf, leak, F32)
    d[:, :, ::3] = 0
    check_fwd(x, d, A, h0, leak, F32)
    check_bwd(x, d, A, h0, go, gf, leak, F32)


OFFSETS = [
    [0, 1, 1, 1, 40, 300],                          # one token, two empty ones, ragged
    [5, 5, 6, 134, 262, 290],                       # tokens in no sequence at both ends, a whole tile
    [0, 300],
    [300, 300, 300],                                # nothing at all
    [0] + list(range(3, 300, 7)) + [300],           # many short ones
    [0, 0],
]


@pytest.mark.parametrize("offsets", OFFSETS)
@pytest.mark.parametrize("H", [1, 2])
@pytest.mark.parametrize("leak,in_dtype,out_dtype", [(True, BF16, F32), (False, F32, F32), (False, BF16, BF16)])
def test_packed(offsets, H, leak, in_dtype, out_dtype):
    x, d, A, h0, go, gf = draw(1, H, 300, 72, in_dtype, seed=len(offsets), rows=len(offsets) - 1)
    check_fwd(x, d, A, h0, leak, out_dtype, offsets)
    check_fwd(x, d, A, None, leak, out_dtype, offsets)
    check_bwd(x, d, A, h0, go, gf, leak, out_dtype, offsets)
    check_bwd(x, d, A, None, go, None, leak, out_dtype, offsets)


def test_packed_long_and_short_together():
    offsets = [0, 3, 2900, 2900, 2950, 4096]
    x, d, A, h0, go, gf = draw(1, 1, 4100, 130, F32, seed=2, rows=5)
    check_fwd(x, d, A, h0, False, F32, offsets)
    check_bwd(x, d, A, h0, go, gf, False, F32, offsets)


@pytest.mark.parametrize("nseq,T,C", [(40, 41000, 768), (10, 20600, 1024)])
def test_packed_long_ones_that_fill_the_device(nseq, T, C):
    # clusters of two and of four over a full device: channels sampled at both ends
    from bayesian_scan_gb300 import kdn
    x, d, A, h0, go, gf = draw(1, 1, T, C, F32, seed=nseq, rows=nseq)
    g = torch.Generator().manual_seed(nseq)
    offsets = torch.tensor([5] + sorted(torch.randint(5, T - 50, (nseq - 1,), generator=g).tolist()) + [T - 50])
    off = offsets.to(torch.int32).cuda()
    dev = [t.cuda() for t in (x, d, A)]
    o, f = kdn.gated_scan_fwd(*dev, h0=h0.cuda(), offsets=off)
    got = kdn.gated_scan_bwd(*dev, o, go.cuda(), h0=h0.cuda(), offsets=off, grad_final_state=gf.cuda())
    o, f, got = o.cpu(), f.cpu(), {n: t.cpu() for n, t in got.items()}
    at = lambda t: t[..., [0, 1, 2, C - 3, C - 2, C - 1]].contiguous()
    ro, rf, eo, ef = plain64.gated_fwd(at(x), at(d), at(A), at(h0), False, offsets)
    plain64.assert_within(at(o), ro, eo, "out")
    plain64.assert_within(at(f), rf, ef, "final_state")
    val, err = plain64.gated_bwd(at(x), at(d), at(A), at(o), at(go), at(h0), False, offsets, at(gf))
    for n in ("x", "d", "A", "h0"):
        plain64.assert_within(at(got[n]), val[n], err[n], "grad_" + n)
    assert kdn.get_device_error() == kdn.KDN_OK


def test_offsets_out_of_range_are_clamped():
    from bayesian_scan_gb300 import kdn
    x, d, A, h0, go, gf = draw(1, 1, 100, 40, F32, seed=4, rows=3)
    want = plain64.gated_fwd(x, d, A, h0, False, torch.tensor([0, 60, 100, 100]))
    off = torch.tensor([-7, 60, 1 << 30, 1 << 30], dtype=torch.int32).cuda()
    o, f = kdn.gated_scan_fwd(x.cuda(), d.cuda(), A.cuda(), h0=h0.cuda(), offsets=off)
    plain64.assert_within(o, want[0], want[2])
    plain64.assert_within(f, want[1], want[3])
    # decreasing ones: which tokens are whose is unspecified, but every access stays in range
    off = torch.tensor([50, 100, 0, 30], dtype=torch.int32).cuda()
    kdn.gated_scan_fwd(x.cuda(), d.cuda(), A.cuda(), h0=h0.cuda(), offsets=off)
    kdn.gated_scan_bwd(x.cuda(), d.cuda(), A.cuda(), o, o, h0=h0.cuda(), offsets=off)
    torch.cuda.synchronize()


def test_what_is_not_finite_stays_in_its_sequence_and_channel():
    x, d, A, h0, go, gf = draw(1, 1, 400, 66, F32, seed=5, rows=3)
    offsets = [0, 150, 151, 400]
    clean = check_fwd(x, d, A, h0, False, F32, offsets)
    x[0, 0, 100, 10] = math.nan
    x[0, 0, 149, 11] = math.inf
    d[0, 0, 20, 12] = math.nan
    from bayesian_scan_gb300 import kdn
    o, f = kdn.gated_scan_fwd(x.cuda(), d.cuda(), A.cuda(), h0=h0.cuda(),
                              offsets=torch.tensor(offsets, dtype=torch.int32).cuda())
    hit = torch.zeros(x.shape, dtype=torch.bool)
    hit[0, 0, 100:150, 10] = hit[0, 0, 149:150, 11] = hit[0, 0, 20:150, 12] = True
    assert torch.equal(~o.cpu().isfinite(), hit)
    assert torch.equal(o.cpu()[~hit], clean[0].cpu()[~hit])
    assert (~f.cpu().isfinite()).nonzero().tolist() == [[0, 0, 10], [0, 0, 11], [0, 0, 12]]
    # rows behind the last sequence may hold anything
    x, d, A, h0, go, gf = draw(1, 1, 200, 66, F32, seed=6, rows=1)
    x[0, 0, 150:], d[0, 0, 150:], go[0, 0, 150:] = math.nan, math.inf, math.nan
    check_fwd(x, d, A, h0, True, F32, [0, 150])
    check_bwd(x, d, A, h0, go, gf, True, F32, [0, 150])


def test_slices_of_a_projection_and_odd_addresses():
    from bayesian_scan_gb300 import kdn
    B, T, C = 2, 90, 48
    for dtype, lead in ((BF16, 0), (BF16, 1), (F32, 3), (BF16, 8)):
        g = torch.Generator().manual_seed(lead)
        wide = torch.randn(B, T, 2 * C + lead + 5, generator=g).to(dtype)
        wide[..., lead + C:] = wide[..., lead + C:].abs()
        x, d = wide[..., lead:lead + C], wide[..., lead + C:lead + 2 * C]
        A, h0 = torch.rand(1, C, generator=g), torch.randn(B, 1, C, generator=g)
        dev = wide.cuda()
        dx, dd = dev[..., lead:lead + C], dev[..., lead + C:lead + 2 * C]
        assert not dx.is_contiguous()
        o, f = kdn.gated_scan_fwd(dx, dd, A[0].cuda(), h0=h0[:, 0].cuda(), leak=True)
        ro, rf, eo, ef = plain64.gated_fwd(x.unsqueeze(1), d.unsqueeze(1), A, h0, True)
        plain64.assert_within(o.unsqueeze(1), ro, eo)
        plain64.assert_within(f.unsqueeze(1), rf, ef)
        go = torch.randn(B, T, C, generator=g).to(dtype)
        got = kdn.gated_scan_bwd(dx, dd, A[0].cuda(), o, go.cuda(), h0=h0[:, 0].cuda(), leak=True)
        val, err = plain64.gated_bwd(x.unsqueeze(1), d.unsqueeze(1), A, o.cpu().unsqueeze(1),
                                     go.unsqueeze(1), h0, True)
        for n in ("x", "d"):
            plain64.assert_within(got[n].unsqueeze(1), val[n], err[n], n)
        plain64.assert_within(got["A"].unsqueeze(0), val["A"], err["A"], "A")
        plain64.assert_within(got["h0"].unsqueeze(1), val["h0"], err["h0"], "h0")
    # dense tensors one element into their storage
    x, d, A, h0, go, gf = draw(2, 1, 40, 64, BF16, seed=8)
    shift = lambda t: torch.cat([torch.zeros(1, dtype=t.dtype), t.flatten()]).cuda()[1:].view(t.shape)
    o, f = kdn.gated_scan_fwd(shift(x), shift(d), shift(A), h0=shift(h0), out=shift(x))
    ro, rf, eo, ef = plain64.gated_fwd(x, d, A, h0)
    plain64.assert_within(o, ro, eo)
    plain64.assert_within(f, rf, ef)


def test_gradients_against_differences():
    """The forward's own differences: L(x + eps v) - L(x - eps v) over 2 eps
    against the gradients' product with v, for each input in turn."""
    from bayesian_scan_gb300 import kdn
    x, d, A, h0, go, gf = draw(2, 1, 40, 24, F32, seed=9, A_lo=0.05)
    cu = [t.cuda() for t in (x, d, A, h0)]
    for leak in (False, True):
        def loss(x, d, A, h0):
            o, f, _, _ = plain64.gated_fwd(x, d, A, h0, leak)
            return float((o * go.double()).sum() + (f * gf.double()).sum())
        out = kdn.gated_scan_fwd(*cu[:3], h0=cu[3], leak=leak)[0]
        got = kdn.gated_scan_bwd(*cu[:3], out, go.cuda(), h0=cu[3], leak=leak, grad_final_state=gf.cuda())
        args = [t.double() for t in (x, d, A, h0)]
        for i, n in enumerate(("x", "d", "A", "h0")):
            v = torch.randn(args[i].shape, generator=torch.Generator().manual_seed(i), dtype=torch.float64)
            eps = 1e-5
            up = loss(*[a + eps * v if j == i else a for j, a in enumerate(args)])
            down = loss(*[a - eps * v if j == i else a for j, a in enumerate(args)])
            want = (up - down) / (2 * eps)
            have = float((got[n].cpu().double() * v).sum())
            # central differences are off by eps^2 L''' (1e-10 of the scale); the gradients by fp32's steps
            scale = float((got[n].cpu().double() * v).abs().sum())
            assert abs(have - want) <= 2e-6 * scale, (n, have, want)


def test_resume_and_single_tokens():
    from bayesian_scan_gb300 import kdn
    x, d, A, h0, _, _ = (t.cuda() for t in draw(3, 2, 70, 100, BF16, seed=10))
    ro, rf, eo, ef = plain64.gated_fwd(x.cpu(), d.cpu(), A.cpu(), h0.cpu(), True)
    o1, f1 = kdn.gated_scan_fwd(x[:, :, :41].contiguous(), d[:, :, :41].contiguous(), A, h0=h0, leak=True,
                                out_dtype=F32)
    state = f1.clone()
    outs = [o1]
    for t in range(41, 70):
        outs.append(kdn.gated_step(x[:, :, t].contiguous(), d[:, :, t].contiguous(), A, state, leak=True,
                                   out_dtype=F32).unsqueeze(2))
    plain64.assert_within(torch.cat(outs, 2), ro, eo)
    plain64.assert_within(state, rf, ef)


@pytest.mark.parametrize("in_dtype,out_dtype", TYPES)
@pytest.mark.parametrize("B,H,C", [(1, 1, 1), (1, 1, 2048), (5, 3, 37), (64, 1, 2048), (3, 1, 4099)])
@pytest.mark.parametrize("leak", [False, True])
def test_step(B, H, C, in_dtype, out_dtype, leak):
    from bayesian_scan_gb300 import kdn
    x, d, A, h0, _, _ = draw(B, H, 1, C, in_dtype, seed=C)
    ro, rf, eo, ef = plain64.gated_fwd(x, d, A, h0, leak)
    x, d, A, state = x[:, :, 0].contiguous().cuda(), d[:, :, 0].contiguous().cuda(), A.cuda(), h0.cuda()
    if H == 1:
        x, d, A, state = x[:, 0], d[:, 0], A[0], state[:, 0]
    kept = state.clone()
    new = torch.empty_like(state)
    o = kdn.gated_step(x, d, A, state, leak=leak, new_state=new, out_dtype=out_dtype)
    assert torch.equal(state, kept)
    o2 = kdn.gated_step(x, d, A, state, leak=leak, out_dtype=out_dtype)
    assert torch.equal(state, new) and torch.equal(o, o2)
    plain64.assert_within(o.reshape(B, H, C), ro[:, :, 0], eo[:, :, 0])
    plain64.assert_within(new.reshape(B, H, C), rf, ef)
    # addresses that no vector load takes
    shift = lambda t: torch.cat([t.flatten()[:1], t.flatten()])[1:].view(t.shape)
    o3 = kdn.gated_step(shift(x), shift(d), shift(A), shift(kept), leak=leak, new_state=shift(new),
                        out=shift(o))
    assert torch.equal(o3, o)


def test_repeats_are_equal_and_streams_and_graphs_work():
    from bayesian_scan_gb300 import kdn
    x, d, A, h0, go, gf = (t.cuda() for t in draw(2, 2, 700, 136, F32, seed=11))
    long = [t.cuda() for t in draw(1, 1, 8000, 40, F32, seed=12)]

    def both(x, d, A, h0, go, gf):
        o, f = kdn.gated_scan_fwd(x, d, A, h0=h0)
        g = kdn.gated_scan_bwd(x, d, A, o, go, h0=h0, grad_final_state=gf)
        return [o, f, *(g[n] for n in ("x", "d", "A", "h0"))]

    for args in ((x, d, A, h0, go, gf), long):
        first = both(*args)
        for a, b in zip(first, both(*args)):
            assert torch.equal(a, b)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = both(*args)
        torch.cuda.current_stream().wait_stream(side)
        for a, b in zip(first, other):
            assert torch.equal(a, b)
        # two graphs of the same calls, replayed in turn and at once, on new inputs
        graphs = []
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                held = both(*args)
            graphs.append((graph, held))
        args[0].mul_(0.5)
        again = both(*args)
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        torch.cuda.synchronize()
        for _ in range(3):
            for (graph, _), s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    graph.replay()
        torch.cuda.synchronize()
        for _, held in graphs:
            for a, b in zip(again, held):
                assert torch.equal(a, b)


def test_parts_in_captured_graphs():
    """A long sequence of few channels takes scratch of its own inside the
    call; captured, the graph holds it, and two graphs do not share it."""
    from bayesian_scan_gb300 import kdn
    x, d, A, h0, go, gf = (t.cuda() for t in draw(1, 1, 60000, 16, F32, seed=30))

    def both():
        o, f = kdn.gated_scan_fwd(x, d, A, h0=h0)
        return [o, f, *kdn.gated_scan_bwd(x, d, A, o, go, h0=h0, grad_final_state=gf).values()]

    first = both()
    ro, rf, eo, ef = plain64.gated_fwd(x[:, :, :9000].cpu(), d[:, :, :9000].cpu(), A.cpu(), h0.cpu())
    plain64.assert_within(first[0][:, :, :9000], ro, eo)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = both()
        graphs.append((graph, held))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for (graph, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for _, held in graphs:
        assert all(torch.equal(a, b) for a, b in zip(first, held))


def test_no_tokens_but_sequences():
    x, d, A, h0, go, gf = draw(1, 2, 0, 24, F32, seed=31, rows=3)
    check_fwd(x, d, A, h0, True, F32, [0, 0, 0, 0])
    check_bwd(x, d, A, h0, go, gf, True, F32, [0, 0, 0, 0])


def test_caller_workspace_and_skipped_gradients():
    from bayesian_scan_gb300 import kdn
    x, d, A, h0, go, gf = (t.cuda() for t in draw(2, 3, 500, 56, F32, seed=13))
    o, _ = kdn.gated_scan_fwd(x, d, A, h0=h0, final_state=False)
    ref = kdn.gated_scan_bwd(x, d, A, o, go, h0=h0, grad_final_state=gf)
    ws = torch.empty(kdn.gated_scan_bwd_workspace(2, 3, 500, 56) + 64, dtype=torch.uint8, device="cuda")
    ws.fill_(255)
    got = kdn.gated_scan_bwd(x, d, A, o, go, h0=h0, grad_final_state=gf, workspace=ws)
    for n in ref:
        assert torch.equal(ref[n], got[n])
    assert (ws[-64:] == 255).all()
    part = kdn.gated_scan_bwd(x, d, A, o, go, h0=h0, grad_final_state=gf, grad_A=False, grad_h0=False)
    assert part["A"] is None and part["h0"] is None
    assert torch.equal(part["x"], ref["x"]) and torch.equal(part["d"], ref["d"])
    # the library's own scratch
    import ctypes
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    gA = torch.empty_like(A)
    gx, gd = torch.empty_like(x), torch.empty_like(d)
    st = kdn.lib.kdn_gated_scan_bwd(None, 56, p(d), 56, p(A), p(h0), None, 0, 0, p(o), p(go), p(gf), p(gx),
                                    p(gd), p(gA), None, 2, 3, 500, 56, 0, 0, None, 0,
                                    ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert st == 0
    assert torch.equal(gA, ref["A"]) and torch.equal(gx, ref["x"]) and torch.equal(gd, ref["d"])


def test_many_rows():
    # more (batch, head) rows than one grid dimension counts, one token each
    from bayesian_scan_gb300 import kdn
    x, d, A, h0, go, gf = draw(70000, 1, 2, 3, F32, seed=14)
    o, f = kdn.gated_scan_fwd(x.cuda(), d.cuda(), A.cuda(), h0=h0.cuda())
    g = kdn.gated_scan_bwd(x.cuda(), d.cuda(), A.cuda(), o, go.cuda(), h0=h0.cuda())
    pick = [0, 1, 65535, 65536, 69999]
    ro, rf, eo, ef = plain64.gated_fwd(x[pick], d[pick], A, h0[pick])
    plain64.assert_within(o[pick], ro, eo)
    plain64.assert_within(f[pick], rf, ef)
    val, err = plain64.gated_bwd(x[pick], d[pick], A, o.cpu()[pick], go[pick], h0[pick])
    for n in ("x", "d", "h0"):
        plain64.assert_within(g[n][pick], val[n], err[n], n)
    # grad A is every row's: against the sum of the parts that grad d is made of (grad d = -A u (h - ..))
    want = (g["d"].double() / A.double().cuda() * d.double().cuda()).sum((0, 2)).cpu()
    assert torch.allclose(g["A"].cpu().double(), want, rtol=0, atol=float(2 ** -24 * 140000 * want.abs().max() + 1e-2))


def test_a_cluster_whose_member_sends_nothing_times_out():
    """Fault injection: one rank of every cluster keeps its maps to itself, so
    every wait of the cluster runs out, the error is reported and the next
    call is right again."""
    from bayesian_scan_gb300 import kdn
    x, d, A, h0, go, gf = draw(1, 1, 6000, 200, F32, seed=15)
    cu = [t.cuda() for t in (x, d, A, h0)]
    assert kdn.get_device_error() == kdn.KDN_OK
    kdn.set_wait_limit_ns(20_000_000)
    kdn.debug_stall_gated_rank(1)
    try:
        kdn.gated_scan_fwd(*cu[:3], h0=cu[3])
        assert kdn.get_device_error() == kdn.KDN_ERR_TIMEOUT
        kdn.gated_scan_bwd(*cu[:3], cu[0], cu[0], h0=cu[3])
        assert kdn.get_device_error() == kdn.KDN_ERR_TIMEOUT
    finally:
        kdn.debug_stall_gated_rank(-1)
        kdn.set_wait_limit_ns(0)
    assert kdn.get_device_error() == kdn.KDN_OK
    check_fwd(x, d, A, h0, False, F32)
    check_bwd(x, d, A, h0, go, gf, False, F32)
    assert kdn.get_device_error() == kdn.KDN_OK


@pytest.mark.parametrize("in_dtype,out_dtype", TYPES)
@pytest.mark.parametrize("C", [64, 66, 63])
def test_clusters_in_every_alignment(C, in_dtype, out_dtype):
    # several rounds of clusters, rows that allow copies of 16, 4 and 2 bytes, an edge in the last tile
    x, d, A, h0, go, gf = draw(3, 1, 1300, C, in_dtype, seed=C)
    for leak in (False, True):
        check_fwd(x, d, A, h0, leak, out_dtype)
        check_bwd(x, d, A, h0, go, gf, leak, out_dtype)


def test_full_device_without_clusters():
    # enough rows that the calls run without clusters (the halves below may not): sampled rows against the plain form
    from bayesian_scan_gb300 import kdn
    x, d, A, h0, go, gf = draw(20, 1, 400, 1024, BF16, seed=16)
    o, f = kdn.gated_scan_fwd(x.cuda(), d.cuda(), A.cuda(), h0=h0.cuda())
    g = kdn.gated_scan_bwd(x.cuda(), d.cuda(), A.cuda(), o, go.bfloat16().cuda(), h0=h0.cuda(), grad_final_state=gf.cuda())
    pick = [0, 7, 19]
    ro, rf, eo, ef = plain64.gated_fwd(x[pick], d[pick], A, h0[pick])
    plain64.assert_within(o[pick], ro, eo, "out")
    plain64.assert_within(f[pick], rf, ef, "final_state")
    val, err = plain64.gated_bwd(x[pick], d[pick], A, o.cpu()[pick], go[pick].bfloat16(), h0[pick], g_final=gf[pick])
    for n in ("x", "d", "h0"):
        plain64.assert_within(g[n][pick], val[n], err[n], "grad_" + n)
    # grad A is linear in the rows' gradients: those of two halves of the batch add up to it, each sum
    # within its own rounding (tokens x half a step) of the magnitudes, here under 3e-4 of the largest
    half = [kdn.gated_scan_bwd(*(t[s].contiguous().cuda() for t in (x, d)), A.cuda(), o[s].contiguous(),
                               go[s].bfloat16().cuda(), h0=h0[s].cuda(), grad_final_state=gf[s].cuda())["A"]
            for s in (slice(0, 10), slice(10, 20))]
    assert (half[0] + half[1] - g["A"]).abs().max() <= 3e-4 * g["A"].abs().max()


def test_two_streams_at_once():
    from bayesian_scan_gb300 import kdn
    sets = [[t.cuda() for t in draw(1, 2, 5000, 96, F32, seed=s)] for s in (20, 21)]
    alone = []
    for x, d, A, h0, go, gf in sets:
        o, f = kdn.gated_scan_fwd(x, d, A, h0=h0)
        alone.append([o, f, *kdn.gated_scan_bwd(x, d, A, o, go, h0=h0, grad_final_state=gf).values()])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for s, (x, d, A, h0, go, gf) in zip(streams, sets):
            with torch.cuda.stream(s):
                o, f = kdn.gated_scan_fwd(x, d, A, h0=h0)
                got.append([o, f, *kdn.gated_scan_bwd(x, d, A, o, go, h0=h0, grad_final_state=gf).values()])
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_a_stream_given_by_hand():
    from bayesian_scan_gb300 import kdn
    x, d, A, h0, go, gf = (t.cuda() for t in draw(2, 1, 90, 64, F32, seed=22))
    ref = kdn.gated_scan_fwd(x, d, A, h0=h0)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    o, f = kdn.gated_scan_fwd(x, d, A, h0=h0, stream=s)
    y = kdn.gated_step(x[:, :, 0].contiguous(), d[:, :, 0].contiguous(), A, h0.clone(), stream=s)
    go, gf = torch.ones_like(x), torch.ones_like(h0)
    want = kdn.gated_scan_bwd(x, d, A, ref[0], go, h0=h0, grad_final_state=gf)
    torch.cuda.synchronize()
    got = kdn.gated_scan_bwd(x, d, A, ref[0], go, h0=h0, grad_final_state=gf, stream=s)
    s.synchronize()
    assert all(torch.equal(want[n], got[n]) for n in want)
    assert torch.equal(o, ref[0]) and torch.equal(f, ref[1]) and y.shape == h0.shape
