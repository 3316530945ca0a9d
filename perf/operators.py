"""Cases of the gated recurrence and of the query/key preparation, with their plain forms.

Operators (``bayesian_scan_gb300.kdn``):

* ``gated_scan_fwd`` -- h_t = alpha_t h_{t-1} + w_t x_t per channel, alpha_t =
  exp(-A d_t), w_t = 1 or 1 - alpha_t (``leak``), over [B,T,C] or [B,H,T,C], or
  over packed sequences;
* ``gated_scan_bwd`` -- its gradients, from the forward's output;
* ``gated_step`` -- one token from a state kept on the device;
* ``qk_norm_rope_fwd`` -- norm of every query and key head, then the position
  rotation (one or several axes), into the scans' [B,H,T,dk] layout;
* ``qk_norm_rope_bwd`` -- its gradients.

``run`` computes either the plain form (elementary torch operations in 32
bits, angles in 64) or, with ``own`` set, makes the framework's calls.
"""
import math

import numpy as np
import torch

own = False

BF16, F32 = "bf16", "fp32"
_DT = {BF16: torch.bfloat16, F32: torch.float32}
_ES = {BF16: 2, F32: 4}


# ---------------------------------------------------------------------------
# the cases

def _scan_case(name, op, B, H, T, C, in_dtype, out_dtype, leak, state, n_seq=0):
    return dict(name=name, op=op, B=B, H=H, T=T, C=C, in_dtype=in_dtype, out_dtype=out_dtype,
                leak=leak, state=state, n_seq=n_seq)


def _qk_case(name, op, B, T, Hq, Hk, dk, in_dtype, out_dtype, norm, weight, rot, axes, interleaved):
    return dict(name=name, op=op, B=B, T=T, Hq=Hq, Hk=Hk, dk=dk, in_dtype=in_dtype,
                out_dtype=out_dtype, norm=norm, weight=weight, rot=rot, axes=axes,
                interleaved=interleaved)


def listed():
    return [
        # training forward of a 750M-shaped layer: 8 sequences of 4096 tokens, 16 x 128 channels
        _scan_case("scan_layer", "scan_fwd", 8, 1, 4096, 2048, BF16, BF16, False, False),
        # one 65536-token context at the same width, convex writes, prefilled from a state
        _scan_case("scan_longctx", "scan_fwd", 1, 1, 65536, 2048, BF16, BF16, True, True),
        # a serving prefill: ragged prompts packed behind one another, padding behind the last, an odd width
        _scan_case("scan_packed", "scan_fwd", 1, 1, 6001, 1000, BF16, F32, False, True, 23),
        # training backward of the layer
        _scan_case("scan_bwd_layer", "scan_bwd", 8, 1, 4096, 2048, BF16, BF16, False, False),
        # training backward in the scans' head layout: few channels, one long ragged sequence, fp32
        _scan_case("scan_bwd_few_heads", "scan_bwd", 1, 4, 9001, 64, F32, F32, True, True),
        # decoding a batch of 128 requests, 16 x 128 channels
        _scan_case("step_decode", "step", 128, 1, 1, 2048, BF16, BF16, False, True),
        # decoding one request: latency alone
        _scan_case("step_one", "step", 1, 1, 1, 2048, BF16, BF16, True, True),
        # queries and keys of the 750M-shaped layer
        _qk_case("qk_layer", "qk_fwd", 8, 4096, 16, 16, 128, BF16, BF16, "rms", True, 128, 1, False),
        # image and video tokens with time, height and width positions, fewer key heads, odd length
        _qk_case("qk_axes", "qk_fwd", 3, 1271, 32, 8, 64, BF16, F32, "rms", True, 64, 3, True),
        # decoding 128 requests at their own positions, keys of unit length
        _qk_case("qk_decode", "qk_fwd", 128, 1, 16, 16, 128, BF16, BF16, "l2", False, 128, 1, False),
        # training backward of the layer's queries and keys: fp32 gradients as the scan's backward gives them
        _qk_case("qk_bwd_layer", "qk_bwd", 8, 4096, 16, 16, 128, BF16, F32, "rms", True, 128, 1, False),
        # the same for a short ragged fp32 batch, half of each head rotated, three axes
        _qk_case("qk_bwd_axes", "qk_bwd", 3, 333, 8, 2, 64, F32, F32, "l2", True, 32, 3, True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["scan_fwd", "scan_fwd", "scan_bwd", "scan_bwd", "step", "qk_fwd", "qk_fwd", "qk_bwd"])
    in_dtype = rng.choice([BF16, BF16, F32])
    out_dtype = rng.choice([in_dtype, F32])
    if op == "step":
        return _scan_case("", op, _log_int(rng, 1, 256), 1, 1, _log_int(rng, 64, 4096), in_dtype,
                          out_dtype, rng.random() < 0.5, True)
    if op in ("scan_fwd", "scan_bwd"):
        most = 1 << 25                    # elements; the largest listed case has 1 << 27
        C = _log_int(rng, 48, 4096)
        if rng.random() < 0.5:
            C = (C + 7) // 8 * 8
        T = _log_int(rng, 1, min(65536, most // C))
        room = max(1, most // (C * T))
        H = rng.choice([1, 1, rng.randint(1, min(16, room))])
        B = _log_int(rng, 1, max(1, min(16, room // H)))
        n_seq = rng.randint(1, min(64, T)) if rng.random() < 0.3 else 0
        if n_seq:
            B = 1
        return _scan_case("", op, B, H, T, C, in_dtype, out_dtype, rng.random() < 0.5,
                          rng.random() < 0.5, n_seq)
    dk = rng.choice([16, 32, 64, 128])
    Hq = rng.randint(1, 32)
    Hk = rng.choice([Hq, rng.randint(1, Hq)])
    T = _log_int(rng, 1, 8192)
    B = _log_int(rng, 1, max(1, min(128, (1 << 25) // (T * (Hq + Hk) * dk))))
    rot = rng.choice([dk, dk, dk // 2])
    return _qk_case("", op, B, T, Hq, Hk, dk, in_dtype, out_dtype, rng.choice(["rms", "l2", "none"]),
                    rng.random() < 0.7, rot, rng.choice([1, 1, 2, 3]), rng.random() < 0.5)


# ---------------------------------------------------------------------------
# the inputs

def _offsets(case, seed):
    """Ragged lengths that fill the rows but for some padding behind the last."""
    r = np.random.RandomState(seed % (1 << 31))
    rows = case["T"] - min(case["T"] - 1, case["T"] // 50)
    cuts = np.sort(r.randint(0, rows + 1, case["n_seq"] - 1))
    return np.concatenate([[0], cuts, [rows]]).astype(np.int32)


def _scan_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, H, T, C = case["B"], case["H"], case["T"], case["C"]
    dt, f32 = _DT[case["in_dtype"]], dict(device="cuda", dtype=torch.float32, generator=g)
    lead = (B,) if H == 1 else (B, H)
    shape = (B, C) if case["op"] == "step" else (*lead, T, C)
    x = torch.randn(shape, **f32).to(dt)
    d = torch.nn.functional.softplus(torch.randn(shape, **f32)).to(dt)
    # memories of about one token to a thousand
    A = torch.exp(torch.empty((C,) if H == 1 else (H, C), device="cuda").uniform_(
        math.log(1e-3), 0.0, generator=g))
    s = dict(case=case, x=x, d=d, A=A, h0=None, offsets=None)
    rows = case["n_seq"] or B
    if case["state"]:
        s["h0"] = torch.randn((rows, C) if H == 1 else (rows, H, C), **f32)
    if case["n_seq"]:
        s["offsets"] = torch.from_numpy(_offsets(case, seed)).cuda()
    return s, g


def _qk_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, T, Hq, Hk, dk = (case[n] for n in ("B", "T", "Hq", "Hk", "dk"))
    dt, f32 = _DT[case["in_dtype"]], dict(device="cuda", dtype=torch.float32, generator=g)
    # queries and keys lie side by side in the rows of one fused projection, with the values behind them
    rows = torch.randn((B, T, (Hq + 2 * Hk) * dk), **f32).to(dt)
    q = rows[:, :, :Hq * dk].unflatten(2, (Hq, dk))
    k = rows[:, :, Hq * dk:(Hq + Hk) * dk].unflatten(2, (Hk, dk))
    s = dict(case=case, q=q, k=k, wq=None, wk=None)
    if case["weight"]:
        s["wq"] = 1 + 0.2 * torch.randn(dk, **f32)
        s["wk"] = 1 + 0.2 * torch.randn(dk, **f32)
    pairs = case["rot"] // 2
    s["inv_freq"] = (1e4 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).float().cuda()
    # each sequence goes on from a place of its own in a long context; the further axes walk a grid
    start = torch.randint(0, 65536, (B, 1), device="cuda", generator=g)
    t = torch.arange(T, device="cuda")
    pos = [start + t]
    if case["axes"] > 1:
        side = max(1, math.isqrt(T))
        pos = [start + t // (side * side) if case["axes"] > 2 else start + t,
               (t // side % side).expand(B, T), (t % side).expand(B, T)][:case["axes"]]
    s["pos"] = torch.stack([p.expand(B, T) for p in pos]).to(torch.int32).contiguous()
    s["axis"] = None
    if case["axes"] > 1:
        s["axis"] = (torch.arange(pairs) * case["axes"] // pairs).to(torch.int32).cuda()
    return s, g


def prepare(case, seed):
    if case["op"].startswith("qk"):
        s, g = _qk_inputs(case, seed)
        if case["op"] == "qk_bwd":
            dt = _DT[case["out_dtype"]]
            for n, H in (("gq", case["Hq"]), ("gk", case["Hk"])):
                s[n] = torch.randn((case["B"], H, case["T"], case["dk"]), device="cuda", generator=g).to(dt)
        return s
    s, g = _scan_inputs(case, seed)
    if case["op"] == "scan_bwd":
        # the forward's output, which a training program keeps, and the gradients that come in
        s["out"] = _plain_scan(s)[0].contiguous()
        s["g"] = torch.randn(s["x"].shape, device="cuda", generator=g).to(_DT[case["out_dtype"]])
        rows = case["n_seq"] or case["B"]
        s["g_final"] = None
        if case["state"]:
            H, C = case["H"], case["C"]
            s["g_final"] = torch.randn((rows, C) if H == 1 else (rows, H, C), device="cuda", generator=g)
    if case["op"] == "step":
        s["h1"] = torch.empty_like(s["h0"])
    if case["n_seq"]:
        # buffers whose rows behind the last sequence stay as they are
        n = ("g_x", "g_d") if case["op"] == "scan_bwd" else ("o",)
        t = case["in_dtype"] if case["op"] == "scan_bwd" else case["out_dtype"]
        for name in n:
            s[name] = torch.zeros(s["x"].shape, device="cuda", dtype=_DT[t])
    return s


# ---------------------------------------------------------------------------
# the plain forms

def _prefix(z, b):
    """h_t = exp(z_t) h_{t-1} + b_t along the last axis but one, from zero, by
    doubling.  The exponents of a window are summed: a product of many factors
    next to 1 would add up their roundings."""
    n = 1
    while n < z.shape[-2]:
        b = torch.cat([b[..., :n, :], torch.addcmul(b[..., n:, :], torch.exp(z[..., n:, :]), b[..., :-n, :])], -2)
        z = torch.cat([z[..., :n, :], z[..., n:, :] + z[..., :-n, :]], -2)
        n *= 2
    return b


def _decay(s):
    x, d = s["x"].float(), s["d"].float()
    A = s["A"]
    if s["case"]["op"] != "step":
        A = A.unsqueeze(-2)
    z = -(A * d)
    return x, d, A, z, -torch.expm1(z) if s["case"]["leak"] else None


def _edges(s, T):
    """First and last rows of the packed sequences, which have any, and which rows lie in one."""
    lo, hi = s["offsets"][:-1].long(), s["offsets"][1:].long()
    some = hi > lo
    row = torch.arange(T, device=lo.device)
    return lo.clamp(max=T - 1), (hi - 1).clamp(min=0), some, ((row >= lo[0]) & (row < hi[-1])).unsqueeze(-1)


def _at(rows, some, T):
    """[T,1]: whether a row is one of these (of those that count)."""
    return (torch.zeros(T, device=rows.device).index_add_(0, rows, some.float()) > 0).unsqueeze(-1)


def _heads_first(h):
    """State rows [n,H,C] in the order of a [1,H,T,C] tensor's rows: [1,H,n,C]."""
    return h.transpose(0, 1).unsqueeze(0) if h.dim() == 3 else h.unsqueeze(0)


def _states_first(h):
    return h.squeeze(0).transpose(0, 1) if h.dim() == 4 else h.squeeze(0)


def _plain_scan(s):
    c = s["case"]
    x, d, A, z, w = _decay(s)
    b = x if w is None else w * x
    dt = _DT[c["out_dtype"]]
    h0 = s["h0"]
    if s["offsets"] is None:
        if h0 is not None:
            b = torch.cat([b[..., :1, :] + torch.exp(z[..., :1, :]) * h0.unsqueeze(-2), b[..., 1:, :]], -2)
        h = _prefix(z, b)
        return h.to(dt), h[..., -1, :].contiguous()
    first, last, some, inside = _edges(s, x.shape[-2])
    if h0 is not None:
        b = b.index_add(-2, first, torch.exp(z[..., first, :]) * _heads_first(h0) * some.float().unsqueeze(-1))
    h = _prefix(z.masked_fill(_at(first, some, x.shape[-2]), -torch.inf), b) * inside
    end = _states_first(h[..., last, :])
    some = some.view(-1, *[1] * (end.dim() - 1))
    final = torch.where(some, end, torch.zeros_like(end) if h0 is None else h0)
    return h.to(dt), final


def _plain_scan_bwd(s):
    c = s["case"]
    x, d, A, z, w = _decay(s)
    g, h, h0 = s["g"].float(), s["out"].float(), s["h0"]
    before = torch.cat([torch.zeros_like(h[..., :1, :]) if h0 is None or s["offsets"] is not None
                        else h0.unsqueeze(-2), h[..., :-1, :]], -2)
    after = torch.cat([z[..., 1:, :], torch.zeros_like(z[..., :1, :])], -2)
    if s["offsets"] is not None:
        first, last, some, inside = _edges(s, x.shape[-2])
        f = some.float().unsqueeze(-1)
        before = before.masked_fill(_at(first, some, x.shape[-2]), 0)
        if h0 is not None:
            before = before.index_add(-2, first, _heads_first(h0) * f)
        after = after.masked_fill(_at(last, some, x.shape[-2]), -torch.inf)
        g = g * inside
        if s["g_final"] is not None:
            g = g.index_add(-2, last, _heads_first(s["g_final"]) * f)
    elif s["g_final"] is not None:
        g = torch.cat([g[..., :-1, :], g[..., -1:, :] + s["g_final"].unsqueeze(-2)], -2)
    dh = _prefix(after.flip(-2), g.flip(-2)).flip(-2)
    u = torch.exp(z) * dh
    m = before if w is None else before - x
    gx = dh if w is None else w * dh
    gd = -A * u * m
    gA = -(d * u * m).sum(-2).sum(0)
    if s["offsets"] is None:
        gh0 = u[..., 0, :]
    else:
        gd = gd * inside
        gx = gx * inside
        start = _states_first(u[..., first, :])
        some = some.view(-1, *[1] * (start.dim() - 1))
        zero = torch.zeros_like(start)
        gh0 = torch.where(some, start, zero if s["g_final"] is None else s["g_final"])
    dt = _DT[c["in_dtype"]]
    return dict(x=gx.to(dt), d=gd.to(dt), A=gA, h0=gh0.contiguous())


def _plain_step(s):
    x, d, A, z, w = _decay(s)
    h = torch.exp(z) * s["h0"] + (x if w is None else w * x)
    return h.to(_DT[s["case"]["out_dtype"]]), h


def _angles(s):
    pos, axis = s["pos"].double(), s["axis"]
    p = pos[0].unsqueeze(-1) if axis is None else pos[axis.long()].permute(1, 2, 0)
    theta = p * s["inv_freq"].double()
    return torch.cos(theta).float().unsqueeze(2), torch.sin(theta).float().unsqueeze(2)


def _halves(y, case):
    n = case["rot"] // 2
    if case["interleaved"]:
        r = y[..., :2 * n].unflatten(-1, (n, 2))
        return r[..., 0], r[..., 1]
    return y[..., :n], y[..., n:2 * n]


def _joined(y1, y2, rest, case):
    r = torch.stack([y1, y2], -1).flatten(-2) if case["interleaved"] else torch.cat([y1, y2], -1)
    return torch.cat([r, rest], -1)


EPS = 1e-6


def _inverse_norm(x, case):
    if case["norm"] == "none":
        return torch.ones_like(x[..., :1])
    s = (x * x).sum(-1, keepdim=True)
    return torch.rsqrt((s / case["dk"] if case["norm"] == "rms" else s) + EPS)


def _plain_qk(s):
    c = s["case"]
    cos, sin = _angles(s)
    both = []
    for x, w in ((s["q"].float(), s["wq"]), (s["k"].float(), s["wk"])):
        y = x * _inverse_norm(x, c)
        if w is not None:
            y = y * w
        y1, y2 = _halves(y, c)
        y = _joined(y1 * cos - y2 * sin, y1 * sin + y2 * cos, y[..., c["rot"]:], c)
        both.append(y.to(_DT[c["out_dtype"]]).transpose(1, 2).contiguous())
    return tuple(both)


def _plain_qk_bwd(s):
    c = s["case"]
    cos, sin = _angles(s)
    n = c["dk"] if c["norm"] == "rms" else 1
    got = {}
    for name, x, w, g in (("q", s["q"].float(), s["wq"], s["gq"]), ("k", s["k"].float(), s["wk"], s["gk"])):
        g = g.float().transpose(1, 2)
        g1, g2 = _halves(g, c)
        g = _joined(g1 * cos + g2 * sin, g2 * cos - g1 * sin, g[..., c["rot"]:], c)
        r = _inverse_norm(x, c)
        t = g if w is None else g * w
        gx = t if c["norm"] == "none" else r * t - x * (r * r * r) * ((t * x).sum(-1, keepdim=True) / n)
        got[name] = gx.to(_DT[c["in_dtype"]]).contiguous()
        if w is not None:
            got["w" + name] = (x * r * g).sum((0, 1, 2))
    return got


# ---------------------------------------------------------------------------
# one pass

def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        from bayesian_scan_gb300 import kdn
        s = state
        if op == "scan_fwd":
            return kdn.gated_scan_fwd(s["x"], s["d"], s["A"], h0=s["h0"], leak=c["leak"], offsets=s["offsets"],
                                      out=s.get("o"), out_dtype=_DT[c["out_dtype"]])
        if op == "scan_bwd":
            return kdn.gated_scan_bwd(s["x"], s["d"], s["A"], s["out"], s["g"], h0=s["h0"], leak=c["leak"],
                                      offsets=s["offsets"], grad_final_state=s["g_final"],
                                      grad_x=s.get("g_x"), grad_d=s.get("g_d"))
        if op == "step":
            # the old state is kept, as a program that may take a token back does
            return kdn.gated_step(s["x"], s["d"], s["A"], s["h0"], leak=c["leak"], new_state=s["h1"],
                                  out_dtype=_DT[c["out_dtype"]]), s["h1"]
        more = dict(wq=s["wq"], wk=s["wk"], norm=c["norm"], eps=EPS, axis=s["axis"], interleaved=c["interleaved"])
        if op == "qk_fwd":
            return kdn.qk_norm_rope_fwd(s["q"], s["k"], s["pos"], s["inv_freq"],
                                        out_dtype=_DT[c["out_dtype"]], **more)
        got = kdn.qk_norm_rope_bwd(s["q"], s["k"], s["gq"], s["gk"], s["pos"], s["inv_freq"], **more)
        return {n: t for n, t in got.items() if t is not None}
    return {"scan_fwd": _plain_scan, "scan_bwd": _plain_scan_bwd, "step": _plain_step,
            "qk_fwd": _plain_qk, "qk_bwd": _plain_qk_bwd}[op](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    i, o = _ES[case["in_dtype"]], _ES[case["out_dtype"]]
    if case["op"].startswith("qk"):
        rows = case["B"] * case["T"]
        n = rows * (case["Hq"] + case["Hk"]) * case["dk"]
        pos = rows * case["axes"] * 4
        if case["op"] == "qk_fwd":
            return {"bytes": n * (i + o) + pos, "flops": 8.0 * n}
        return {"bytes": n * (2 * i + o) + pos, "flops": 16.0 * n}
    n = case["B"] * case["H"] * case["T"] * case["C"]
    states = (case["n_seq"] or case["B"]) * case["H"] * case["C"] * 4
    few = case["H"] * case["C"] * 4
    if case["op"] == "scan_bwd":
        return {"bytes": n * ((3 + case["leak"]) * i + 2 * o) + few * 2 + states * (3 if case["state"] else 1),
                "flops": 10.0 * n}
    return {"bytes": n * (2 * i + o) + few + states * (2 if case["state"] else 1), "flops": 5.0 * n}


# ---------------------------------------------------------------------------
# the definitions, in 64 bits, token by token

def _sequences(s):
    """(state row, batch row, first token, end) of every sequence."""
    if s["offsets"] is None:
        return [(b, b, 0, s["x"].shape[-2]) for b in range(s["x"].shape[0])]
    o = s["offsets"].tolist()
    return [(n, 0, o[n], o[n + 1]) for n in range(len(o) - 1)]


def _exact_scan(s):
    c = s["case"]
    x, d = s["x"].double(), s["d"].double()
    out = torch.zeros(x.shape, device="cuda", dtype=torch.float64)
    if s["offsets"] is None:          # all batches at once
        h = s["h0"].double() if s["h0"] is not None else torch.zeros(x[..., 0, :].shape, device="cuda", dtype=torch.float64)
        gate = torch.exp(-s["A"].double().unsqueeze(-2) * d)
        if c["leak"]:
            x = x * -torch.expm1(-s["A"].double().unsqueeze(-2) * d)
        for t in range(x.shape[-2]):
            h = torch.addcmul(x[..., t, :], gate[..., t, :], h)
            out[..., t, :] = h
        return out, h
    rows = []
    A = s["A"].double()
    for n, b, lo, hi in _sequences(s):
        h = s["h0"][n].double() if s["h0"] is not None else torch.zeros(A.shape, device="cuda", dtype=torch.float64)
        for t in range(lo, hi):
            z = -A * d[b, ..., t, :]
            h = torch.exp(z) * h + (-torch.expm1(z) if c["leak"] else 1.0) * x[b, ..., t, :]
            out[b, ..., t, :] = h
        rows.append(h)
    return out, torch.stack(rows)


def _exact_scan_bwd(s):
    c = s["case"]
    A = s["A"].double()
    x, d, g, out = (s[n].double() for n in ("x", "d", "g", "out"))
    gx, gd = torch.zeros_like(x), torch.zeros_like(x)
    gA, starts = torch.zeros_like(A), []
    seqs = _sequences(s)
    if s["offsets"] is None:
        seqs = [(slice(None), slice(None), 0, x.shape[-2])]
    for n, b, lo, hi in seqs:
        like = s["x"][b][..., 0, :]
        zero = torch.zeros(like.shape, device="cuda", dtype=torch.float64)
        into = s["g_final"][n].double() if s["g_final"] is not None else zero
        h0 = s["h0"][n].double() if s["h0"] is not None else zero
        for t in range(hi - 1, lo - 1, -1):
            dt = d[b][..., t, :]
            dh = g[b][..., t, :] + into
            z = -A * dt
            alpha = torch.exp(z)
            prev = out[b][..., t - 1, :] if t > lo else h0
            dalpha = dh * (prev - x[b][..., t, :]) if c["leak"] else dh * prev
            gx[b, ..., t, :] = dh * -torch.expm1(z) if c["leak"] else dh
            gd[b, ..., t, :] = -A * alpha * dalpha
            part = -dt * alpha * dalpha
            gA += part.sum(0) if part.dim() > gA.dim() else part
            into = alpha * dh
        starts.append(into)
    return dict(x=gx, d=gd, A=gA, h0=starts[0] if s["offsets"] is None else torch.stack(starts))


def _exact_qk(x, w, s):
    """The prepared rows of one projection by rotating complex numbers."""
    c = s["case"]
    if c["norm"] == "rms":
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
    elif c["norm"] == "l2":
        x = x / torch.sqrt(x.square().sum(-1, keepdim=True) + EPS)
    if w is not None:
        x = w * x
    n = c["rot"] // 2
    lanes = torch.arange(2 * n, device="cuda")
    one, two = (lanes[::2], lanes[1::2]) if c["interleaved"] else (lanes[:n], lanes[n:])
    axis = torch.zeros(n, dtype=torch.long, device="cuda") if s["axis"] is None else s["axis"].long()
    turn = torch.stack([s["pos"][a].double() * f for a, f in zip(axis.tolist(), s["inv_freq"].double())], -1)
    z = torch.complex(x[..., one], x[..., two]) * torch.polar(torch.ones_like(turn), turn).unsqueeze(2)
    y = x.clone()
    y[..., one] = z.real
    y[..., two] = z.imag
    return y.transpose(1, 2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("scan_fwd", "scan_bwd") and case["T"] > 20000 and case["n_seq"]:
        return None                   # tens of seconds of single tokens
    if case["op"] == "scan_fwd":
        return _exact_scan(s)
    if case["op"] == "scan_bwd":
        return _exact_scan_bwd(s)
    if case["op"] == "step":
        z = -s["A"].double() * s["d"].double()
        h = torch.exp(z) * s["h0"].double() + s["x"].double() * (-torch.expm1(z) if case["leak"] else 1.0)
        return h, h
    if case["op"] == "qk_fwd":
        return tuple(_exact_qk(s[n].double(), None if s["w" + n] is None else s["w" + n].double(), s) for n in "qk")
    got = {}
    for n in "qk":                    # by differentiating the definition
        x = s[n].double().detach().requires_grad_()
        w = None if s["w" + n] is None else s["w" + n].double().requires_grad_()
        _exact_qk(x, w, s).backward(s["g" + n].double())
        got[n] = x.grad
        if w is not None:
            got["w" + n] = w.grad
    return got
