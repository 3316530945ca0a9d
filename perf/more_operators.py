"""Cases of the gated delta rule and of the residual's addition with its norm, with their plain forms.

Operators (``bayesian_scan_gb300.kdn``):

* ``delta_scan_fwd`` -- S_t = alpha_t S_{t-1} + beta_t (v_t - alpha_t S_{t-1} k_t) k_t^T,
  o_t = S_t q_t, alpha_t = exp(-A d_t), per head a d_v x d_k state, over
  [B,H,T,.] or over packed sequences;
* ``delta_scan_bwd`` -- its gradients;
* ``delta_step`` -- one token from a state kept on the device;
* ``add_rms_norm_fwd`` -- s = x + residual, y = s / rms(s) * weight, y in bf16,
  fp32 or in 8 bits with a scale for each 128 elements;
* ``add_rms_norm_bwd`` -- its gradients.

``run`` computes either the plain form (elementary torch operations in 32
bits, exponents and long sums in 64) or, with ``own`` set, makes the
framework's calls.
"""
import math

import numpy as np
import torch

own = False

BF16, F32, E4M3 = "bf16", "fp32", "e4m3"
_DT = {BF16: torch.bfloat16, F32: torch.float32, E4M3: torch.float8_e4m3fn}
_ES = {BF16: 2, F32: 4, E4M3: 1}


# ---------------------------------------------------------------------------
# the cases

def _delta_case(name, op, B, H, T, dk, dv, in_dtype, out_dtype, state, n_seq=0):
    return dict(name=name, op=op, B=B, H=H, T=T, dk=dk, dv=dv, in_dtype=in_dtype, out_dtype=out_dtype,
                state=state, n_seq=n_seq)


def _norm_case(name, op, rows, C, in_dtype, res_dtype, out_dtype, weight):
    return dict(name=name, op=op, rows=rows, C=C, in_dtype=in_dtype, res_dtype=res_dtype,
                out_dtype=out_dtype, weight=weight)


def listed():
    return [
        # training forward of a 750M-shaped layer: 8 sequences of 4096 tokens, 16 heads of 128
        _delta_case("delta_layer", "delta_fwd", 8, 16, 4096, 128, 128, BF16, BF16, False),
        # one 65536-token context at the same width, prefilled from a state and handed on
        _delta_case("delta_longctx", "delta_fwd", 1, 16, 65536, 128, 128, BF16, BF16, True),
        # a serving prefill: ragged prompts packed behind one another, padding behind the last, 32 heads of 64
        _delta_case("delta_packed", "delta_fwd", 1, 32, 6001, 64, 64, BF16, F32, True, 23),
        # a short odd batch in fp32, values narrower than keys
        _delta_case("delta_odd", "delta_fwd", 3, 5, 333, 64, 32, F32, F32, True),
        # training backward of the layer
        _delta_case("delta_bwd_layer", "delta_bwd", 8, 16, 4096, 128, 128, BF16, BF16, False),
        # training backward of a long ragged fp32 sequence with few heads, states' gradients both ways
        _delta_case("delta_bwd_few", "delta_bwd", 1, 4, 2501, 64, 64, F32, F32, True),
        # decoding a batch of 128 requests
        _delta_case("delta_decode", "delta_step", 128, 16, 1, 128, 128, BF16, BF16, True),
        # decoding one request: latency alone
        _delta_case("delta_one", "delta_step", 1, 16, 1, 128, 128, BF16, BF16, True),
        # before the projection of the layer: 32768 tokens of 2048 channels
        _norm_case("norm_layer", "norm_fwd", 32768, 2048, BF16, BF16, BF16, True),
        # the same for a projection in 8 bits, decoding 128 requests, fp32 residual
        _norm_case("norm_decode8", "norm_fwd", 128, 2048, BF16, F32, E4M3, True),
        # training backward before the layer's projection
        _norm_case("norm_bwd_layer", "norm_bwd", 32768, 2048, BF16, BF16, BF16, True),
        # the same for an odd batch of an odd width in fp32
        _norm_case("norm_bwd_odd", "norm_bwd", 1271, 1000, F32, F32, F32, True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["delta_fwd", "delta_fwd", "delta_fwd", "delta_bwd", "delta_bwd", "delta_step",
                     "norm_fwd", "norm_fwd", "norm_bwd"])
    in_dtype = rng.choice([BF16, BF16, F32])
    out_dtype = rng.choice([in_dtype, F32])
    if op.startswith("norm"):
        res = rng.choice([in_dtype, F32])
        C = _log_int(rng, 64, 8192)
        if rng.random() < 0.7:
            C = (C + 7) // 8 * 8
        rows = _log_int(rng, 1, min(65536, (1 << 25) // C))
        if op == "norm_fwd" and rng.random() < 0.4:
            out_dtype = E4M3
        return _norm_case("", op, rows, C, in_dtype, res, out_dtype, rng.random() < 0.8)
    dk = rng.choice([16, 32, 64, 64, 128, 128, 128])
    dv = dk if rng.random() < 0.75 else rng.choice([16, 32, 64, 128])
    if op == "delta_step":
        return _delta_case("", op, _log_int(rng, 1, 128), _log_int(rng, 1, 32), 1, dk, dv, in_dtype, out_dtype, True)
    T = _log_int(rng, 1, 32768) if op == "delta_fwd" else _log_int(rng, 2, 8192)
    room = max(1, ((1 << 19) if op == "delta_fwd" else (1 << 17)) // T)        # token-heads; the longest case has 1 << 20
    H = _log_int(rng, 1, min(32, room))
    B = _log_int(rng, 1, max(1, min(16, room // H)))
    n_seq = rng.randint(1, min(32, T)) if rng.random() < 0.3 and T <= 8192 else 0
    if n_seq:
        B = 1
    return _delta_case("", op, B, H, T, dk, dv, in_dtype, out_dtype, rng.random() < 0.5, n_seq)


# ---------------------------------------------------------------------------
# the inputs

def _lengths(case, seed):
    """Ragged lengths that fill the tokens but for some padding behind the last."""
    r = np.random.RandomState(seed % (1 << 31))
    rows = case["T"] - min(case["T"] - 1, case["T"] // 50)
    cuts = np.sort(r.randint(0, rows + 1, case["n_seq"] - 1))
    return np.diff(np.concatenate([[0], cuts, [rows]])).astype(int).tolist()


def _delta_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, H, T, dk, dv = (case[n] for n in ("B", "H", "T", "dk", "dv"))
    dt, f32 = _DT[case["in_dtype"]], dict(device="cuda", dtype=torch.float32, generator=g)
    lead = (B, H) if case["op"] == "delta_step" else (B, H, T)
    # queries and keys of unit length, as the mixer's preparation leaves them
    unit = lambda n: torch.nn.functional.normalize(torch.randn((*lead, n), **f32), dim=-1).to(dt)  # noqa: E731
    s = dict(case=case, q=unit(dk), k=unit(dk), v=torch.randn((*lead, dv), **f32).to(dt))
    s["beta"] = torch.sigmoid(torch.randn(lead, **f32)).to(dt)
    s["d"] = torch.nn.functional.softplus(torch.randn(lead, **f32)).to(dt)
    # memories of about one token to a thousand
    s["A"] = torch.exp(torch.empty(H, device="cuda").uniform_(math.log(1e-3), 0.0, generator=g))
    s["lens"] = _lengths(case, seed) if case["n_seq"] else None
    s["offsets"] = s["S0"] = None
    rows = case["n_seq"] or B
    if case["n_seq"]:
        s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(s["lens"])]).astype(np.int32)).cuda()
    if case["state"]:
        s["S0"] = torch.randn((rows, H, dv, dk), **f32) * 0.3
    return s, g


def prepare(case, seed):
    if case["op"].startswith("norm"):
        g = torch.Generator(device="cuda").manual_seed(seed)
        shape, f32 = (case["rows"], case["C"]), dict(device="cuda", dtype=torch.float32, generator=g)
        s = dict(case=case, weight=None)
        if case["weight"]:
            s["weight"] = 1 + 0.2 * torch.randn(case["C"], **f32)
        # the residual's rows have sizes of their own, as they grow through a model's layers
        size = torch.exp(torch.randn(case["rows"], 1, **f32))
        s["residual"] = (size * torch.randn(shape, **f32)).to(_DT[case["res_dtype"]])
        if case["op"] == "norm_fwd":
            s["x"] = torch.randn(shape, **f32).to(_DT[case["in_dtype"]])
        else:
            # the sum that the forward left, and the gradients that come in
            s["grad_y"] = torch.randn(shape, **f32).to(_DT[case["out_dtype"]])
            s["grad_sum"] = torch.randn(shape, **f32).to(_DT[case["res_dtype"]])
        return s
    s, g = _delta_inputs(case, seed)
    f32 = dict(device="cuda", dtype=torch.float32, generator=g)
    if case["op"] == "delta_bwd":
        s["g"] = torch.randn(s["v"].shape, **f32).to(_DT[case["out_dtype"]])
        s["g_final"] = torch.randn(s["S0"].shape, **f32) if case["state"] else None
    if case["op"] == "delta_step":
        s["S1"] = torch.empty_like(s["S0"])
    if case["n_seq"]:
        # buffers whose tokens behind the last sequence stay as they are
        if case["op"] == "delta_bwd":
            s["bufs"] = {"grad_" + n: torch.zeros_like(s[n]) for n in ("q", "k", "v", "beta", "d")}
        else:
            s["bufs"] = dict(out=torch.zeros(s["v"].shape, device="cuda", dtype=_DT[case["out_dtype"]]))
    return s


# ---------------------------------------------------------------------------
# the plain forms

CHUNK = 64


def _padded(s):
    """Where the tokens of [N,H,L] sequences, L whole chunks, lie in the rows
    of [B,H,T], and which of them there are: (batch [N,1], token [N,L], there
    [N,L])."""
    B, T = s["case"]["B"], s["case"]["T"]
    lens = s["lens"] or [T] * B
    L = max(CHUNK, -(-max(lens) // CHUNK) * CHUNK)
    n = torch.tensor(lens, device="cuda").unsqueeze(1)
    first = torch.zeros_like(n) if s["lens"] is None else torch.cumsum(n, 0) - n
    t = torch.arange(L, device="cuda")
    there = t < n
    batch = torch.arange(B, device="cuda").unsqueeze(1) if s["lens"] is None else torch.zeros_like(n)
    return batch, torch.where(there, first + t, 0), there


def _chunks(x, at):
    """[B,H,T,...] -> fp32 [N,H,chunks,CHUNK,...] with zeros where no token is."""
    batch, token, there = at
    x = x[batch, :, token].float()                           # [N,L,H,...]
    x = x * there.view(*there.shape, *[1] * (x.dim() - 2))
    return x.transpose(1, 2).unflatten(2, (-1, CHUNK))


def _tokens(x, at, into):
    """[N,H,chunks,CHUNK,...] into the rows [B,H,T,...] that it came from."""
    batch, token, there = at
    x = x.flatten(2, 3).transpose(1, 2)
    n = there.nonzero(as_tuple=True)
    into.transpose(1, 2)[batch.expand_as(token)[n], token[n]] = x[n].to(into.dtype)
    return into


def _mm(a, b):
    return torch.matmul(a, b)


def _parts(s, at):
    """What a chunk's tokens say of one another."""
    p = {n: _chunks(s[n], at) for n in ("q", "k", "v", "beta", "d")}
    z = (-s["A"].double().view(-1, 1, 1) * p["d"].double()).cumsum(-1)       # log decay since the chunk began
    ratio = (z.unsqueeze(-1) - z.unsqueeze(-2)).tril()
    low = torch.ones(CHUNK, CHUNK, device="cuda").tril()
    E = torch.exp(ratio).float() * low
    strict = E.tril(-1)
    kt = p["k"].transpose(-1, -2)
    G = _mm(p["k"], kt) * strict
    p.update(E=E, strict=strict, P=_mm(p["q"], kt) * E, eg=torch.exp(z).float().unsqueeze(-1),
             w=torch.exp(z[..., -1:] - z).float().unsqueeze(-1), end=torch.exp(z[..., -1]).float())
    # X = -G (1 + beta G)^-1 by blocks of 1, 2, 4, ...: X21 = -(1 + X22 beta) G21 (1 + beta X11)
    b = p["beta"].unsqueeze(-1)
    eye = torch.eye(CHUNK, device="cuda")
    X, i, size = torch.zeros_like(G), torch.arange(CHUNK, device="cuda"), 1
    while size < CHUNK:
        block = i // size
        pair = (block.unsqueeze(1) == block + 1) & (block % 2 == 0)          # row's block follows an even column's
        X = X - _mm(eye + X * b.transpose(-1, -2), _mm(G * pair, eye + b * X)) * pair
        size *= 2
    p["X"], p["b"] = X, b
    return p


def _start(s, p):
    if s["S0"] is not None:
        return s["S0"]
    N, H, _, _, dk = p["k"].shape
    return torch.zeros((N, H, p["v"].shape[-1], dk), device="cuda")


def _walk(s, p):
    """The chunks one after another: their first states, r and the last state."""
    S, states, rs = _start(s, p), [], []
    for c in range(p["k"].shape[2]):
        states.append(S)
        z = p["v"][:, :, c] - p["eg"][:, :, c] * _mm(p["k"][:, :, c], S.transpose(-1, -2))
        r = z + _mm(p["X"][:, :, c], p["b"][:, :, c] * z)
        rs.append(r)
        u = p["b"][:, :, c] * r
        S = p["end"][:, :, c, None, None] * S + _mm(u.transpose(-1, -2), p["w"][:, :, c] * p["k"][:, :, c])
    return torch.stack(states, 2), torch.stack(rs, 2), S


def _plain_delta(s):
    at = _padded(s)
    p = _parts(s, at)
    states, r, end = _walk(s, p)
    o = p["eg"] * _mm(p["q"], states.transpose(-1, -2)) + _mm(p["P"], p["b"] * r)
    into = s["bufs"]["out"] if s["lens"] else torch.empty(s["v"].shape, device="cuda",
                                                          dtype=_DT[s["case"]["out_dtype"]])
    out = _tokens(o, at, into)
    return (out, end) if s["case"]["state"] else out


def _plain_delta_bwd(s):
    at = _padded(s)
    p = _parts(s, at)
    states, r, end = _walk(s, p)
    go = _chunks(s["g"], at)
    eg, w, b, last = p["eg"], p["w"], p["b"], p["end"][..., None, None]
    D = torch.zeros_like(end) if s["g_final"] is None else s["g_final"]
    ends, ys = [], []
    for c in reversed(range(go.shape[2])):
        ends.append(D)
        du = (_mm(p["P"][:, :, c].transpose(-1, -2), go[:, :, c])
              + _mm(w[:, :, c] * p["k"][:, :, c], D.transpose(-1, -2)))
        y = du + _mm(p["X"][:, :, c].transpose(-1, -2), b[:, :, c] * du)
        ys.append(y)
        D = (last[:, :, c] * D + _mm(go[:, :, c].transpose(-1, -2), eg[:, :, c] * p["q"][:, :, c])
             - _mm((b[:, :, c] * y).transpose(-1, -2), eg[:, :, c] * p["k"][:, :, c]))
    ends, y = torch.stack(ends[::-1], 2), torch.stack(ys[::-1], 2)
    u, lam = b * r, b * y
    dP = _mm(go, u.transpose(-1, -2)) * p["E"]
    dG = -_mm(lam, u.transpose(-1, -2)) * p["strict"]
    gq = eg * _mm(go, states) + _mm(dP, p["k"])
    read = -eg * _mm(lam, states) + _mm(dG, p["k"])
    into_end = w * _mm(u, ends)
    write = _mm(dP.transpose(-1, -2), p["q"]) + _mm(dG.transpose(-1, -2), p["k"]) + into_end
    c = ((p["q"].double() * gq).sum(-1) + (p["k"].double() * read).sum(-1) - (p["k"].double() * write).sum(-1))
    left = ((ends.double() * states).sum((-1, -2)) * p["end"] + (p["k"].double() * into_end).sum((-1, -2)))
    c = torch.cat([c[..., :-1], c[..., -1:] + left.unsqueeze(-1)], -1)
    ga = c.flip(-1).cumsum(-1).flip(-1)                      # of each token's log decay
    got = dict(q=gq, k=read + write, v=lam, beta=(r * y).sum(-1), d=(-s["A"].view(-1, 1, 1) * ga).float())
    got = {n: _tokens(x, at, s["bufs"]["grad_" + n] if s["lens"] else torch.empty_like(s[n]))
           for n, x in got.items()}
    got["A"] = -(p["d"].double() * ga).sum((-1, -2)).sum(0).float()
    if s["case"]["state"]:
        got["S0"] = D
    return got


def _plain_step(s):
    a = torch.exp(-s["A"] * s["d"].float())[..., None, None]
    k, q = s["k"].float().unsqueeze(-1), s["q"].float().unsqueeze(-1)
    S = a * s["S0"]
    u = s["beta"].float()[..., None, None] * (s["v"].float().unsqueeze(-1) - (S * k.transpose(-1, -2)).sum(-1, keepdim=True))
    S = S + u * k.transpose(-1, -2)
    return (S * q.transpose(-1, -2)).sum(-1).to(_DT[s["case"]["out_dtype"]]), S


EPS, GROUP, TOP = 1e-6, 128, 448.0


def _rstd(t):
    return torch.rsqrt(t.square().mean(-1, keepdim=True) + EPS)


def _groups(y):
    """[rows, C] in groups of 128 channels, the last filled up with zeros."""
    return torch.nn.functional.pad(y, (0, -y.shape[-1] % GROUP)).unflatten(-1, (-1, GROUP))


def _plain_norm(s):
    total = (s["x"].float() + s["residual"].float()).to(s["residual"].dtype)
    t = total.float()
    y = t * _rstd(t)
    if s["weight"] is not None:
        y = y * s["weight"]
    if s["case"]["out_dtype"] != E4M3:
        return y.to(_DT[s["case"]["out_dtype"]]), total
    groups = _groups(y)
    scale = groups.abs().amax(-1) / TOP
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    y8 = (groups / scale.unsqueeze(-1)).flatten(-2)[..., :y.shape[-1]].to(torch.float8_e4m3fn)
    return y8, total, scale


def _plain_norm_bwd(s):
    t, gy = s["residual"].float(), s["grad_y"].float()
    r = _rstd(t)
    n = t * r
    gw = (gy * n).double().sum(0).float()
    g = gy if s["weight"] is None else gy * s["weight"]
    g = r * (g - n * (g * n).mean(-1, keepdim=True)) + s["grad_sum"].float()
    got = dict(residual=g.to(s["residual"].dtype), x=g.to(_DT[s["case"]["in_dtype"]]))
    if s["weight"] is not None:
        got["weight"] = gw
    return got


# ---------------------------------------------------------------------------
# one pass

def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        from bayesian_scan_gb300 import kdn
        s = state
        if op == "norm_fwd":
            y, total, scale = kdn.add_rms_norm_fwd(s["x"], s["residual"], weight=s["weight"], eps=EPS,
                                                   out_dtype=_DT[c["out_dtype"]])
            return (y, total) if scale is None else (y, total, scale)
        if op == "norm_bwd":
            got = kdn.add_rms_norm_bwd(s["residual"], s["grad_y"], weight=s["weight"], grad_sum=s["grad_sum"],
                                       eps=EPS, x_dtype=_DT[c["in_dtype"]])
            return {n: t for n, t in got.items() if t is not None}
        args = [s[n] for n in ("q", "k", "v", "beta", "d", "A")]
        if op == "delta_step":
            # the old state is kept, as a program that may take a token back does
            return kdn.delta_step(*args, s["S0"], new_state=s["S1"], out_dtype=_DT[c["out_dtype"]]), s["S1"]
        if op == "delta_fwd":
            out, end = kdn.delta_scan_fwd(*args, S0=s["S0"], offsets=s["offsets"], final_state=c["state"],
                                          out_dtype=_DT[c["out_dtype"]], **s.get("bufs", {}))
            return (out, end) if c["state"] else out
        got = kdn.delta_scan_bwd(*args, s["g"], S0=s["S0"], offsets=s["offsets"], grad_final_state=s["g_final"],
                                 grad_S0=c["state"], **s.get("bufs", {}))
        return {n: t for n, t in got.items() if t is not None}
    return {"delta_fwd": _plain_delta, "delta_bwd": _plain_delta_bwd, "delta_step": _plain_step,
            "norm_fwd": _plain_norm, "norm_bwd": _plain_norm_bwd}[op](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    i, o = _ES[case["in_dtype"]], _ES[case["out_dtype"]]
    if case["op"].startswith("norm"):
        n, r = case["rows"] * case["C"], _ES[case["res_dtype"]]
        if case["op"] == "norm_bwd":
            return {"bytes": n * (3 * r + o + (i if i != r else 0)) + 8 * case["C"], "flops": 10.0 * n}
        scales = case["rows"] * -(-case["C"] // GROUP) * 4 if case["out_dtype"] == E4M3 else 0
        return {"bytes": n * (i + 2 * r + o) + scales + 4 * case["C"], "flops": 6.0 * n}
    B, H, T, dk, dv = (case[n] for n in ("B", "H", "T", "dk", "dv"))
    n = B * H * T
    states = (case["n_seq"] or B) * H * dk * dv * 4
    if case["op"] == "delta_bwd":
        return {"bytes": n * (i * 2 * (2 * dk + dv + 2) + o * dv) + H * 8 + states * (3 if case["state"] else 0),
                "flops": 18.0 * n * dk * dv}
    return {"bytes": n * (i * (2 * dk + dv + 2) + o * dv) + H * 4 + states * (2 if case["state"] else 0),
            "flops": 6.0 * n * dk * dv}


# ---------------------------------------------------------------------------
# the definitions, in 64 bits, token by token

def _groups_of_sequences(s):
    """(state rows, batch rows, first token, end): sequences that are walked together."""
    c = s["case"]
    if s["lens"] is not None:
        at = 0
        for n, length in enumerate(s["lens"]):
            yield [n], [0], at, at + length
            at += length
        return
    kept = c["T"] * c["H"] * c["dk"] * c["dv"] * 8 if c["op"] == "delta_bwd" else 1
    step = max(1, int(2.4e10 // kept))
    for b in range(0, c["B"], step):
        rows = list(range(b, min(c["B"], b + step)))
        yield rows, rows, 0, c["T"]


def _exact_forward(s, rows, batch, lo, hi, each):
    q, k, v, beta, d = (s[n][batch, :, lo:hi].double() for n in ("q", "k", "v", "beta", "d"))
    alpha = torch.exp(-s["A"].double().view(-1, 1) * d)
    dv, dk = s["case"]["dv"], s["case"]["dk"]
    S = (s["S0"][rows].double() if s["S0"] is not None
         else torch.zeros((len(rows), s["case"]["H"], dv, dk), device="cuda", dtype=torch.float64))
    for t in range(hi - lo):
        S = alpha[:, :, t, None, None] * S
        miss = v[:, :, t, :, None] - torch.matmul(S, k[:, :, t, :, None])
        S = torch.addcmul(S, beta[:, :, t, None, None] * miss, k[:, :, t, None, :])
        each(t, S, torch.matmul(S, q[:, :, t, :, None]).squeeze(-1))
    return S


def _exact_delta(s):
    out, ends = torch.zeros(s["v"].shape, device="cuda", dtype=torch.float64), []
    for rows, batch, lo, hi in _groups_of_sequences(s):
        def each(t, S, o):
            out[batch[0]:batch[-1] + 1, :, lo + t] = o
        ends.append(_exact_forward(s, rows, batch, lo, hi, each))
    return (out, torch.cat(ends)) if s["case"]["state"] else out


def _exact_delta_bwd(s):
    got = {n: torch.zeros(s[n].shape, device="cuda", dtype=torch.float64) for n in ("q", "k", "v", "beta", "d")}
    gA, starts = torch.zeros_like(s["A"], dtype=torch.float64), []
    A = s["A"].double()
    for rows, batch, lo, hi in _groups_of_sequences(s):
        kept = []
        end = _exact_forward(s, rows, batch, lo, hi, lambda t, S, o: kept.append(S))
        before = s["S0"][rows].double() if s["S0"] is not None else torch.zeros_like(end)
        q, k, v, beta, d, g = (s[n][batch, :, lo:hi].double() for n in ("q", "k", "v", "beta", "d", "g"))
        alpha = torch.exp(-A.view(-1, 1) * d)
        D = s["g_final"][rows].double() if s["g_final"] is not None else torch.zeros_like(end)
        here = slice(batch[0], batch[-1] + 1)
        for t in range(hi - lo - 1, -1, -1):
            S, prev = kept[t], kept[t - 1] if t else before
            kt, qt, gt = k[:, :, t, :, None], q[:, :, t, :, None], g[:, :, t, :, None]
            a, b = alpha[:, :, t, None, None], beta[:, :, t, None, None]
            got["q"][here, :, lo + t] = torch.matmul(S.transpose(-1, -2), gt).squeeze(-1)
            D = D + gt * qt.transpose(-1, -2)
            # S = M + b m k^T with M = a prev, m = v - M k
            M = a * prev
            m = v[:, :, t, :, None] - torch.matmul(M, kt)
            Dk = torch.matmul(D, kt)
            got["beta"][here, :, lo + t] = (Dk * m).sum((-1, -2))
            gm = b * Dk
            got["v"][here, :, lo + t] = gm.squeeze(-1)
            got["k"][here, :, lo + t] = (torch.matmul(D.transpose(-1, -2), b * m)
                                         - torch.matmul(M.transpose(-1, -2), gm)).squeeze(-1)
            gM = D - gm * kt.transpose(-1, -2)
            ga = (gM * M).sum((-1, -2))                      # of log alpha
            got["d"][here, :, lo + t] = -A * ga
            gA -= (d[:, :, t] * ga).sum(0)
            D = a * gM
        starts.append(D)
    got["A"] = gA
    if s["case"]["state"]:
        got["S0"] = torch.cat(starts)
    return got


def _exact_norm(total, weight):
    n = total / torch.sqrt((total * total).sum(-1, keepdim=True) / total.shape[-1] + EPS)
    return n if weight is None else n * weight


def exact(case, seed):
    s = prepare(case, seed)
    w = None if s.get("weight") is None else s["weight"].double()
    if case["op"] == "norm_fwd":
        total = s["x"].double() + s["residual"].double()
        y = _exact_norm(total.to(s["residual"].dtype).double(), w)
        if case["out_dtype"] != E4M3:
            return y, total
        edges = range(0, case["C"], GROUP)
        scale = torch.stack([y[:, c:c + GROUP].abs().amax(-1) / TOP for c in edges], -1)
        return torch.cat([y[:, c:c + GROUP] / scale[:, n:n + 1] for n, c in enumerate(edges)], -1), total, scale
    if case["op"] == "norm_bwd":                             # by differentiating the definition
        t = s["residual"].double().requires_grad_()
        w = None if w is None else w.requires_grad_()
        (_exact_norm(t, w) * s["grad_y"].double()).sum().backward()
        g = t.grad + s["grad_sum"].double()
        return dict(residual=g, x=g) if w is None else dict(residual=g, x=g, weight=w.grad)
    if case["op"] == "delta_step":
        c = dict(case, T=1, n_seq=0, op="delta_fwd")
        one = dict(s, case=c, **{n: s[n].unsqueeze(2) for n in ("q", "k", "v", "beta", "d")})
        out, end = _exact_delta(one)
        return out.squeeze(2), end
    return _exact_delta(s) if case["op"] == "delta_fwd" else _exact_delta_bwd(s)
