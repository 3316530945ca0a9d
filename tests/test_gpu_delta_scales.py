"""The delta rule's outputs and gradients are linear in v (with S0), in grad_out
(with grad_final_state) and in q (grad_final_state with it, as D is a sum of
do q^T): a power of two on one of them is a power of two on each result, to the
bit, as operands have powers of two of their own and fp32 and bf16 are far
from the ends of their ranges."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def kdn():
    from bayesian_scan_gb300 import kdn as k
    return k


# token by token, in chunks, narrow heads with zeros behind, in parts
@pytest.mark.parametrize("T,dk,dv,dt", [(200, 64, 64, F32), (200, 128, 128, BF16), (200, 64, 64, BF16), (200, 128, 32, BF16),
                                        (2500, 128, 128, BF16), (2100, 64, 64, BF16)])
@pytest.mark.parametrize("v,g,q", [(-40, 0, 0), (0, -40, 0), (40, 0, 0), (0, 40, 0), (-45, -45, 0), (50, 50, 0), (-60, 20, 0),
                                   (0, 0, -20), (0, 0, -40), (0, 0, 20), (0, 0, 60), (-30, -30, -30), (30, -50, 40)])
def test_powers_of_two_pass_through(kdn, T, dk, dv, dt, v, g, q):
    r = torch.Generator(device="cuda").manual_seed(T + dk)
    n = lambda *s: torch.randn(*s, device="cuda", generator=r)  # noqa: E731
    unit = lambda x: torch.nn.functional.normalize(x, dim=-1)  # noqa: E731
    x = dict(q=unit(n(1, 2, T, dk)), k=unit(n(1, 2, T, dk)), v=n(1, 2, T, dv), beta=torch.sigmoid(n(1, 2, T)),
             d=torch.nn.functional.softplus(n(1, 2, T)))
    x = dict({m: t.to(dt) for m, t in x.items()}, A=torch.tensor([0.2, 0.03], device="cuda"))
    S0, gf, go = n(1, 2, dv, dk), n(1, 2, dv, dk), n(1, 2, T, dv).to(dt)

    def run(v, g, q):
        y = dict(x, v=x["v"] * 2.0 ** v, q=x["q"] * 2.0 ** q)
        o, end = kdn.delta_scan_fwd(**y, S0=S0 * 2.0 ** v, out_dtype=F32)
        got = kdn.delta_scan_bwd(**y, grad_out=go * 2.0 ** g, S0=S0 * 2.0 ** v, grad_final_state=gf * 2.0 ** (g + q))
        return dict(got, o=o, end=end)

    want, got = run(0, 0, 0), run(v, g, q)
    by = dict(o=v + q, end=v, q=v + g, v=g + q, S0=g + q, k=v + g + q, beta=v + g + q, d=v + g + q, A=v + g + q)
    for name, p in by.items():
        a, b = got[name].double(), want[name].double() * 2.0 ** p
        if name == "A" and p <= -90:
            # pairs 36 powers of two of decay and more apart are no normal numbers here: a token's sum of up to
            # 2^13 such terms is off by 2^13 2^-149, far below a step of the largest, but may turn each addition of
            # A's sum, over the tokens and the chunks' shares, to the neighbouring number
            terms = (x["d"].double() * want["d"].double()).abs().sum((0, 2)) / x["A"].double() * 2.0 ** p
            assert ((a - b).abs() <= (T + 64) * 2.0 ** -23 * terms).all(), name
        else:
            assert torch.equal(a, b), name
