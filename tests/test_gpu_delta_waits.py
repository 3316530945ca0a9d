"""The delta rule's waits on the tensor cores end: with a chunk that is never
announced (fault injection) the calls return, the error is reported, and the
next call is right again."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def kdn():
    from bayesian_scan_gb300 import kdn as k
    return k


def draw(B, H, T, dk, dv, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    unit = lambda x: torch.nn.functional.normalize(x, dim=-1)  # noqa: E731
    x = dict(q=unit(n(B, H, T, dk)), k=unit(n(B, H, T, dk)), v=n(B, H, T, dv), beta=torch.sigmoid(n(B, H, T)),
             d=torch.nn.functional.softplus(n(B, H, T)))
    x = {name: t.to(BF16).cuda() for name, t in x.items()}
    return dict(x, A=0.1 * torch.rand(H, generator=g).cuda()), n(B, H, dv, dk).cuda(), n(B, H, T, dv).to(BF16).cuda()


# one walk a head, with the first, a middle and the last chunk left out; narrow heads; walks in parts; more heads than SMs
@pytest.mark.parametrize("B,H,T,dk,dv,chunk", [(1, 2, 300, 128, 128, 0), (1, 2, 300, 128, 128, 2), (1, 2, 300, 128, 128, 4),
                                               (1, 2, 300, 64, 64, 1), (1, 1, 2500, 128, 128, 1), (20, 16, 200, 128, 128, 1)])
def test_a_chunk_that_never_comes_times_out(kdn, B, H, T, dk, dv, chunk):
    x, S0, go = draw(B, H, T, dk, dv, T + dk)
    out, end = kdn.delta_scan_fwd(**x, S0=S0)
    grads = kdn.delta_scan_bwd(**x, grad_out=go, S0=S0)
    assert kdn.get_device_error() == kdn.KDN_OK
    kdn.set_wait_limit_ns(20_000_000)
    kdn.debug_stall_delta_chunk(chunk)
    try:
        kdn.delta_scan_fwd(**x, S0=S0)
        assert kdn.get_device_error() == kdn.KDN_ERR_TIMEOUT
        kdn.delta_scan_bwd(**x, grad_out=go, S0=S0)
        assert kdn.get_device_error() == kdn.KDN_ERR_TIMEOUT
    finally:
        kdn.debug_stall_delta_chunk(-1)
        kdn.set_wait_limit_ns(0)
    assert kdn.get_device_error() == kdn.KDN_OK
    again, end2 = kdn.delta_scan_fwd(**x, S0=S0)
    assert torch.equal(again, out) and torch.equal(end2, end)
    more = kdn.delta_scan_bwd(**x, grad_out=go, S0=S0)
    assert all(torch.equal(more[n], grads[n]) for n in grads)
    assert kdn.get_device_error() == kdn.KDN_OK


def test_a_chunk_that_no_sequence_has_stalls_nothing(kdn):
    x, S0, go = draw(1, 2, 300, 128, 128, 3)
    want = kdn.delta_scan_fwd(**x, S0=S0)[0]
    kdn.debug_stall_delta_chunk(5)
    try:
        assert torch.equal(kdn.delta_scan_fwd(**x, S0=S0)[0], want)
        kdn.delta_scan_bwd(**x, grad_out=go, S0=S0)
    finally:
        kdn.debug_stall_delta_chunk(-1)
    assert kdn.get_device_error() == kdn.KDN_OK
