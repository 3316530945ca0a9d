"""Calls on a stream given by hand, while torch's current stream still reads
memory that it has already let go."""
import pytest
import torch

from bayesian_scan_gb300 import kdn

pytestmark = pytest.mark.gpu


def test_memory_of_the_current_stream_is_left_alone():
    # the current stream is kept busy; a tensor that it has yet to copy is let go of, and calls on
    # another stream allocate tensors of its size
    B, T, C = 4, 4096, 512
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(B, T, C, device="cuda", generator=g)
    d, A = torch.rand(B, T, C, device="cuda", generator=g), torch.rand(C, device="cuda", generator=g)
    q, go = x.unflatten(2, (4, 128)), torch.randn(B, 4, T, 128, device="cuda", generator=g)
    want = kdn.gated_scan_fwd(x, d, A)
    back = kdn.gated_scan_bwd(x, d, A, want[0], x)
    prepared = kdn.qk_norm_rope_fwd(q, None)[0]
    grad = kdn.qk_norm_rope_bwd(q, None, go, None, grad_w=True)
    copies = [torch.empty_like(x) for _ in range(8)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)                         # some 50 ms, which no call below waits for
    for i, c in enumerate(copies):
        c.copy_(torch.full_like(x, float(i)))              # the tensor copied from is free once queued
    got = kdn.gated_scan_fwd(x, d, A, stream=s)
    got_back = kdn.gated_scan_bwd(x, d, A, want[0], x, stream=s)
    got_prepared = kdn.qk_norm_rope_fwd(q, None, stream=s)[0]
    got_grad = kdn.qk_norm_rope_bwd(q, None, go, None, grad_w=True, stream=s)
    torch.cuda.synchronize()
    for i, c in enumerate(copies):
        assert (c == float(i)).all()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert all(torch.equal(back[n], got_back[n]) for n in back)
    assert torch.equal(prepared, got_prepared)
    assert torch.equal(grad["q"], got_grad["q"]) and torch.equal(grad["wq"], got_grad["wq"])
