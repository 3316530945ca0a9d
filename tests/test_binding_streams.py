"""A call that is given a stream takes what it allocates from that stream's own
memory: a block that torch's current stream has let go may still be read by
work queued there, which the given stream does not wait for.  No GPU: the
tensors are host ones that say they are CUDA tensors, the library is not
called, and torch's stream context only records that it is entered."""
import contextlib

import pytest
import torch

from bayesian_scan_gb300 import kdn


class Dev(torch.Tensor):
    is_cuda = True

    def get_device(self):
        return 0


class Stream:
    cuda_stream = 7

    def __init__(self):
        self.device = torch.device("cuda", 0)


class Library:
    """Every call returns KDN_OK; the workspace queries are the library's."""

    def __init__(self, lib):
        self.lib = lib

    def __getattr__(self, name):
        return getattr(self.lib, name) if name.endswith("_workspace") else lambda *args: 0


def dev(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(Dev)


@pytest.fixture
def under(monkeypatch):
    """Records of (function, streams it was called under)."""
    seen, inside = [], []

    @contextlib.contextmanager
    def stream_context(s):
        inside.append(s)
        yield
        inside.pop()

    def recording(f):
        def call(*args, **kw):
            seen.append((f.__name__, tuple(inside)))
            with torch._C.DisableTorchFunctionSubclass():
                return f(*args, **kw).as_subclass(Dev)
        return call

    # on a machine without a GPU an allocation "on cuda" is one on the host
    def empty(*args, device=None, **kw):
        return real_empty(*args, **kw)

    real_empty = torch.empty
    empty.__name__ = "empty"
    monkeypatch.setattr(torch.cuda, "stream", stream_context)
    monkeypatch.setattr(torch, "empty", recording(empty))
    monkeypatch.setattr(torch, "empty_like", recording(torch.empty_like))
    monkeypatch.setattr(kdn, "lib", Library(kdn.lib))
    monkeypatch.setattr(kdn, "_on_one_device", lambda *args, **kw: None)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    monkeypatch.setattr(Dev, "record_stream", lambda self, s: None)
    return seen


def diag():
    B, H, T, d = 2, 3, 5, 16
    return (*(dev(B, H, T, d) for _ in range(4)), dev(B, H, T), dev(H))


def gated():
    return dev(2, 5, 8), dev(2, 5, 8), dev(8)


# calls, and how many allocations each has to make
CALLS = {
    "diag_scan_fwd": (lambda **kw: kdn.diag_scan_fwd(*diag(), **kw), 2),
    "diag_mobius_scan_fwd": (
        lambda **kw: kdn.diag_mobius_scan_fwd(*diag(), *(dev(6, 5) for _ in range(4)), dev(6), **kw), 3),
    "lin_scan_fwd": (lambda **kw: kdn.lin_scan_fwd(*diag(), **kw), 2),
    "diag_scan_bwd": (lambda **kw: kdn.diag_scan_bwd(*diag(), dev(2, 3, 5, 16), **kw), 8),
    "diag_step": (lambda **kw: kdn.diag_step(
        *(dev(2, 3, 16) for _ in range(4)), dev(2, 3), dev(3), dev(2, 2, 3, 16, 16), **kw), 1),
    "mobius_scan": (lambda **kw: kdn.mobius_scan(*(dev(4, 7) for _ in range(4)), dev(4), **kw), 1),
    "gated_scan_fwd": (lambda **kw: kdn.gated_scan_fwd(*gated(), **kw), 2),
    "gated_scan_fwd, other type": (lambda **kw: kdn.gated_scan_fwd(*gated(), out_dtype=torch.bfloat16, **kw), 2),
    "gated_scan_bwd": (lambda **kw: kdn.gated_scan_bwd(*gated(), dev(2, 5, 8), dev(2, 5, 8), **kw), 5),
    "gated_scan_bwd, from a state": (
        lambda **kw: kdn.gated_scan_bwd(*gated(), dev(2, 5, 8), dev(2, 5, 8), h0=dev(2, 8), **kw), 5),
    "gated_step": (lambda **kw: kdn.gated_step(dev(2, 8), dev(2, 8), dev(8), dev(2, 8), **kw), 1),
    "qk_norm_rope_fwd": (lambda **kw: kdn.qk_norm_rope_fwd(dev(2, 5, 3, 32), dev(2, 5, 1, 32), **kw), 2),
    "qk_norm_rope_bwd": (lambda **kw: kdn.qk_norm_rope_bwd(
        dev(2, 5, 3, 32), dev(2, 5, 1, 32), dev(2, 3, 5, 32), dev(2, 1, 5, 32), wq=dev(32), grad_w=True, **kw), 5),
}


@pytest.mark.parametrize("name", CALLS)
def test_allocations_are_the_given_streams(name, under):
    call, n = CALLS[name]
    s = Stream()
    call(stream=s)
    assert len(under) == n and all(streams == (s,) for _, streams in under), under
    # without a stream: torch's current one, whatever it is
    under.clear()
    call()
    assert len(under) == n and all(streams == () for _, streams in under), under
