"""What the binding does around the gated recurrence's and the query/key
preparation's calls: devices, sizes, streams and buffers.  Nothing here
launches a kernel; device tensors are stood in for by objects."""
import itertools

import pytest
import torch

from bayesian_scan_gb300 import kdn


class On:
    """A tensor as far as the device checks look at one."""

    def __init__(self, device):
        self.device_index, self.is_cuda = device, device >= 0
        self.device = torch.device("cuda", device) if device >= 0 else torch.device("cpu")

    def get_device(self):
        return self.device_index


@pytest.mark.parametrize("n", [1, 2, 3, 4])
def test_every_operand_is_on_the_current_device(n, monkeypatch):
    # host tensors (-1), the current device's (0) and another's (1), None among them, in every order
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    for devices in itertools.product((-1, 0, 1, None), repeat=n):
        given = [d for d in devices if d is not None]
        want = bool(given) and all(d == 0 for d in given)
        tensors = [None if d is None else On(d) for d in devices]
        assert kdn._here(None, *tensors) == want, devices
        assert not kdn._here("a stream", *tensors)


def meta(*shape, dtype=torch.float32):
    return torch.empty(shape, device="meta", dtype=dtype)


BIG = 2 ** 32 + 5      # cut to 32 bits: 5


@pytest.mark.parametrize("call", [
    lambda: kdn.gated_scan_fwd(meta(1, BIG, 1), meta(1, BIG, 1), meta(1)),
    lambda: kdn.gated_scan_fwd(meta(BIG, 1, 1), meta(BIG, 1, 1), meta(1)),
    lambda: kdn.gated_scan_fwd(meta(1, BIG, 1, 1), meta(1, BIG, 1, 1), meta(BIG, 1)),
    lambda: kdn.gated_scan_fwd(meta(1, 2, BIG), meta(1, 2, BIG), meta(BIG)),
    lambda: kdn.gated_scan_fwd(meta(1, 2, 1), meta(1, 2, 1), meta(1), offsets=meta(BIG + 1, dtype=torch.int32)),
    lambda: kdn.gated_scan_bwd(meta(1, BIG, 1), meta(1, BIG, 1), meta(1), meta(1, BIG, 1), meta(1, BIG, 1)),
    lambda: kdn.gated_step(meta(BIG, 1), meta(BIG, 1), meta(1), meta(BIG, 1)),
    lambda: kdn.gated_step(meta(2, BIG, 1), meta(2, BIG, 1), meta(BIG, 1), meta(2, BIG, 1)),
    lambda: kdn.qk_norm_rope_fwd(meta(1, BIG, 1, 16), meta(1, BIG, 1, 16)),
    lambda: kdn.qk_norm_rope_fwd(meta(BIG, 1, 1, 16), None),
    lambda: kdn.qk_norm_rope_fwd(None, meta(1, 1, BIG, 16)),
    lambda: kdn.qk_norm_rope_bwd(meta(1, BIG, 1, 16), None, meta(1, 1, BIG, 16), None),
    lambda: kdn.gated_scan_bwd_workspace(BIG, 1, 1, 1),
    lambda: kdn.gated_scan_bwd_workspace(1, 1, 1, 1, nseq=BIG),
    lambda: kdn.qk_norm_rope_bwd_workspace(1, 1, BIG, 1, 16),
])
def test_sizes_that_32_bits_do_not_hold_are_refused(call):
    with pytest.raises(ValueError, match=r"below 2\*\*31"):
        call()


def test_a_workspace_is_as_long_as_it_says():
    # one byte seen a million times is not a workspace; nor is every second byte
    x, A, q = torch.zeros(2, 5, 8), torch.zeros(8), torch.zeros(2, 5, 3, 32)
    g = torch.zeros(2, 3, 5, 32)
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(1 << 20), torch.zeros(1 << 21, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace must be contiguous"):
            kdn.gated_scan_bwd(x, x, A, x, x, workspace=ws)
        with pytest.raises(ValueError, match="workspace must be contiguous"):
            kdn.qk_norm_rope_bwd(q, q, g, g, grad_w=True, workspace=ws)


def test_the_diagonal_backward_s_workspace_too():
    class Dev(torch.Tensor):
        is_cuda = True

    q, v, d = (torch.zeros(1, 2, 5, 16).as_subclass(Dev) for _ in range(3))
    d = d[..., 0].contiguous()
    ws = torch.zeros(1, dtype=torch.uint8).expand(1 << 24)
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        kdn.diag_scan_bwd(q, q, v, v, d, torch.zeros(2), v, workspace=ws)


@pytest.mark.parametrize("Hq,Hk", [(0, 2), (2, 0)])
@pytest.mark.parametrize("weight", [False, True])
def test_no_heads_have_zero_weight_gradients(Hq, Hk, weight, monkeypatch):
    # a tensor of no heads adds nothing to its weight's gradient, which no kernel writes
    empty = torch.empty

    def poisoned(*args, **kw):
        t = empty(*args, **kw)
        return t.fill_(float("nan")) if t.is_floating_point() else t

    monkeypatch.setattr(torch, "empty", poisoned)
    monkeypatch.setattr(torch, "empty_like", lambda t, **kw: poisoned(t.shape, dtype=t.dtype))
    monkeypatch.setattr(kdn.lib, "kdn_qk_norm_rope_bwd", lambda *args: 0)
    monkeypatch.setattr(kdn, "_on_one_device", lambda *args, **kw: None)
    monkeypatch.setattr(kdn, "_stream", lambda s: 0)
    q, k = torch.zeros(2, 5, Hq, 32), torch.zeros(2, 5, Hk, 32)
    w = torch.ones(32) if weight else None
    got = kdn.qk_norm_rope_bwd(q, k, torch.zeros(2, Hq, 5, 32), torch.zeros(2, Hk, 5, 32), wq=w, wk=w, grad_w=True)
    none, some = ("wq", "wk") if Hq == 0 else ("wk", "wq")
    assert got[none].shape == (32,) and (got[none] == 0).all()
    assert got[some].isnan().all()                           # (the library's to write)


@pytest.mark.parametrize("call", [
    lambda: kdn.qk_norm_rope_fwd(meta(1, 1, 1, 2 ** 32 + 16), None),
    lambda: kdn.qk_norm_rope_bwd(meta(1, 1, 1, 2 ** 32 + 16), None, meta(1, 1, 1, 2 ** 32 + 16), None),
])
def test_a_head_that_32_bits_do_not_hold_is_refused(call):
    with pytest.raises(ValueError, match=r"below 2\*\*31"):
        call()
