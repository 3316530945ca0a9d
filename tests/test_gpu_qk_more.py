"""Queries and keys: calls beside the ordinary ones."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hk", [(0, 2), (3, 0)])
def test_a_tensor_without_heads(Hq, Hk):
    # as if it were not given, but for its empty output and its weight's gradient of zeros
    from bayesian_scan_gb300 import kdn
    g = torch.Generator().manual_seed(1)
    q, k = torch.randn(2, 5, Hq, 32, generator=g).cuda(), torch.randn(2, 5, Hk, 32, generator=g).cuda()
    gq, gk = torch.randn(2, Hq, 5, 32, generator=g).cuda(), torch.randn(2, Hk, 5, 32, generator=g).cuda()
    w, f = torch.rand(32, generator=g).cuda(), torch.rand(16, generator=g).cuda()
    both = kdn.qk_norm_rope_fwd(q, k, inv_freq=f, wq=w, wk=w)
    alone = kdn.qk_norm_rope_fwd(q if Hq else None, k if Hk else None, inv_freq=f, wq=w, wk=w)
    back = kdn.qk_norm_rope_bwd(q, k, gq, gk, inv_freq=f, wq=w, wk=w)
    want = kdn.qk_norm_rope_bwd(q if Hq else None, k if Hk else None, gq, gk, inv_freq=f, wq=w, wk=w)
    for i, (n, H, heads) in enumerate((("q", Hq, (2, Hq, 5, 32)), ("k", Hk, (2, Hk, 5, 32)))):
        assert both[i].shape == heads and back[n].shape == (2, 5, H, 32)
        if H:
            assert torch.equal(both[i], alone[i])
            assert torch.equal(back[n], want[n]) and torch.equal(back["w" + n], want["w" + n])
        else:
            assert (back["w" + n] == 0).all()


@pytest.mark.parametrize("T", [5, 1500])
def test_the_weight_of_a_tensor_without_heads_is_not_touched(T):
    # (through the C ABI: an address that is no place for a weight, with half of the head rotated)
    import ctypes
    from bayesian_scan_gb300 import kdn
    g = torch.Generator().manual_seed(2)
    q, f = torch.randn(2, T, 16, 32, generator=g).cuda(), torch.rand(8, generator=g).cuda()
    go = torch.randn(2, 16, T, 32, generator=g).cuda()
    want = kdn.qk_norm_rope_fwd(q, None, inv_freq=f)[0]
    back = kdn.qk_norm_rope_bwd(q, None, go, None, inv_freq=f)["q"]
    out, gq = torch.empty_like(want), torch.empty_like(q)
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    nowhere, stream = ctypes.c_void_p(20), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert kdn.lib.kdn_qk_norm_rope_fwd(p(q), 512, None, 0, None, nowhere, 1, 1e-6, None, 1, p(f), None, 16, 0, p(out),
                                        None, 2, T, 16, 0, 32, 0, 0, stream) == 0
    assert kdn.lib.kdn_qk_norm_rope_bwd(p(q), 512, None, 0, None, nowhere, 1, 1e-6, None, 1, p(f), None, 16, 0, p(go),
                                        None, p(gq), 512, None, 0, None, None, 2, T, 16, 0, 32, 0, 0, None, 0,
                                        stream) == 0
    assert torch.equal(out, want) and torch.equal(gq, back)
