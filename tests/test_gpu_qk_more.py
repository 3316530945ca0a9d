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
