"""What AdapterProjection owns, and the calls of the adapters' classes that are refused before any CUDA
call (no GPU is touched)."""
import pytest
import torch

BF = torch.bfloat16


@pytest.fixture(scope="module")
def g():
    import grouped_expert_gemm_gb300 as g
    from grouped_expert_gemm_gb300 import build
    build.build()
    return g


def tables(d=64, n=72, r=8, N=2):
    return dict(weight=torch.zeros(d, n, dtype=BF), a=torch.zeros(N, r, d, dtype=BF),
                b=torch.zeros(N, r, n, dtype=BF), scale=torch.zeros(N))


def test_gradient_buffers_are_made_with_the_object(g):
    """A capture of the first backward records no clearing of them."""
    m = g.AdapterProjection(4, **tables(), device="cpu")
    dx, da, db, ws = m._grads
    assert dx.shape == (4, 64) and da.shape == (2, 8, 64) and db.shape == (2, 8, 72)
    assert not (dx.any() or da.any() or db.any()) and ws.numel() == m.ws_bytes
    m = g.AdapterProjection(4, **tables(), device="cpu", gradients=False)
    assert m._grads is None
    with pytest.raises(ValueError, match="without gradients"):
        m.backward(torch.zeros(4, 72, dtype=BF))
