"""What a row attended on its own, at the ends of fp32's range, joined with a prefix."""
import math

import pytest
import torch

import hierarchical_top_block_gb300 as pisa

pytestmark = pytest.mark.gpu
DEV = "cuda"
LARGEST = torch.finfo(torch.float32).max


def normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


@pytest.mark.parametrize("own", [-LARGEST, -3e38, -1e9, 0.0, 1e9, 3e38, LARGEST])
@pytest.mark.parametrize("N,length", [(40, 0), (40, 40), (30000, 30000)])
@pytest.mark.parametrize("Rn", [2, 6, 20, 50])
@pytest.mark.parametrize("bits", [8, 16])
def test_own_results_far_away(bits, Rn, N, length, own):
    """Masks of the type's lowest value give such log-sum-exps: finite, so an empty prefix leaves o_own as it is,
    and a prefix with keys outweighs it."""
    g = torch.Generator(device=DEV).manual_seed(N + Rn)
    H_q, d = 4, 64
    q, oo = normal(g, Rn, H_q, d), normal(g, Rn, H_q, d)
    K, V, ks, vs = normal(g, 1, 1, N, d), normal(g, 1, 1, N, d), None, None
    if bits == 8:
        K, V = ((x.float() * 20).round().clamp(-127, 127).to(torch.int8) for x in (K, V))
        ks, vs = (torch.full((1, 1, N), 0.05, device=DEV) for _ in range(2))
    n = torch.tensor([length], dtype=torch.int32, device=DEV)
    ll = torch.full((Rn, H_q), own, device=DEV)
    alone, lse_alone = pisa.pisa_prefix_attn(q, K, V, n, k_scale=ks, v_scale=vs)
    o, lse = pisa.pisa_prefix_attn(q, K, V, n, k_scale=ks, v_scale=vs, o_own=oo, lse_own=ll)
    if length == 0 or own > 1e8:  # the own result as it is
        assert torch.equal(o, oo) and torch.equal(lse, ll)
    elif own < -1e8:
        assert torch.equal(o, alone) and torch.equal(lse, lse_alone)
    else:  # weights of 1 and e^lse, whose logarithm is at least log of `length` less the logits' range
        want = torch.logaddexp(lse_alone.double(), ll.double())
        assert (lse.double() - want).abs().max() <= 2.0 ** -17 + 2.0 ** -22 * want.abs().max()
    assert pisa.pisa_get_last_device_error() == 0
