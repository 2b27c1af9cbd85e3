"""Value scales that are no numbers: an infinity (a cache that another program filled) shows in the outputs, and
the log-sum-exp, which no value is part of, stays right."""
import math

import pytest
import torch

import cache_helpers as R
import hierarchical_top_block_gb300 as pisa

pytestmark = pytest.mark.gpu
DEV = "cuda"


def cache(g, N, d):
    K, V = (torch.randn((1, 1, N, d), generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    (kc, ks, _), (vc, vs, _) = R.quantise64(K), R.quantise64(V)
    return kc, vc, ks, vs


def expected(q, kc, ks):
    k = kc[0, 0].double() * ks[0, 0].double()[:, None]
    _, lse, _, tl = R.attend64(q.double(), k, torch.zeros_like(k))
    return lse, tl


@pytest.mark.parametrize("scale", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("Rn", [2, 6, 20, 50])
@pytest.mark.parametrize("N", [100, 5000])
def test_prefix(N, Rn, scale):
    g = torch.Generator(device=DEV).manual_seed(N + Rn)
    kc, vc, ks, vs = cache(g, N, 64)
    q = torch.randn((Rn, 4, 64), generator=g, device=DEV).to(torch.bfloat16)
    vs[0, 0, N // 3] = scale
    n = torch.tensor([N], dtype=torch.int32, device=DEV)
    o, lse = pisa.pisa_prefix_attn(q, kc, vc, n, k_scale=ks, v_scale=vs)
    l, tl = expected(q.reshape(-1, 64), kc, ks)
    assert not torch.isfinite(o).any()
    R.close(lse.reshape(-1), l, tl, "lse")
    assert pisa.pisa_get_last_device_error() == 0


@pytest.mark.parametrize("scale", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("H_q", [4, 16])
@pytest.mark.parametrize("N", [100, 2048])
def test_selected_blocks(N, H_q, scale):
    g = torch.Generator(device=DEV).manual_seed(N + H_q)
    kc, vc, ks, vs = cache(g, N, 64)
    q = torch.randn((1, H_q, 64), generator=g, device=DEV).to(torch.bfloat16)
    vs[0, 0, N // 3] = scale
    idx = torch.arange(32, dtype=torch.int32, device=DEV).reshape(1, 1, 32)
    idx = torch.where(idx < -(-N // 64), idx, -1)
    O, L = pisa.pisa_sparse_attn_cache(q, kc, vc, ks, vs, idx, torch.tensor([N - 1], dtype=torch.int32, device=DEV))
    l, tl = expected(q[0], kc, ks)
    assert not torch.isfinite(O).any()
    R.close(L[0], l, tl, "LSE")
    assert pisa.pisa_get_last_device_error() == 0
