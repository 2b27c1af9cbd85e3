"""The paged cache where its arithmetic is pushed: references that rise again and again."""
import math

import pytest
import torch

import cache_helpers as R
import hierarchical_top_block_gb300 as pisa
import paged_helpers as H
from paged_helpers import DEV, Paged

pytestmark = pytest.mark.gpu


def no_error():
    assert pisa.pisa_get_last_device_error() == 0


LEVELS = {
    "rising": lambda j: j,                    # every step's logits far above those of all before
    "pairs": lambda j: j // 2,                # only every other step's: the other stream's reference stays
    "saw": lambda j: j // 2 + 2 * (j % 3),    # up and down, the peaks rising
    "falling": lambda j: -j,                  # a reference far above what comes: weights that vanish
    "late": lambda j: 0 * j + 9 * (j == j.max()),
}


@pytest.mark.parametrize("d,S", [(64, 16), (128, 64)])
@pytest.mark.parametrize("G,new", [(4, 5), (16, 3), (8, 16), (4, 40), (2, 128)])
@pytest.mark.parametrize("levels", LEVELS)
def test_references_rise(d, S, G, new, levels):
    """Steps of 128 keys whose logits differ by tens from one to the next, a dozen of them a block: tiles of at most 128 rows
    (streams by steps; 20, 48 and 128 rows) and of more (by rows), so that each stream makes weights again and rescales
    its output sums several times.  Blocks take about 13 steps: 128 jobs of 16 over 152 blocks."""
    B, H_kv, n = 16, 8, 2000
    c = Paged([n - new - 7 * (b % 5) for b in range(B)], [new] * B, H_kv, d, S, seed=new + d)
    along = torch.full((d,), d ** -0.5, device=DEV)
    step = 12 * math.sqrt(d) / 8  # q has 8 along it: 12 a level in the logits
    for b in range(B):
        level = LEVELS[levels](torch.arange(c.lens[b] + new, device=DEV) // 128).float() * step
        k = 0.3 * c.rand(c.lens[b] + new, H_kv, d).float() + level[:, None, None] * along
        c.put(b, k.to(torch.bfloat16), c.rand(c.lens[b] + new, H_kv, d))
    q = (0.5 * c.rand(c.R, H_kv * G, d).float() + 8 * along).to(torch.bfloat16)
    wo, wl, bo, bl = H.attend_many(c, q)
    for _ in range(3):
        o, lse = pisa.pisa_paged_attn(q, c.K, c.V, c.table, c.len, row_start=c.rows)
        R.close(o, wo, bo, "o")
        R.close(lse, wl, bl, "lse")
    no_error()
