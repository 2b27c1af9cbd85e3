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


@pytest.mark.parametrize("d,S", [(64, 16), (64, 32), (128, 16), (128, 64)])
@pytest.mark.parametrize("G,new", [(1, 1), (4, 1), (16, 1), (4, 3), (16, 5), (4, 40), (4, 90)])
@pytest.mark.parametrize("long", [False, True])
def test_infinite_values(d, S, G, new, long):
    """Values of +-infinity and NaN among the keys that every row sees: the output has them, whichever kernel runs (few rows,
    streams by steps, by rows), and its other columns are as always."""
    n = 5000 if long else 150
    c = Paged([n, 40, n // 2], [new] * 3, 2, d, S, seed=G + new)
    for b in range(3):
        k, v = c.get(c.K, b, c.lens[b]), c.get(c.V, b, c.lens[b])
        last = c.lens[b] - 1
        v[0, 0, 0] = v[last, 0, 1] = v[17, 0, d - 1] = math.inf
        v[5, 0, 2] = v[6, 0, 2] = -math.inf
        v[8, 0, 3], v[last, 0, 3] = math.inf, -math.inf  # their sum is no number
        v[9, 1, 9] = math.nan
        c.put(b, k, v)
    q = c.rand(c.R, 2 * G, d)
    o, lse = pisa.pisa_paged_attn(q, c.K, c.V, c.table, c.len, row_start=c.rows, causal=False)
    wo, wl, bo, bl = H.attend(c, q, causal=False)
    assert wo.isposinf().any() and wo.isneginf().any() and wo.isnan().any()
    R.close(o, wo, bo.nan_to_num(0), "o")
    R.close(lse, wl, bl, "lse")
    no_error()


@pytest.mark.parametrize("d,S", [(64, 16), (64, 32), (128, 64)])
@pytest.mark.parametrize("G,new", [(4, 1), (16, 1), (4, 3), (4, 20), (4, 90)])
def test_large_values(d, S, G, new):
    """Values of 5e37 at keys whose logits rise by half from one to the next.  The largest weight is 1 and the sums of weights of
    them are at most 1 / (1 - e^-0.5) < 2.6, so with weights of at most 1 no sum is above 1.3e38 and the output is finite; with
    weights relative to a reference 2^3 and more below the largest logit it is not."""
    B, H_kv, n = 6, 4, 5000
    c = Paged([n - 31 * b for b in range(B)], [new] * B, H_kv, d, S, seed=G + new)
    along = torch.full((d,), d ** -0.5, device=DEV)
    for b in range(B):
        k, v = c.get(c.K, b, c.lens[b]).clone(), c.get(c.V, b, c.lens[b]).clone()
        for i in range(11):
            at = 400 * i + 333
            k[at] = ((1 + 0.25 * i) * math.sqrt(d) * along).to(torch.bfloat16)  # logit 2 + i / 2 for q of 2 along it
            v[at] = torch.where(torch.arange(d, device=DEV) % 2 == 0, 5e37, -5e37).to(torch.bfloat16)
        c.put(b, k, v)
    q = (0.3 * c.rand(c.R, H_kv * G, d).float() + 2 * along).to(torch.bfloat16)
    o, lse = pisa.pisa_paged_attn(q, c.K, c.V, c.table, c.len, row_start=c.rows)
    wo, wl, bo, bl = H.attend_many(c, q)
    assert wo.abs().max() > 1e36
    R.close(o, wo, bo, "o")
    R.close(lse, wl, bl, "lse")
    no_error()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,new", [(4, [1, 1, 1]), (4, [3, 1, 4]), (16, [1, 1, 1]), (4, [70, 1, 40]), (16, [20, 17, 8]), (1, [300, 257, 130])])
@pytest.mark.parametrize("accumulate", [False, True])
def test_weights_of_rows_that_saw_nothing(d, G, new, accumulate):
    """Rows with lse = -inf give nothing, whatever lies in q there; the others' weights are as always."""
    H_kv = 2
    c = Paged([700, 40, 129], new, H_kv, d, 16, seed=d + G)
    q = c.rand(c.R, H_kv * G, d, scale=1.5)
    _, lse = pisa.pisa_paged_attn(q, c.K, c.V, c.table, c.len, row_start=c.rows)
    off = torch.rand((c.R, H_kv * G), generator=c.g, device=DEV) < 0.3
    off[c.R - 1, 0], off[0, -1] = True, True
    lse[off] = -math.inf
    w = c.w.clone()
    want, bound = H.weights(c, q, lse)
    bad = torch.tensor([math.nan, math.inf, -math.inf, 1e38], device=DEV)[torch.arange(int(off.sum()), device=DEV) % 4]
    q[off] = bad[:, None].to(torch.bfloat16)
    pisa.pisa_paged_weights(q, lse, c.K, w, c.table, c.len, row_start=c.rows, accumulate=accumulate)
    live = ~want.isnan()
    assert (w[~live] == -7).all()
    if accumulate:  # one more sum
        want, bound = want - 7, bound + 2.0 ** -24 * (want + 7)
    R.close(w[live], want[live], bound[live], "w")
    # no row of a sequence saw anything: no key gets anything
    lse.fill_(-math.inf)
    q.fill_(math.nan)
    w = c.w.clone()
    pisa.pisa_paged_weights(q, lse, c.K, w, c.table, c.len, row_start=c.rows, accumulate=accumulate)
    assert (w[~live] == -7).all() and (w[live] == (-7 if accumulate else 0)).all()
    no_error()


@pytest.mark.parametrize("G", [1, 16])
def test_weights_without_rows_in_the_smallest_pool(G):
    """One page of 16 keys, no token at all: a call that puts weights in place clears them, and reads neither q nor, in its
    stead, a row of the pool (which holds NaN behind the sequence's end)."""
    c = Paged([7], [0], 1, 64, 16, M=1, spare=0)
    q, lse = torch.empty(0, G, 64, dtype=torch.bfloat16, device=DEV), torch.empty(0, G, device=DEV)
    for rows in (None, c.rows):
        c.w.fill_(-7)
        pisa.pisa_paged_weights(q, lse, c.K, c.w, c.table, c.len, row_start=rows, accumulate=False)
        got = c.w.flatten().tolist()
        assert got == [0.0] * 7 + [-7.0] * 9
    no_error()
