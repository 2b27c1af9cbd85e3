"""The paged cache: write, attention, weights and eviction against their 64-bit forms, alone and in a run."""
import math

import pytest
import torch

import cache_helpers as R
import hierarchical_top_block_gb300 as pisa
import paged_helpers as H
from paged_helpers import DEV, Paged, i32

pytestmark = pytest.mark.gpu


def no_error():
    assert pisa.pisa_get_last_device_error() == 0


BAD_INDEX = 5


# ---- write -----------------------------------------------------------------------------------
@pytest.mark.parametrize("d,H_kv,S,lens,new", [
    (64, 1, 16, [0], [1]), (128, 8, 64, [0, 63, 64, 1000], [1, 1, 1, 1]), (64, 2, 16, [0, 5, 15, 16, 31], [33, 0, 1, 17, 100]),
    (128, 3, 32, [7, 0], [0, 0]), (128, 8, 16, [100, 3], [3000, 2500])])
def test_write(d, H_kv, S, lens, new):
    c = Paged(lens, new, H_kv, d, S, gap=2)
    K, V, w = c.K.clone(), c.V.clone(), c.w.clone()
    fused = c.rand(c.R, 3 * H_kv + 1, d)  # rows of a wider projection
    k, v = fused[:, 1:H_kv + 1], fused[:, H_kv + 1:2 * H_kv + 1]
    for b in range(c.B):
        page, row = (x[lens[b]:] for x in c.at(b, lens[b] + new[b]))
        rows = slice(c.first[b], c.first[b + 1])
        K[page, :, row], V[page, :, row], w[page, :, row] = k[rows], v[rows], 0
    pisa.pisa_paged_write(k, v, c.K, c.V, c.table, c.len, row_start=c.rows, w=c.w)
    for got, want in ((c.K, K), (c.V, V)):
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    assert torch.equal(c.w, w)
    no_error()
    # contiguous rows, no weights
    c.w.fill_(3)
    c.K.fill_(1)
    pisa.pisa_paged_write(k.contiguous(), v.contiguous(), c.K, c.V, c.table, c.len, row_start=c.rows)
    for b in range(c.B):
        assert torch.equal(c.get(c.K, b, lens[b] + new[b])[lens[b]:], k[c.first[b]:c.first[b + 1]])
    assert (c.w == 3).all()


def test_write_bad():
    c = Paged([10, 20, 30, 5], [4, 4, 4, 4], 2, 64, 16, M=3)
    k = c.rand(c.R, 2, 64)
    c.table[0, 0] = -1      # entry 0 of sequence 0 names no page
    c.table[1, 1] = c.P     # entry 1 (rows 16 ..) of sequence 1 neither
    lens = i32(10, 20, 46, -1)  # sequence 2: 46 + 4 > 48
    want = c.K.clone()
    pisa.pisa_paged_write(k, k, c.K, c.V, c.table, lens, row_start=c.rows)
    assert torch.equal(c.K.view(torch.int16), want.view(torch.int16))
    assert pisa.pisa_get_last_device_error() == BAD_INDEX
    rows = i32(0, 4, 2, 40, 16)  # decreasing, and past the end
    pisa.pisa_paged_write(k, k, c.K, c.V, c.table, c.len, row_start=rows)
    assert pisa.pisa_get_last_device_error() == BAD_INDEX


# ---- attention ---------------------------------------------------------------------------------
def check_attn(c, G, causal=True, scale=0.0, uniform=False, gone=(), qscale=1.5):
    q = c.rand(c.R, c.H_kv * G, c.d, scale=qscale)
    o = torch.full_like(q, 5)
    lse = torch.full(q.shape[:2], 5.0, device=DEV)
    pisa.pisa_paged_attn(q, c.K, c.V, c.table, c.len, row_start=None if uniform else c.rows, causal=causal, scale=scale, o=o, lse=lse)
    wo, wl, bo, bl = H.attend(c, q, causal, scale if scale > 0 else None, gone)
    nobody = wl.isnan()
    assert (o[nobody] == 5).all() and (lse[nobody] == 5).all()
    R.close(o[~nobody], wo[~nobody], bo[~nobody], "o")
    R.close(lse[~nobody], wl[~nobody], bl[~nobody], "lse")
    return q, o, lse


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,H_kv", [(1, 2), (2, 1), (4, 2), (8, 1), (16, 1)])
@pytest.mark.parametrize("S", [16, 64, 256])
def test_attn_one_token(d, G, H_kv, S):
    c = Paged([0, 1, 15, 16, 127, 128, 129, 1000, 2047], [1] * 9, H_kv, d, S, seed=G + S)
    check_attn(c, G, uniform=True)
    no_error()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 4, 16])
@pytest.mark.parametrize("S", [16, 32, 128])
def test_attn_few_tokens(d, G, S):
    c = Paged([0, 300, 17, 1, 999, 126], [3, 0, 1, 5, 2, 4], 2, d, S, seed=S, gap=1)
    check_attn(c, G)
    check_attn(c, G, causal=False)
    no_error()


@pytest.mark.parametrize("d,G,S,lens,new", [
    (64, 1, 16, [0], [300]), (128, 1, 64, [0, 130], [257, 129]), (128, 4, 16, [0, 77, 500], [200, 1, 64]),
    (64, 8, 128, [1000, 0], [33, 95]), (128, 16, 64, [129], [40]), (128, 2, 512, [250, 0, 3], [128, 512, 0]),
    (64, 16, 32, [31, 2000], [16, 17])])
@pytest.mark.parametrize("causal", [True, False])
def test_attn_chunks(d, G, S, lens, new, causal):
    check_attn(Paged(lens, new, 2, d, S, seed=len(new), gap=3), G, causal)
    no_error()


def test_attn_many_sequences():
    """More sequences than a warp has lanes, empty ones among them."""
    lens = [(37 * i) % 400 for i in range(75)]
    new = [(i * 5) % 7 if i % 3 else 0 for i in range(75)]
    check_attn(Paged(lens, new, 1, 64, 16, seed=9), 4)
    new[40] = 150
    check_attn(Paged(lens, new, 1, 64, 16, seed=9), 4)
    no_error()


@pytest.mark.parametrize("d,G,H_kv,S,lens,new", [
    # tensor cores: 300 and more jobs over the SMs, sequences longer and shorter than the one before, several a block
    (64, 1, 16, 128, [0, 0, 0, 0], [1500, 600, 1100, 200]),
    (128, 2, 8, 16, [0, 900, 130, 0, 77, 1], [300, 40, 513, 900, 128, 700]),
    (64, 4, 8, 32, [(97 * i) % 500 for i in range(40)], [1 + (61 * i) % 150 for i in range(40)]),
    # few rows: thousands of jobs
    (64, 4, 8, 16, [(211 * i) % 700 for i in range(150)], [1 + i % 2 for i in range(150)]),
    (128, 16, 8, 64, [(433 * i) % 1500 for i in range(90)], [1] * 90)])
def test_many_jobs(d, G, H_kv, S, lens, new):
    """More jobs than blocks: every one of a block's jobs is found, with the next sequence's after a longer one's."""
    c = Paged(lens, new, H_kv, d, S, seed=H_kv + S)
    q = c.rand(c.R, H_kv * G, d, scale=1.5)
    o, lse = pisa.pisa_paged_attn(q, c.K, c.V, c.table, c.len, row_start=c.rows)
    wo, wl, bo, bl = H.attend_many(c, q)
    R.close(o, wo, bo, "o")
    R.close(lse, wl, bl, "lse")
    w = c.w.clone()
    pisa.pisa_paged_weights(q, lse, c.K, w, c.table, c.len, row_start=c.rows, accumulate=False)
    want, bound = H.weights(c, q, lse)
    live = ~want.isnan()
    assert (w[~live] == -7).all()
    R.close(w[live], want[live], bound[live], "w")
    no_error()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [5, 30, 40])
def test_attn_waits_for_memory(d, new):
    """Many keys for few rows: the softmax runs ahead of the tiles.  Checked by attending in two halves of the heads."""
    B, H_kv, G, S = 48, 4, 8, 16
    c = Paged([1500 + 37 * b for b in range(B)], [new] * B, H_kv, d, S, seed=new)
    q = c.rand(c.R, H_kv * G, d, scale=1.5)
    o, lse = pisa.pisa_paged_attn(q, c.K, c.V, c.table, c.len, row_start=c.rows)
    no_error()
    for h in range(H_kv):
        heads = slice(h * G, (h + 1) * G)
        o1, lse1 = pisa.pisa_paged_attn(q[:, heads].contiguous(), c.K[:, h:h + 1].contiguous(), c.V[:, h:h + 1].contiguous(),
                                        c.table, c.len, row_start=c.rows)
        # twice attend64's bounds, with sum w |v| <= max |v| < 6 and |q| . |k| <= |q| |k| < 3 sqrt(d) 2 sqrt(d)
        e = (d + 8) * R.F * 6 * math.sqrt(d)
        assert (o[:, heads].float() - o1.float()).abs().max() <= 2 * ((R.U + 4 * e + 2.0 ** -16) * 6 + R.U * 6)
        assert (lse[:, heads] - lse1).abs().max() <= 2 * (2 * e + 2.0 ** -18 + 2.0 ** -22 * 16)
    no_error()


def test_attn_strided_rows_and_scale():
    c = Paged([100, 40], [3, 70], 2, 128, 32)
    fused = c.rand(c.R, 12, 128)
    q = fused[:, :8]
    for scale in (0.0, 0.3):
        o, lse = pisa.pisa_paged_attn(q, c.K, c.V, c.table, c.len, row_start=c.rows, scale=scale)
        o2, lse2 = pisa.pisa_paged_attn(q.contiguous(), c.K, c.V, c.table, c.len, row_start=c.rows, scale=scale)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        check_attn(c, 4, scale=scale)
    no_error()


@pytest.mark.parametrize("new", [[1, 1, 1], [2, 1, 40], [300, 5, 1]])
def test_attn_absent_pages(new):
    """Negative entries stand for pages that are gone: a sequence may lose its first pages, one in the middle or all."""
    c = Paged([200, 500, 30], new, 2, 128, 16, M=48)
    gone = {(0, 0), (0, 5), (1, 7), (1, 8), (1, 30)} | {(2, i) for i in range(48)}
    table = c.table.clone()
    for b, i in gone:
        table[b, i] = -1 - i
    q = c.rand(c.R, 8, 128)
    o, lse = pisa.pisa_paged_attn(q, c.K, c.V, table, c.len, row_start=c.rows)
    wo, wl, bo, bl = H.attend(c, q, gone=gone)
    R.close(o, wo, bo, "o")
    R.close(lse, wl, bl, "lse")
    no_error()
    assert (lse[c.first[2]:] == -math.inf).all() and (o[c.first[2]:] == 0).all()
    w = c.w.clone()
    pisa.pisa_paged_weights(q, lse, c.K, w, table, c.len, row_start=c.rows, accumulate=False)
    want, bound = H.weights(c, q, lse, gone=gone)
    live = ~want.isnan()
    assert (w[~live] == -7).all()
    R.close(w[live], want[live], bound[live], "w")
    no_error()
    table[1, 30] = c.P  # one that never was: the same, and flagged
    o2, lse2 = pisa.pisa_paged_attn(q, c.K, c.V, table, c.len, row_start=c.rows)
    assert pisa.pisa_get_last_device_error() == BAD_INDEX
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("big", [False, True])
def test_attn_bad_lengths(big):
    n = 90 if big else 2
    c = Paged([10, 20, 30], [n, n, n], 2, 64, 16, M=8)
    q = c.rand(c.R, 8, 64)
    o, lse = torch.full_like(q, 5), torch.full((c.R, 8), 5.0, device=DEV)
    lens = i32(10, 8 * 16 - n + 1, -3)
    pisa.pisa_paged_attn(q, c.K, c.V, c.table, lens, row_start=c.rows, o=o, lse=lse)
    assert pisa.pisa_get_last_device_error() == BAD_INDEX
    assert (o[n:] == 5).all() and (lse[n:] == 5).all()
    wo, wl, bo, bl = H.attend(c, q)
    R.close(o[:n], wo[:n], bo[:n], "o")
    w = c.w.clone()
    pisa.pisa_paged_weights(q, wl.float(), c.K, w, c.table, lens, row_start=c.rows)
    assert pisa.pisa_get_last_device_error() == BAD_INDEX
    for b in (1, 2):
        page, row = c.at(b, c.lens[b] + n)
        assert (w[page, :, row] == -7).all()
    # row bounds out of range are brought into range and flagged
    pisa.pisa_paged_attn(q, c.K, c.V, c.table, c.len, row_start=i32(-1, n, n // 2, c.R + 9))
    assert pisa.pisa_get_last_device_error() == BAD_INDEX


@pytest.mark.parametrize("new", [1, 2, 100])
def test_attn_extreme_values(new):
    """Logits far apart, of +- thousands, and rows whose keys are all alike."""
    c = Paged([260], [new], 1, 128, 64)
    k = c.get(c.K, 0, 260 + new)
    for f in (0.0, 100.0):
        c.put(0, (k.float() * f).to(torch.bfloat16), c.get(c.V, 0, 260 + new))
        check_attn(c, 4, qscale=3.0)
    no_error()


def test_attn_nan_shows():
    c = Paged([100], [1], 1, 64, 16)
    c.put(0, c.rand(101, 1, 64), c.rand(101, 1, 64))
    k = c.get(c.K, 0, 101)
    k[7, 0, 3] = math.nan
    c.put(0, k, c.get(c.V, 0, 101))
    q = c.rand(1, 4, 64)
    o, lse = pisa.pisa_paged_attn(q, c.K, c.V, c.table, c.len)
    assert o.isnan().all() and lse.isnan().all()


@pytest.mark.parametrize("new", [[1, 1, 1], [200, 3, 90]])
def test_one_page_a_sequence(new):
    """A cache [B][H_kv][N_cap][d] of the other entry points, as pages; and the same keys in small pages."""
    lens, S = [2000, 77, 500], 4096
    c = Paged(lens, new, 2, 128, S, M=1, spare=0)
    q = c.rand(c.R, 8, 128, scale=1.5)
    o, lse = pisa.pisa_paged_attn(q, c.K, c.V, c.table, c.len, row_start=c.rows)
    wo, wl, bo, bl = H.attend_many(c, q)
    R.close(o, wo, bo, "o")
    R.close(lse, wl, bl, "lse")
    w = c.w.clone()
    pisa.pisa_paged_weights(q, lse, c.K, w, c.table, c.len, row_start=c.rows, accumulate=False)
    small = Paged(lens, new, 2, 128, 16, seed=5)
    for b in range(3):
        n = lens[b] + new[b]
        small.put(b, c.get(c.K, b, n), c.get(c.V, b, n))
    o2, lse2 = pisa.pisa_paged_attn(q, small.K, small.V, small.table, c.len, row_start=c.rows)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    w2 = small.w.clone()
    pisa.pisa_paged_weights(q, lse, small.K, w2, small.table, c.len, row_start=c.rows, accumulate=False)
    for b in range(3):
        assert torch.equal(c.get(w, b, lens[b] + new[b]), small.get(w2, b, lens[b] + new[b]))
    no_error()


def test_a_thousand_sequences():
    lens, new = [(7 * i) % 40 for i in range(1100)], [1 if i % 5 else 0 for i in range(1100)]
    c = Paged(lens, new, 2, 64, 16, seed=1)
    q = c.rand(c.R, 4, 64, scale=1.5)
    o, lse = pisa.pisa_paged_attn(q, c.K, c.V, c.table, c.len, row_start=c.rows)
    wo, wl, bo, bl = H.attend_many(c, q)
    R.close(o, wo, bo, "o")
    R.close(lse, wl, bl, "lse")
    w = c.w.clone()
    pisa.pisa_paged_weights(q, lse, c.K, w, c.table, c.len, row_start=c.rows, accumulate=False)
    want, bound = H.weights(c, q, lse)
    live = ~want.isnan()
    R.close(w[live], want[live], bound[live], "w")
    no_error()


def test_two_streams():
    """Calls of two sets of sequences at once, on streams other than the current one, each with its own scratch."""
    cases = [Paged([3000, 5], [300, 1], 4, 128, 16, seed=1), Paged([100 * i for i in range(30)], [1] * 30, 4, 128, 64, seed=2)]
    qs = [c.rand(c.R, 16, 128, scale=1.5) for c in cases]
    want = [pisa.pisa_paged_attn(q, c.K, c.V, c.table, c.len, row_start=c.rows) for c, q in zip(cases, qs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(20):
        for i, (c, q) in enumerate(zip(cases, qs)):
            with torch.cuda.stream(streams[i]):
                got[i].append(pisa.pisa_paged_attn(q, c.K, c.V, c.table, c.len, row_start=c.rows))
    torch.cuda.synchronize()
    for g, (o, lse) in zip(got, want):
        assert all(torch.equal(x, o) and torch.equal(y, lse) for x, y in g)
    no_error()


@pytest.mark.parametrize("T,G", [(1, 4), (70, 4)])
def test_far_pages(T, G):
    """Pages behind 2^31 elements of the pool: offsets of keys, values and weights in 64 bits."""
    H_kv, d, S, n = 8, 128, 64, 700
    P = (1 << 31) // (H_kv * S * d) + 2 * (n // S + 1) + 8
    K = torch.empty((P, H_kv, S, d), dtype=torch.bfloat16, device=DEV)
    V, w = torch.empty_like(K), torch.zeros((P, H_kv, S), device=DEV)
    m = -(-n // S)
    c = Paged([n - T], [T], H_kv, d, S, seed=3)
    table = torch.arange(P - m, P, device=DEV, dtype=torch.int32).flip(0)[None].contiguous()
    g = lambda x: c.get(x, 0, n)  # noqa: E731
    pisa.pisa_paged_write(g(c.K), g(c.V), K, V, table, i32(0), w=w)
    q = c.rand(T, H_kv * G, d, scale=1.5)
    o, lse = pisa.pisa_paged_attn(q, K, V, table, c.len)
    wo, wl, bo, bl = H.attend(c, q)
    R.close(o, wo, bo, "o")
    R.close(lse, wl, bl, "lse")
    pisa.pisa_paged_weights(q, lse, K, w, table, c.len)
    want, bound = H.weights(c, q, lse)
    at = torch.arange(n, device=DEV)
    got = w[table[0, at // S].long(), :, at % S]
    R.close(got, g(want), g(bound), "w")
    new = torch.arange(3, device=DEV, dtype=torch.int32)[None] + (P - m - 3)
    new_len, kept = pisa.pisa_paged_evict(K, V, w, table, i32(n), new, 150)
    j = torch.arange(150, device=DEV)
    for h in range(H_kv):
        assert torch.equal(K[new[0, j // S].long(), h, j % S], g(c.K)[kept[0, h].long(), h])
    assert new_len.tolist() == [150]
    no_error()


# ---- weights -----------------------------------------------------------------------------------
def check_weights(c, G, causal=True, accumulate=False, scale=0.0):
    q = c.rand(c.R, c.H_kv * G, c.d, scale=1.5)
    lse = torch.full((c.R, c.H_kv * G), math.nan, device=DEV)
    pisa.pisa_paged_attn(q, c.K, c.V, c.table, c.len, row_start=c.rows, causal=causal, scale=scale, lse=lse)
    w = c.w.clone()
    pisa.pisa_paged_weights(q, lse, c.K, w, c.table, c.len, row_start=c.rows, causal=causal, scale=scale, accumulate=accumulate)
    want, bound = H.weights(c, q, lse, causal, scale if scale > 0 else None)
    live = ~want.isnan()
    assert (w[~live] == -7).all()
    if accumulate:  # one more sum, of numbers up to 7 + want
        want, bound = want - 7, bound + 2.0 ** -24 * (want + 7)
    R.close(w[live], want[live], bound[live], "w")
    if not accumulate:  # every row and head gave 1 in all
        assert abs(float(w[live].double().sum()) - sum(c.new) * G * c.H_kv) <= float(bound[live].sum()) + 1e-5 * sum(c.new) * G * c.H_kv
    no_error()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,S,lens,new", [
    (1, 16, [0], [1]), (4, 64, [0, 1000, 63, 64], [1, 1, 1, 1]), (16, 32, [300, 0, 127], [3, 0, 1]), (8, 16, [129, 5], [33, 70]),
    (2, 128, [0, 250], [257, 129]), (1, 256, [500], [300])])
@pytest.mark.parametrize("accumulate", [False, True])
def test_weights(d, G, S, lens, new, accumulate):
    check_weights(Paged(lens, new, 2, d, S, seed=S, gap=1), G, accumulate=accumulate)
    check_weights(Paged(lens, new, 2, d, S, seed=S + 1), G, causal=False, accumulate=accumulate, scale=0.2)


def test_weights_without_rows():
    c = Paged([100, 0, 17], [0, 0, 0], 2, 64, 16)
    q, lse = c.rand(0, 4, 64), torch.zeros(0, 4, device=DEV)
    before = c.w.clone()
    pisa.pisa_paged_weights(q, lse, c.K, c.w, c.table, c.len)
    assert torch.equal(c.w, before)
    pisa.pisa_paged_weights(q, lse, c.K, c.w, c.table, c.len, accumulate=False)
    for b, n in enumerate(c.lens):
        page, row = c.at(b, n)
        assert (c.w[page, :, row] == 0).all()
        before[page, :, row] = 0
    assert torch.equal(c.w, before)


# ---- eviction ----------------------------------------------------------------------------------
def check_evict(c, keep, sinks, recent, n=None, gone=(), table=None):
    n = c.lens if n is None else n
    S = c.S
    M_new = -(-keep // S) + 1
    new_table = torch.full((c.B, M_new), -1, dtype=torch.int32, device=DEV)
    need, at = [-(-min(x, keep) // S) for x in n], 0
    for b, x in enumerate(need):
        new_table[b, :x] = c.spare[at:at + x]
        at += x
    assert at <= len(c.spare)
    K, V, w = c.K.clone(), c.V.clone(), c.w.clone()
    want = H.evict(c, w, n, keep, sinks, recent, gone)
    new_len, kept = pisa.pisa_paged_evict(c.K, c.V, c.w, c.table if table is None else table, i32(*n), new_table, keep,
                                          sinks=sinks, recent=recent)
    for b in range(c.B):
        for h in range(c.H_kv):
            idx = want[b * c.H_kv + h]
            assert kept[b, h].tolist() == idx + [-1] * (keep - len(idx)), (b, h)
            src = torch.tensor(idx, device=DEV, dtype=torch.long)
            j = torch.arange(len(idx), device=DEV)
            to, page = new_table[b, j // S].long(), c.table[b, src // S].long()
            for x, y in ((c.K, K), (c.V, V), (c.w, w)):
                y[to, h, j % S] = y[page, h, src % S]
        assert int(new_len[b]) == len(want[b * c.H_kv])
    for x, y in ((c.K, K), (c.V, V)):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))
    assert torch.equal(c.w.view(torch.int32), w.view(torch.int32))
    # the list in scratch memory instead
    c2 = pisa.pisa_paged_evict(c.K, c.V, c.w, c.table if table is None else table, i32(*n), new_table, keep, sinks=sinks,
                               recent=recent, want_kept=False)
    assert c2[1] is None and torch.equal(c2[0], new_len) and torch.equal(c.K.view(torch.int16), K.view(torch.int16))
    no_error()


@pytest.mark.parametrize("d,H_kv,S,lens,keep,sinks,recent", [
    (64, 1, 16, [1], 1, 0, 0), (64, 2, 16, [100, 0, 17, 64], 32, 4, 8), (128, 3, 64, [1000, 999, 130], 129, 0, 0),
    (128, 2, 32, [500, 600], 100, 40, 60), (64, 1, 16, [50], 1, 0, 1), (64, 2, 16, [4097, 5000, 9000], 700, 4, 64),
    (64, 1, 256, [40000, 5], 4096, 1, 100), (128, 1, 128, [130000], 1000, 4, 32), (64, 1, 16, [300], 299, 0, 0),
    (64, 2, 16, [9000, 300], 8999, 0, 0)])
@pytest.mark.parametrize("kind", ["spread", "ties", "odd"])
def test_evict(d, H_kv, S, lens, keep, sinks, recent, kind):
    spare = sum(-(-min(n, keep) // S) for n in lens) + 2
    c = Paged(lens, [0] * len(lens), H_kv, d, S, seed=keep, spare=spare)
    w = torch.randn(c.w.shape, generator=c.g, device=DEV).exp()
    if kind == "ties":
        w = (w * 2).floor()
    if kind == "odd":  # NaN, infinities, zeros of both signs, negative and tiny numbers
        odd = torch.tensor([math.nan, math.inf, -math.inf, 0.0, -0.0, -1.0, 1e-42, -1e-42, 3.0], device=DEV)
        w = odd[torch.randint(0, 9, w.shape, generator=c.g, device=DEV)]
    c.w.copy_(w)
    check_evict(c, keep, sinks, recent)


@pytest.mark.parametrize("n", [600, 6000])
def test_evict_absent_pages(n):
    c = Paged([n, n // 2], [0, 0], 2, 64, 16, spare=40)
    c.w.copy_(torch.rand(c.w.shape, generator=c.g, device=DEV))
    gone = {(0, 0), (0, 3), (0, (n - 1) // 16), (1, 2)}
    table = c.table.clone()
    for b, i in gone:
        table[b, i] = -1
    check_evict(c, 200, 20, 30, gone=gone, table=table)
    gone |= {(1, i) for i in range(n // 32 + 1) if i > 4}
    for b, i in gone:
        table[b, i] = -1
    check_evict(c, 200, 20, 30, gone=gone, table=table)  # fewer keys than wanted


def test_evict_bad():
    c = Paged([100, 100, 100], [0, 0, 0], 1, 64, 16, spare=12)
    c.w.fill_(1)
    new_table = c.spare[:12].reshape(3, 4).contiguous()
    new_table[1, 1] = c.P
    lens = i32(100, 100, c.M * 16 + 1)
    K, new_len = c.K.clone(), i32(7, 7, 7)
    _, kept = pisa.pisa_paged_evict(c.K, c.V, c.w, c.table, lens, new_table, 50, new_len=new_len)
    assert pisa.pisa_get_last_device_error() == BAD_INDEX
    assert new_len.tolist() == [50, 50, 7]
    assert (kept[2] == -1).all() and kept[1, 0].tolist() == list(range(50))
    for b, pages in ((0, range(4)), (1, (0, 2, 3))):
        for j in range(50):
            if j // 16 in pages:
                K[new_table[b, j // 16].long(), 0, j % 16] = K[c.table[b, j // 16].long(), 0, j % 16]
    assert torch.equal(c.K.view(torch.int16), K.view(torch.int16))


# ---- together ----------------------------------------------------------------------------------
@pytest.mark.parametrize("d,G,S", [(64, 4, 16), (128, 8, 64)])
def test_run(d, G, S):
    """Prompts, drafts, an eviction between decode steps: each step against the 64-bit form of what the cache held."""
    B, H_kv = 3, 2
    c = Paged([0] * B, [300, 40, 129], H_kv, d, S, spare=200, M=64)
    # room to grow: every sequence gets pages of its own up to 512 keys
    pool = c.spare
    need = [-(-x // S) for x in c.new]
    full = 512 // S
    for b in range(B):
        more = full - need[b]
        c.table[b, need[b]:full] = pool[:more]
        pool = pool[more:]
    c.w.fill_(0)
    total = [0] * B
    for step, new in enumerate(([300, 40, 129], [1, 1, 1], [2, 0, 5], [1, 1, 1])):
        if step == 2:  # down to 100 keys a head
            keep = 100
            new_table = torch.full_like(c.table, -1)
            for b in range(B):
                n = -(-min(total[b], keep) // S)
                new_table[b, :n] = pool[:n]
                pool = pool[n:]
                n0 = -(-keep // S)
                new_table[b, n:n0 + 2] = pool[:n0 + 2 - n]
                pool = pool[n0 + 2 - n:]
            new_len, kept = pisa.pisa_paged_evict(c.K, c.V, c.w, c.table, i32(*total), new_table, keep, sinks=4, recent=16)
            want = H.evict(c, c.w, total, keep, 4, 16)
            assert [x[x >= 0].tolist() for x in kept.reshape(-1, keep)] == want
            total = new_len.tolist()
            assert total == [min(keep, x) for x in [301, 41, 130]]
            c.table = new_table
        c.lens, c.new = list(total), list(new)
        c.first = [sum(new[:i]) for i in range(B + 1)]
        c.R, c.rows, c.len = c.first[-1], i32(*c.first), i32(*total)
        k, v, q = c.rand(c.R, H_kv, d), c.rand(c.R, H_kv, d), c.rand(c.R, H_kv * G, d, scale=1.5)
        pisa.pisa_paged_write(k, v, c.K, c.V, c.table, c.len, row_start=c.rows, w=c.w)
        for b in range(B):
            assert torch.equal(c.get(c.K, b, total[b] + new[b])[total[b]:], k[c.first[b]:c.first[b + 1]])
        o, lse = pisa.pisa_paged_attn(q, c.K, c.V, c.table, c.len, row_start=c.rows)
        wo, wl, bo, bl = H.attend(c, q)
        R.close(o, wo, bo, "o")
        R.close(lse, wl, bl, "lse")
        before = c.w.clone()
        pisa.pisa_paged_weights(q, lse, c.K, c.w, c.table, c.len, row_start=c.rows)
        want, bound = H.weights(c, q, lse)
        live = ~want.isnan()
        want = want + before.double()
        R.close(c.w[live], want[live], (bound + 2.0 ** -24 * want.abs())[live], "w")
        total = [a + b for a, b in zip(total, new)]
    no_error()


def test_same_every_time_and_in_graphs():
    c = Paged([500, 3, 100, 1000], [60, 1, 0, 2], 2, 128, 16, spare=60)
    q = c.rand(c.R, 16, 128)
    new_table = c.spare[:40].reshape(4, 10).contiguous()
    w = torch.zeros_like(c.w)
    o, lse = pisa.pisa_paged_attn(q, c.K, c.V, c.table, c.len, row_start=c.rows)
    pisa.pisa_paged_weights(q, lse, c.K, w, c.table, c.len, row_start=c.rows)
    first = [x.clone() for x in (o, lse, w)]
    shape, params = pisa.make_shape(4, c.R, 16, 2, 128), pisa.make_params(1)
    need = pisa.pisa_paged_attn_workspace_bytes(shape, params, pisa.pisa_pages(c.P, 16, c.M))
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    kept = torch.empty((4, 2, 150), dtype=torch.int32, device=DEV)
    new_len = i32(0, 0, 0, 0)
    n = i32(560, 4, 100, 1002)

    def calls():
        w.zero_()
        pisa.pisa_paged_attn(q, c.K, c.V, c.table, c.len, row_start=c.rows, o=o, lse=lse, ws=ws)
        pisa.pisa_paged_weights(q, lse, c.K, w, c.table, c.len, row_start=c.rows)
        pisa.pisa_paged_evict(c.K, c.V, w, c.table, n, new_table, 150, recent=8, new_len=new_len, kept=kept)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    k1 = kept.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for _ in range(3):
        for x in (o, lse, w, kept):
            x.fill_(9)
        ws.fill_(255)
        graph.replay()
        # (the eviction puts kept keys' weights beside the new pages)
        live = torch.ones(c.P, dtype=torch.bool, device=DEV)
        live[new_table.long()] = False
        for x, y in zip((o, lse, w[live]), (first[0], first[1], first[2][live])):
            assert torch.equal(x, y)
        assert torch.equal(kept, k1)
    no_error()
