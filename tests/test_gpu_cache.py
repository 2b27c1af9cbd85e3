"""The 8-bit cache on the GPU: rows quantised as they are written, rows read back, and the attention
of new tokens over selected blocks of it, against plain forms in 64 bits."""
import math

import pytest
import torch

import cache_helpers as R
import hierarchical_top_block_gb300 as pisa

pytestmark = pytest.mark.gpu
DEV = "cuda"


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(torch.bfloat16)


def empty_cache(B, H, N, d, fill=77):
    q = [torch.full((B, H, N, d), fill, dtype=torch.int8, device=DEV) for _ in range(2)]
    s = [torch.full((B, H, N), 0.5, device=DEV) for _ in range(2)]
    return q[0], q[1], s[0], s[1]


def filled_cache(g, B, H, N, d):
    K, V = normal(g, B, H, N, d), normal(g, B, H, N, d)
    kc, ks, _ = R.quantise64(K)
    vc, vs, _ = R.quantise64(V)
    return kc, vc, ks, vs


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def no_error():
    assert pisa.pisa_get_last_device_error() == 0


# ---- write -------------------------------------------------------------------------------
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,T,N", [(1, 1, 1, 1), (3, 2, 1, 65), (2, 3, 17, 40), (1, 8, 1000, 1003), (5, 1, 129, 700), (3, 5, 4001, 4100)])
@pytest.mark.parametrize("ragged", [False, True])
def test_write(d, B, H, T, N, ragged):
    g = gen(T * 7 + d)
    k, v = normal(g, B, H, T, d), normal(g, B, H, T, d, scale=30)
    n = torch.randint(0, T + 1, (B,), generator=g, device=DEV).int() if ragged else torch.full((B,), T, device=DEV).int()
    ln = (torch.rand(B, generator=g, device=DEV) * (N - n + 1)).int().clamp(max=N - n).int()
    Kq, Vq, ks, vs = empty_cache(B, H, N, d)
    want = [x.clone() for x in (Kq, Vq, ks, vs)]
    ko, vo = torch.full_like(k, 3), torch.full_like(v, 3)
    wo = [ko.clone(), vo.clone()]
    for i, x in enumerate((k, v)):
        c, s, val = R.quantise64(x)
        for b in range(B):
            nb, lb = int(n[b]), int(ln[b])
            want[i][b, :, lb:lb + nb], want[2 + i][b, :, lb:lb + nb] = c[b, :, :nb], s[b, :, :nb]
            wo[i][b, :, :nb] = val[b, :, :nb]
    before = ln.clone()
    pisa.pisa_cache_write(k, v, Kq, Vq, ks, vs, ln, new_len=n if ragged else None, k_out=ko, v_out=vo)
    for got, w in zip((Kq, Vq, ks, vs, ko, vo, ln), want + wo + [before]):
        assert torch.equal(got, w)
    # without the values out, the same cache; with one side's, the other is not written
    K2, V2, k2, v2 = empty_cache(B, H, N, d)
    pisa.pisa_cache_write(k, v, K2, V2, k2, v2, ln, new_len=n if ragged else None)
    K3, V3, k3, v3 = empty_cache(B, H, N, d)
    v3o = torch.full_like(v, 3)
    pisa.pisa_cache_write(k, v, K3, V3, k3, v3, ln, new_len=n if ragged else None, v_out=v3o)
    for got, w in zip((K2, V2, k2, v2, K3, V3, k3, v3, v3o), want + want + [wo[1]]):
        assert torch.equal(got, w)
    no_error()


@pytest.mark.parametrize("d", [64, 128])
def test_write_hard_rows(d):
    """Zeros, subnormals, the largest and smallest values, halves between codes, infinities and NaN."""
    rows = [torch.zeros(d), -torch.zeros(d)]
    tiny = torch.zeros(d)
    tiny[3], tiny[5] = 2.0 ** -133, -2.0 ** -133
    rows.append(tiny)
    rows.append(torch.linspace(-1, 1, d) * 2.0 ** -126)
    rows.append(torch.linspace(-1, 1, d) * 3.38e38)
    # |x| = (k + 1/2) / 127 of the maximum, exactly: a = 127, x = k + 1/2 (k < 127: at most 8 bits)
    half = torch.arange(d).float() * (2 if d == 64 else 1) % 127 + 0.5
    half[0] = 127
    half[1::2] *= -1
    rows += [half, half * 2.0 ** -130, half * 2.0 ** 100]
    one = torch.full((d,), 1e-30)
    one[d - 1] = -5.0
    rows.append(one)
    for bad in (math.inf, -math.inf, math.nan):
        x = torch.linspace(-2, 2, d)
        x[7] = bad
        rows.append(x)
    g = torch.Generator().manual_seed(1)
    rows += [torch.randn(d, generator=g) * 2.0 ** e for e in range(-130, 120, 10)]
    x = torch.stack(rows).to(torch.bfloat16).to(DEV)[None, None]
    n = x.shape[2]
    Kq, Vq, ks, vs = empty_cache(1, 1, n, d)
    ko, vo = torch.empty_like(x), torch.empty_like(x)
    pisa.pisa_cache_write(x, -x, Kq, Vq, ks, vs, i32(0), k_out=ko, v_out=vo)
    for y, q, s, o in ((x, Kq, ks, ko), (-x, Vq, vs, vo)):
        c, sc, val = R.quantise64(y)
        assert torch.equal(q, c)
        assert torch.equal(s.nan_to_num(-1), sc.nan_to_num(-1)) and torch.equal(s.isnan(), sc.isnan())
        assert torch.equal(o.float().nan_to_num(-1), val.float().nan_to_num(-1))
    no_error()


def test_write_every_quotient():
    """Every pair of significands, at differences of the exponents where a code can change."""
    d = 128
    X = torch.arange(128, 256, device=DEV).float()
    rows = []
    for M in range(128, 256):
        for e in range(0, 10):
            r = X * 2.0 ** -e
            r = torch.where(r > M, r / 2, r)
            r[0] = M
            rows.append(r)
    x = torch.stack(rows).to(torch.bfloat16)
    assert torch.equal(x.float(), torch.stack(rows))
    x = x.reshape(1, 1, -1, d)
    Kq, Vq, ks, vs = empty_cache(1, 1, x.shape[2], d)
    pisa.pisa_cache_write(x, (x.float() * 2.0 ** -90).to(torch.bfloat16), Kq, Vq, ks, vs, i32(0))
    c, s, _ = R.quantise64(x)
    assert torch.equal(Kq, c) and torch.equal(Vq, c) and torch.equal(ks, s)


def test_write_one_token_in_place():
    B, H, N, d = 6, 4, 30, 128
    g = gen(3)
    k, v = normal(g, B, H, d), normal(g, B, H, d)
    Kq, Vq, ks, vs = empty_cache(B, H, N, d)
    ln = torch.arange(B, device=DEV).int() * 5
    want = [R.quantise64(k), R.quantise64(v)]
    pisa.pisa_cache_write(k, v, Kq, Vq, ks, vs, ln, k_out=k, v_out=v)
    at = (torch.arange(B, device=DEV)[:, None], torch.arange(H, device=DEV)[None], ln.long()[:, None])
    for (c, s, val), q, sc, o in zip(want, (Kq, Vq), (ks, vs), (k, v)):
        assert torch.equal(q[at], c) and torch.equal(sc[at], s) and torch.equal(o, val)


@pytest.mark.parametrize("ln,n", [((-1, 0), (2, 2)), ((0, 9), (2, 2)), ((0, 0), (2, -1)), ((0, 3), (2, 5)), ((2 ** 31 - 1, 0), (2, 2))])
def test_write_lengths_that_do_not_fit(ln, n):
    B, H, T, N, d = 2, 2, 4, 10, 64
    g = gen(1)
    k, v = normal(g, B, H, T, d), normal(g, B, H, T, d)
    Kq, Vq, ks, vs = empty_cache(B, H, N, d)
    pisa.pisa_cache_write(k, v, Kq, Vq, ks, vs, i32(*ln), new_len=i32(*n))
    assert pisa.pisa_get_last_device_error() == 5
    c, s, _ = R.quantise64(k)
    for b in range(B):
        ok = 0 <= n[b] <= T and 0 <= ln[b] <= N - n[b]
        want = torch.full((H, N, d), 77, dtype=torch.int8, device=DEV)
        if ok:
            want[:, ln[b]:ln[b] + n[b]] = c[b, :, :n[b]]
        assert torch.equal(Kq[b], want)
    no_error()


# ---- read --------------------------------------------------------------------------------
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,T,N", [(1, 1, 1, 1), (2, 3, 7, 100), (3, 2, 333, 500), (4, 8, 64, 64), (3, 5, 4001, 4100)])
@pytest.mark.parametrize("ragged", [False, True])
def test_read(d, B, H, T, N, ragged):
    g = gen(T + d)
    Kq, Vq, ks, vs = filled_cache(g, B, H, N, d)
    n = torch.randint(0, T + 1, (B,), generator=g, device=DEV).int() if ragged else torch.full((B,), T, device=DEV).int()
    st = (torch.rand(B, generator=g, device=DEV) * (N - n + 1)).int().clamp(max=N - n).int() if ragged else n * 0
    ko = torch.full((B, H, T, d), 5.0, dtype=torch.bfloat16, device=DEV)
    vo = ko.clone()
    pisa.pisa_cache_read(Kq, Vq, ks, vs, T, start=st if ragged else None, length=n if ragged else None, k_out=ko, v_out=vo)
    only_k, none = pisa.pisa_cache_read(Kq, None, ks, None, T, start=st, length=n)
    assert none is None
    none, only_v = pisa.pisa_cache_read(None, Vq, None, vs, T, start=st, length=n)
    assert none is None
    for q, s, o, only in ((Kq, ks, ko, only_k), (Vq, vs, vo, only_v)):
        val = (q.float() * s[..., None]).to(torch.bfloat16)
        for b in range(B):
            nb, sb = int(n[b]), int(st[b])
            assert torch.equal(o[b, :, :nb], val[b, :, sb:sb + nb]) and (o[b, :, nb:] == 5).all()
            assert torch.equal(only[b, :, :nb], val[b, :, sb:sb + nb]) and (only[b, :, nb:] == 0).all()
    no_error()


def test_read_ranges_that_do_not_fit():
    g = gen(2)
    Kq, Vq, ks, vs = filled_cache(g, 4, 1, 20, 64)
    out, _ = pisa.pisa_cache_read(Kq, None, ks, None, 6, start=i32(-1, 15, 0, 3), length=i32(4, 6, 7, 6))
    assert pisa.pisa_get_last_device_error() == 5
    assert (out[:3] == 0).all() and (out[3] != 0).any()


# ---- attention over selected blocks ------------------------------------------------------------
def sparse64(q, Kq, Vq, ks, vs, idx, ln, n, scale=None):
    """Plain form over [B, T, H_q, d]; rows not in use: zeros."""
    B, T, H_q, d = q.shape
    H, N = Kq.shape[1:3]
    G = H_q // H
    o = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros((B, T, H_q), dtype=torch.float64, device=DEV)
    to, tl = torch.zeros_like(o), torch.zeros_like(lse)
    for b in range(B):
        for t in range(int(n[b])):
            for h in range(H):
                blocks = [int(x) for x in idx[b, h, t].tolist() if 0 <= x < -(-N // 64)]
                keys = [c for j in blocks for c in range(64 * j, 64 * j + 64) if c <= int(ln[b]) + t]
                at = torch.tensor(keys, dtype=torch.long, device=DEV)
                k = Kq[b, h, at].double() * ks[b, h, at].double()[:, None]
                v = Vq[b, h, at].double() * vs[b, h, at].double()[:, None]
                s = slice(h * G, h * G + G)
                o[b, t, s], lse[b, t, s], to[b, t, s], tl[b, t, s] = R.attend64(
                    q[b, t, s].double(), k, v, scale, vs[b, h, at].double())
    return o, lse, to, tl


def lists(g, B, H, T, K, N, ln):
    """Own block and random earlier ones, ascending, -1 behind; some lists short."""
    idx = torch.full((B, H, T, K), -1, dtype=torch.int32)
    r = torch.rand((B, H, T, -(-N // 64)), generator=g, device=DEV).cpu()
    for b in range(B):
        for t in range(T):
            own = min(int(ln[b]) + t, N - 1) // 64
            for h in range(H):
                others = sorted(range(own), key=lambda j: r[b, h, t, j])[: max(0, K - 1 - (b + t) % 3)]
                sel = sorted(others + [own])
                idx[b, h, t, : len(sel)] = torch.tensor(sel)
    return idx.to(DEV)


@pytest.mark.parametrize("B,T,H_q,H,d,K,N", [
    (1, 1, 1, 1, 64, 1, 1), (1, 1, 16, 1, 128, 16, 4096), (2, 1, 4, 4, 64, 4, 333), (3, 1, 32, 8, 128, 16, 2000),
    (1, 5, 16, 1, 64, 32, 3001), (2, 3, 8, 1, 128, 8, 700), (40, 2, 16, 8, 128, 8, 130), (2, 8, 32, 2, 128, 32, 2500),
    (1, 1, 2, 1, 128, 32, 5000), (300, 1, 2, 1, 64, 3, 200),
    (60, 2, 32, 2, 128, 9, 1500), (90, 1, 32, 2, 64, 17, 1999)])
@pytest.mark.parametrize("ragged", [False, True])
def test_sparse(B, T, H_q, H, d, K, N, ragged):
    g = gen(B + 10 * T + K)
    Kq, Vq, ks, vs = filled_cache(g, B, H, N, d)
    q = normal(g, B, T, H_q, d, scale=1.5)
    n = torch.full((B,), T, device=DEV).int()
    ln = torch.full((B,), N - T, device=DEV).int()
    if ragged:
        n = torch.randint(0, T + 1, (B,), generator=g, device=DEV).int()
        ln = torch.randint(0, N - T + 1, (B,), generator=g, device=DEV).int()
    idx = lists(g, B, H, T, K, N, ln)
    # what lies behind a sequence's tokens is nobody's business
    for b in range(B):
        ks[b, :, int(ln[b]) + T:] = math.nan
        vs[b, :, int(ln[b]) + T:] = math.inf
    O = torch.full(q.shape, 9.0, dtype=torch.bfloat16, device=DEV)
    L = torch.full((B, T, H_q), 9.0, device=DEV)
    got, lse = pisa.pisa_sparse_attn_cache(q, Kq, Vq, ks, vs, idx, ln, new_len=n if ragged else None, O=O, LSE=L)
    assert got is O and lse is L
    o, l, to, tl = sparse64(q, Kq, Vq, ks, vs, idx, ln, n)
    use = torch.arange(T, device=DEV)[None] < n[:, None]
    assert (O[~use] == 9).all() and (L[~use] == 9).all()
    R.close(O[use], o[use], to[use], "O")
    R.close(L[use], l[use], tl[use], "LSE")
    no_error()


def test_sparse_lists_and_masks():
    """Lists that name nothing, blocks not begun yet, a block twice, numbers past the cache."""
    B, T, H_q, H, d, K, N = 1, 6, 4, 2, 64, 4, 300
    g = gen(9)
    Kq, Vq, ks, vs = filled_cache(g, B, H, N, d)
    q = normal(g, B, T, H_q, d)
    ln = i32(70)
    idx = torch.full((B, H, T, K), -1, dtype=torch.int32, device=DEV)
    idx[0, :, 1] = i32(2, 3, 4, -1)          # all behind the query
    idx[0, :, 2] = i32(-1, 0, -1, -5)        # holes
    idx[0, :, 3] = i32(1, 1, 0, 1)           # twice counts twice, in any order
    idx[0, :, 4] = i32(0, 5, 1 << 30, 1)     # past the cache: skipped and flagged
    idx[0, :, 5] = i32(0, 1, -1, -1)
    O, L = pisa.pisa_sparse_attn_cache(q, Kq, Vq, ks, vs, idx, ln)
    assert pisa.pisa_get_last_device_error() == 5
    o, l, to, tl = sparse64(q, Kq, Vq, ks, vs, idx, ln, i32(T))
    R.close(O, o, to, "O")
    R.close(L, l, tl, "LSE")
    assert (O[0, :2] == 0).all() and torch.isneginf(L[0, :2]).all()


def test_sparse_extreme_logits():
    """Logits far outside the range of exp: the running maximum carries them; a NaN row shows."""
    g = gen(4)
    Kq, Vq, ks, vs = filled_cache(g, 1, 1, 256, 128)
    q = normal(g, 1, 1, 16, 128, scale=40)
    ks[0, 0, 200:] *= 300
    idx = i32(0, 1, 2, 3).reshape(1, 1, 1, 4)
    O, L = pisa.pisa_sparse_attn_cache(q, Kq, Vq, ks, vs, idx, i32(255))
    o, l, to, tl = sparse64(q, Kq, Vq, ks, vs, idx, i32(255), i32(1))
    R.close(L, l, tl, "LSE")
    R.close(O, o, to, "O")
    ks[0, 0, 17] = math.nan
    O, L = pisa.pisa_sparse_attn_cache(q, Kq, Vq, ks, vs, idx, i32(255))
    assert O.isnan().all() and L.isnan().all()
    only = i32(0, -1, -1, -1).reshape(1, 1, 1, 4)
    ks[0, 0, :] = math.nan
    O, L = pisa.pisa_sparse_attn_cache(q, Kq, Vq, ks, vs, only, i32(255))
    assert O.isnan().all() and L.isnan().all()


@pytest.mark.parametrize("spread", [5, 90])
@pytest.mark.parametrize("H_q", [4, 16])
def test_sparse_value_scales_far_apart(spread, H_q):
    """Value scales 2^-spread .. 2^spread times their own, rising and falling over the keys; some of 0."""
    g = gen(14)
    N, d, K = 640, 128, 10
    Kq, Vq, ks, vs = filled_cache(g, 2, 1, N, d)
    ramp = torch.linspace(-spread, spread, N, device=DEV).round().exp2()
    vs[0] *= ramp
    vs[1] *= ramp.flip(0)
    vs[:, :, 3::89] = 0
    q = normal(g, 2, 1, H_q, d)
    idx = torch.arange(K, dtype=torch.int32, device=DEV).expand(2, 1, 1, K).contiguous()
    ln, n = i32(N - 1, N - 1), i32(1, 1)
    O, lse = pisa.pisa_sparse_attn_cache(q, Kq, Vq, ks, vs, idx, ln)
    o, l, to, tl = sparse64(q, Kq, Vq, ks, vs, idx, ln, n)
    R.close(O, o, to, "O")
    R.close(lse, l, tl, "LSE")


def test_sparse_lengths_that_do_not_fit():
    g = gen(5)
    Kq, Vq, ks, vs = filled_cache(g, 3, 1, 100, 64)
    q = normal(g, 3, 2, 2, 64)
    idx = torch.zeros((3, 1, 2, 1), dtype=torch.int32, device=DEV)
    O, L = pisa.pisa_sparse_attn_cache(q, Kq, Vq, ks, vs, idx, i32(-1, 99, 50), new_len=i32(2, 2, 2))
    assert pisa.pisa_get_last_device_error() == 5
    assert (O[:2] == 0).all() and (O[2] != 0).any()


def test_far_rows():
    """Offsets past 32 bits: the last rows of a cache of more than 4 GB."""
    B, H, N, d = 1, 8, (1 << 22) + 9, 128
    g = gen(6)
    Kq, Vq = (torch.zeros((B, H, N, d), dtype=torch.int8, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros((B, H, N), device=DEV) for _ in range(2))
    T = 70
    k, v, q = normal(g, B, H, T, d), normal(g, B, H, T, d), normal(g, B, 1, H, d)
    ln = i32(N - T)
    pisa.pisa_cache_write(k, v, Kq, Vq, ks, vs, ln)
    rk, rv = pisa.pisa_cache_read(Kq, Vq, ks, vs, T, start=ln)
    for x, got, c in ((k, rk, Kq), (v, rv, Vq)):
        code, _, val = R.quantise64(x)
        assert torch.equal(got, val) and torch.equal(c[:, :, N - T:], code)
    last = (N - 1) // 64
    idx = i32(last - 1, last).reshape(1, 1, 1, 2).expand(B, H, 1, 2).contiguous()
    O, L = pisa.pisa_sparse_attn_cache(q, Kq, Vq, ks, vs, idx, i32(N - 1))
    o, l, to, tl = sparse64(q, Kq, Vq, ks, vs, idx, i32(N - 1), i32(1))
    R.close(O, o, to, "O")
    R.close(L, l, tl, "LSE")
    no_error()
