"""Attention over a shared prefix on the GPU, alone and together with the decode operators, against
plain forms in 64 bits."""
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


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def no_error():
    assert pisa.pisa_get_last_device_error() == 0


def prefix(g, P, H, N, d, bits, lens, behind=True):
    """Caches with what must not be read (NaN, infinities) behind every length."""
    K, V = normal(g, P, H, N, d), normal(g, P, H, N, d)
    if bits == 16:
        if behind:
            for p in range(P):
                K[p, :, lens[p]:] = math.nan
                V[p, :, lens[p]:] = math.inf
        return K, V, None, None
    kc, ks, _ = R.quantise64(K)
    vc, vs, _ = R.quantise64(V)
    if behind:
        for p in range(P):
            ks[p, :, lens[p]:] = math.nan
            vs[p, :, lens[p]:] = math.inf
    return kc, vc, ks, vs


def prefix64(q, K, V, ks, vs, lens, rows, o_own=None, lse_own=None, scale=None):
    R_, H_q, d = q.shape
    P, H = K.shape[:2]
    G = H_q // H
    o = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    lse = torch.full((R_, H_q), -math.inf, dtype=torch.float64, device=DEV)
    to, tl = torch.zeros_like(o), torch.zeros_like(lse)
    for p in range(P):
        a, b = rows[p], rows[p + 1]
        for h in range(H):
            k, v = K[p, h, :lens[p]].double(), V[p, h, :lens[p]].double()
            if ks is not None:
                k, v = k * ks[p, h, :lens[p]].double()[:, None], v * vs[p, h, :lens[p]].double()[:, None]
            s = slice(h * G, h * G + G)
            r = R.attend64(q[a:b, s].double().reshape(-1, d), k, v, scale, None if vs is None else vs[p, h, :lens[p]].double())
            if o_own is not None:
                r = R.join64(*r, o_own[a:b, s].double().reshape(-1, d), lse_own[a:b, s].double().reshape(-1))
            for dst, x in zip((o, lse, to, tl), r):
                dst[a:b, s] = x.reshape(dst[a:b, s].shape)
    return o, lse, to, tl


CASES = [  # R, H_q, H, d, N, lens, rows
    (1, 1, 1, 64, 1, [1], [0, 1]),
    (3, 4, 1, 64, 1000, [1000], [0, 3]),
    (1, 16, 1, 128, 5000, [4999], [0, 1]),
    (5, 8, 4, 128, 129, [128], [0, 5]),
    (64, 32, 8, 128, 700, [700], [0, 64]),
    (130, 4, 2, 64, 1030, [1025], [0, 130]),
    (33, 16, 2, 128, 300, [257, 0, 300, 1], [0, 9, 12, 12, 33]),
    (40, 8, 1, 64, 513, [0, 512, 513], [0, 20, 40, 40]),
    (300, 16, 1, 128, 400, [399, 128], [0, 10, 300]),
    (7, 2, 2, 128, 64, [3] * 7, [0, 1, 2, 3, 4, 5, 6, 7]),
    (70, 2, 1, 64, 90, list(range(20, 90)), list(range(71))),
    (1024, 16, 1, 64, 260, [260], [0, 1024]),
    (513, 1, 1, 128, 131, [131], [0, 513]),
    (2000, 2, 1, 64, 5000, [4321], [0, 2000]),
    (90, 16, 4, 128, 3000, [2990], [0, 90]),
    # long enough for every ring of tiles to turn many times, by few, some and many rows
    (2, 16, 8, 128, 60000, [59999], [0, 2]),
    (16, 16, 8, 64, 70000, [70000], [0, 16]),
    (6, 32, 4, 128, 50001, [50001], [0, 6]),
    (37, 16, 4, 128, 50001, [49999], [0, 37]),
    # blocks that meet two jobs and more, of groups of different sizes
    (150, 16, 8, 128, 6000, [5000, 6000, 3], [0, 60, 140, 150]),
    (9, 16, 8, 128, 20000, [19999, 777, 20000], [0, 3, 8, 9]),
    (12, 32, 8, 64, 20000, [19000, 5, 20000, 64], [0, 4, 4, 9, 12]),
    (1600, 8, 8, 64, 700, list(range(100, 700, 15)), list(range(0, 1601, 40))),
    (64, 32, 8, 64, 4000, [3999], [0, 64]),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"R{c[0]}_{c[1]}x{c[2]}_d{c[3]}_N{c[4]}_P{len(c[5])}")
@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("own", [False, True])
def test_prefix(case, bits, own):
    Rn, H_q, H, d, N, lens, rows = case
    P = len(lens)
    g = gen(Rn + N + bits)
    q = normal(g, Rn, H_q, d, scale=1.5)
    K, V, ks, vs = prefix(g, P, H, N, d, bits, lens)
    oo = ll = None
    if own:
        oo = normal(g, Rn, H_q, d, scale=0.2)
        ll = torch.randn((Rn, H_q), generator=g, device=DEV) * 3 + 5
        ll[::3] = -math.inf
        oo[::3] = math.nan  # nothing is taken of these
    want = prefix64(q, K, V, ks, vs, lens, rows, oo, ll)
    o, lse = pisa.pisa_prefix_attn(q, K, V, i32(*lens), row_start=i32(*rows), k_scale=ks, v_scale=vs, o_own=oo, lse_own=ll)
    R.close(lse, want[1], want[3], "lse")
    R.close(o, want[0], want[2], "o")
    again, _ = pisa.pisa_prefix_attn(q, K, V, i32(*lens), row_start=i32(*rows), k_scale=ks, v_scale=vs, o_own=oo, lse_own=ll)
    assert torch.equal(o, again)  # the same in every run
    if P == 1 and rows == [0, Rn]:
        alone, _ = pisa.pisa_prefix_attn(q, K, V, i32(*lens), k_scale=ks, v_scale=vs, o_own=oo, lse_own=ll, want_lse=False)
        assert torch.equal(o, alone)
    if own:  # in place
        a, b = pisa.pisa_prefix_attn(q, K, V, i32(*lens), row_start=i32(*rows), k_scale=ks, v_scale=vs, o_own=oo,
                                     lse_own=ll, o=oo, lse=ll)
        assert a is oo and torch.equal(a, o) and torch.equal(b, lse)
    no_error()


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("Rn", [12, 200])
def test_rows_outside_the_groups_stay(bits, Rn):
    g = gen(3)
    q = normal(g, Rn, 8, 64)
    lens, rows = [130, 77], [2, 5, Rn - 3]
    K, V, ks, vs = prefix(g, 2, 2, 150, 64, bits, lens)
    o = torch.full((Rn, 8, 64), 4.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((Rn, 8), 4.0, device=DEV)
    pisa.pisa_prefix_attn(q, K, V, i32(*lens), row_start=i32(*rows), k_scale=ks, v_scale=vs, o=o, lse=lse)
    want = prefix64(q, K, V, ks, vs, lens, rows)
    inside = slice(2, Rn - 3)
    R.close(o[inside], want[0][inside], want[2][inside], "o")
    R.close(lse[inside], want[1][inside], want[3][inside], "lse")
    for x in (o, lse):
        assert (x[:2] == 4).all() and (x[Rn - 3:] == 4).all()


@pytest.mark.parametrize("Rn", [10, 160])
def test_bounds_and_lengths_out_of_range(Rn):
    """Brought into range and flagged."""
    g = gen(8)
    q = normal(g, Rn, 2, 64)
    K, V, ks, vs = prefix(g, 3, 1, 40, 64, 8, [40] * 3, behind=False)
    lens, rows = [41, -3, 40], [-2, 4, 4, Rn + 9]
    o, lse = pisa.pisa_prefix_attn(q, K, V, i32(*lens), row_start=i32(*rows), k_scale=ks, v_scale=vs)
    assert pisa.pisa_get_last_device_error() == 5
    want = prefix64(q, K, V, ks, vs, [40, 0, 40], [0, 4, 4, Rn])
    R.close(o, want[0], want[2], "o")
    R.close(lse, want[1], want[3], "lse")


@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("Rn", [2, 140])
def test_extreme_logits(own, bits, Rn):
    """Maxima that move by far more than exp's range from step to step, growing and shrinking; and a NaN
    in a prefix, with and without own results to join."""
    g = gen(11)
    N, d = 1500, 128
    q = normal(g, Rn, 4, d, scale=10)
    K, V, ks, vs = prefix(g, 1, 2, N, d, bits, [N])
    oo = ll = None
    if own:
        oo, ll = normal(g, Rn, 4, d), torch.randn((Rn, 4), generator=g, device=DEV) * 200
    ramp = torch.cat([torch.linspace(0.01, 8, N // 2), torch.linspace(8, 0.01, N - N // 2)]).to(DEV)
    if bits == 8:
        ks *= ramp
    else:
        K = (K.float() * ramp[:, None]).to(torch.bfloat16)
    want = prefix64(q, K, V, ks, vs, [N], [0, Rn], oo, ll, scale=0.3)
    o, lse = pisa.pisa_prefix_attn(q, K, V, i32(N), k_scale=ks, v_scale=vs, o_own=oo, lse_own=ll, scale=0.3)
    R.close(lse, want[1], want[3], "lse")
    R.close(o, want[0], want[2], "o")
    bad = K.clone()
    if bits == 8:
        ks[0, 0, 700] = math.nan
    else:
        bad[0, 0, 700, 5] = math.nan
    o, lse = pisa.pisa_prefix_attn(q, bad, V, i32(N), k_scale=ks, v_scale=vs, o_own=oo, lse_own=ll, scale=0.3)
    assert o[:, :2].isnan().all() and lse[:, :2].isnan().all() and not o[:, 2:].isnan().any()
    no_error()


@pytest.mark.parametrize("spread", [5, 90])
@pytest.mark.parametrize("Rn,P", [(1, 1), (40, 1), (2, 2), (140, 2)])
def test_value_scales_far_apart(spread, Rn, P):
    """Scales 2^-spread .. 2^spread, rising over one prefix and falling over the other; some of 0."""
    g = gen(13)
    N, d = 1280, 64
    q = normal(g, Rn, 4, d)
    lens, rows = [N, N - 1][:P], [0, Rn] if P == 1 else [0, Rn // 2, Rn]
    K, V, ks, vs = prefix(g, P, 2, N, d, 8, lens, behind=False)
    ramp = torch.linspace(-spread, spread, N, device=DEV).round().exp2()
    vs[0] = ramp
    vs[P - 1, 1] = ramp.flip(0)
    vs[:, :, 5::97] = 0
    oo, ll = normal(g, Rn, 4, d), torch.randn((Rn, 4), generator=g, device=DEV) * 3 + 7
    for own in ((None, None), (oo, ll)):
        want = prefix64(q, K, V, ks, vs, lens, rows, *own)
        o, lse = pisa.pisa_prefix_attn(q, K, V, i32(*lens), row_start=i32(*rows), k_scale=ks, v_scale=vs, o_own=own[0],
                                       lse_own=own[1])
        R.close(lse, want[1], want[3], "lse")
        R.close(o, want[0], want[2], "o")
    no_error()


@pytest.mark.parametrize("Rn", [4, 150])
def test_far_prefix(Rn):
    """Offsets past 32 bits: the last prefixes and keys of a cache of more than 4 GB."""
    P, H, N, d = 3, 4, (1 << 21) + 5, 128
    g = gen(12)
    K = torch.zeros((P, H, N, d), dtype=torch.int8, device=DEV)
    V = torch.zeros_like(K)
    ks, vs = (torch.zeros((P, H, N), device=DEV) for _ in range(2))
    tail = 300
    for c, s in ((K, ks), (V, vs)):
        code, sc, _ = R.quantise64(normal(g, H, tail, d))
        c[P - 1, :, N - tail:], s[P - 1, :, N - tail:] = code, sc
    q = normal(g, Rn, 8, d, scale=3)
    lens, rows = [0, 1, N], [0, 1, 1, Rn]
    o, lse = pisa.pisa_prefix_attn(q, K, V, i32(*lens), row_start=i32(*rows), k_scale=ks, v_scale=vs)
    for h in range(H):
        k = K[P - 1, h, N - tail:].double() * ks[P - 1, h, N - tail:].double()[:, None]
        v = V[P - 1, h, N - tail:].double() * vs[P - 1, h, N - tail:].double()[:, None]
        a, b, to, tl = R.attend64(q[1:, 2 * h:2 * h + 2].double().reshape(-1, d), k, v, vs=vs[P - 1, h, N - tail:].double())
        # the zero keys before the tail: weight 1 and value 0 each
        j = R.join64(a, b, to, tl, torch.zeros_like(a), torch.full_like(b, math.log(N - tail)))
        # a sum of 2^21 weights in at least 8 * 152 parts of at most 2^11 terms: 2^11 F relative, 2.4e-4
        R.close(lse[1:, 2 * h:2 * h + 2].reshape(-1), j[1], j[3] + 2 ** 11 * R.F, "lse")
        R.close(o[1:, 2 * h:2 * h + 2].reshape(-1, d), j[0], j[2] + 2 ** 11 * R.F * j[0].abs(), "o")
    no_error()


# ---- together, as they are used ----------------------------------------------------------------
@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("B,H_q,H,d", [(3, 8, 2, 128), (40, 16, 1, 64)])
def test_serving_run(bits, B, H_q, H, d):
    """A shared prompt, then decode steps: each sequence's own tokens by the sparse decode step (all their
    blocks selected, so exact) over its own cache, joined with the prompt; and by the 8-bit cache."""
    g = gen(B)
    G, NP, steps, cap, K_sel = H_q // H, 300, 70, 128, 2
    pk, pv = normal(g, 1, H, NP, d), normal(g, 1, H, NP, d)
    if bits == 8:
        Kp, Vp = (torch.zeros((1, H, NP + 20, d), dtype=torch.int8, device=DEV) for _ in range(2))
        ks, vs = (torch.zeros((1, H, NP + 20), device=DEV) for _ in range(2))
        cut = 111  # the prompt arrives in two pieces
        pisa.pisa_cache_write(pk[:, :, :cut].contiguous(), pv[:, :, :cut].contiguous(), Kp, Vp, ks, vs, i32(0))
        pisa.pisa_cache_write(pk[:, :, cut:].contiguous(), pv[:, :, cut:].contiguous(), Kp, Vp, ks, vs, i32(cut))
        rk, rv = pisa.pisa_cache_read(Kp, Vp, ks, vs, NP)
        pk64, pv64 = (x[:, :, :NP].double() * s[:, :, :NP].double()[..., None] for x, s in ((Kp, ks), (Vp, vs)))
        for got, w in ((rk, pk64), (rv, pv64)):
            assert (got.double() - w).abs().le(R.U * w.abs()).all()
    else:
        Kp, Vp, ks, vs = pk, pv, None, None
        pk64, pv64 = pk.double(), pv.double()
    Kc, Vc = (torch.zeros((B, H, cap, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    Pc = torch.zeros((B, H, pisa.pisa_pyramid_nodes(cap), d), dtype=torch.bfloat16, device=DEV)
    seq = torch.zeros(B, dtype=torch.int32, device=DEV)
    K8, V8 = (torch.zeros((B, H, cap, d), dtype=torch.int8, device=DEV) for _ in range(2))
    s8, t8 = (torch.zeros((B, H, cap), device=DEV) for _ in range(2))
    for step in range(steps):
        q, k, v = normal(g, B, H_q, d), normal(g, B, H, d), normal(g, B, H, d)
        before = seq.clone()
        lse = torch.empty((B, H_q), device=DEV)
        idx = torch.empty((B, H, K_sel), dtype=torch.int32, device=DEV)
        o = pisa.pisa_decode_step(q, k, v, Kc, Vc, Pc, seq, K_sel, lse=lse, idx_out=idx)
        oj, lj = pisa.pisa_prefix_attn(q, Kp, Vp, i32(NP), k_scale=ks, v_scale=vs, o_own=o, lse_own=lse)
        pisa.pisa_cache_write(k, v, K8, V8, s8, t8, before)
        o8, l8 = pisa.pisa_sparse_attn_cache(q, K8, V8, s8, t8, idx, before)
        o8, l8 = pisa.pisa_prefix_attn(q, Kp, Vp, i32(NP), k_scale=ks, v_scale=vs, o_own=o8, lse_own=l8, o=o8, lse=l8)
        if step % 23 and step != steps - 1:
            continue
        n = step + 1
        for b in (0, B - 1):
            for h in range(H):
                s = slice(h * G, h * G + G)
                own = (Kc[b, h, :n].double(), Vc[b, h, :n].double())
                own8 = (K8[b, h, :n].double() * s8[b, h, :n].double()[:, None],
                        V8[b, h, :n].double() * t8[b, h, :n].double()[:, None])
                for (kk, vv), og, lg in ((own, oj, lj), (own8, o8, l8)):
                    kk, vv = torch.cat([pk64[0, h], kk]), torch.cat([pv64[0, h], vv])
                    # (as if all values were codes of one scale: the larger bound)
                    a, l, to, tl = R.attend64(q[b, s].double(), kk, vv, vs=torch.ones_like(vv[:, 0]))
                    # two parts joined: the lse of each is off by tl, the own result was rounded to bf16 on its
                    # way (U of it, at most U sum w|v|, within `to` once more)
                    R.close(lg[b, s], l, 2 * tl, "lse")
                    R.close(og[b, s], a, 2 * to + 2 * tl[:, None] * vv.abs().amax(), "o")
    assert (seq == steps).all()
    no_error()


def test_graph_and_streams():
    """Captured and replayed with new inputs; two graphs with a scratch each, on two streams."""
    g = gen(21)
    B, H_q, H, d, N, K_sel = 8, 16, 2, 128, 600, 4
    q = normal(g, B, H_q, d)
    k, v = normal(g, B, H, d), normal(g, B, H, d)
    Kp, Vp, ks, vs = prefix(g, 1, H, 500, d, 8, [500])
    K8, V8 = (torch.zeros((B, H, N, d), dtype=torch.int8, device=DEV) for _ in range(2))
    s8, t8 = (torch.zeros((B, H, N), device=DEV) for _ in range(2))
    fill, fillv = normal(g, B, H, 300, d), normal(g, B, H, 300, d)
    pisa.pisa_cache_write(fill, fillv, K8, V8, s8, t8, torch.zeros(B, dtype=torch.int32, device=DEV))
    seq = torch.full((B,), 300, dtype=torch.int32, device=DEV)
    idx = i32(0, 2, 3, 4).expand(B, H, K_sel).contiguous()
    plen = i32(500)

    def step(out):
        pisa.pisa_cache_write(k, v, K8, V8, s8, t8, seq)
        o, l = pisa.pisa_sparse_attn_cache(q, K8, V8, s8, t8, idx, seq)
        out["o"], out["l"] = pisa.pisa_prefix_attn(q, Kp, Vp, plen, k_scale=ks, v_scale=vs, o_own=o, lse_own=l)

    eager = {}
    step(eager)
    torch.cuda.synchronize()
    kept = []
    for _ in range(2):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        out = {}
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step(out)
        kept.append((graph, out, s))
    torch.cuda.synchronize()
    for rep in range(3):
        q.copy_(normal(g, B, H_q, d))
        k.copy_(normal(g, B, H, d))
        seq.fill_(300 + rep)
        step(eager)
        torch.cuda.synchronize()
        for graph, out, s in kept:  # at once: the same rows are written with the same values
            out["o"].zero_()
        torch.cuda.synchronize()
        for graph, out, s in kept:
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for graph, out, s in kept:
            assert torch.equal(out["o"], eager["o"]) and torch.equal(out["l"], eager["l"])
    no_error()


def test_phases_are_timed():
    g = gen(2)
    Kp, Vp, ks, vs = prefix(g, 1, 1, 100, 64, 8, [100])
    q = normal(g, 2, 1, 64)
    pisa.pisa_phase_timing(True)
    try:
        pisa.pisa_prefix_attn(q, Kp, Vp, i32(100), k_scale=ks, v_scale=vs)
        pisa.pisa_cache_read(Kp, Vp, ks, vs, 100)
        pisa.pisa_cache_write(normal(g, 1, 1, 64), normal(g, 1, 1, 64), Kp, Vp, ks, vs, i32(0))
        pisa.pisa_sparse_attn_cache(q[:1], Kp, Vp, ks, vs, i32(0).reshape(1, 1, 1), i32(3))
        t = pisa.pisa_phase_times()
    finally:
        pisa.pisa_phase_timing(False)
    for name in ("cache_write", "cache_read", "sparse_attn_cache", "prefix_attn"):
        assert t[name][1] == 1 and t[name][0] > 0
