"""Workloads of the serving operators over an 8-bit key/value cache and over a shared prefix.

Four operators, each in its plain form (elementary torch operations in 32 bits) and as the
library's call (``own``):

  write    quantise new K and V rows into the 8-bit cache and give back the values it then holds
  read     read rows of the 8-bit cache back as bf16
  sparse   attention of a sequence's new tokens over selected 64-key blocks of the 8-bit cache
  prefix   attention of a batch over a prefix that its sequences share (bf16 or 8-bit), joined by
           log-sum-exp with what each sequence attended on its own

The quantiser: a = max|x| of a row, scale = a / 127, code = sign(x) floor(127 |x| / a + 1/2).
"""
import math

import numpy as np
import torch

own = False

C = 64  # keys a block


# ---- cases ---------------------------------------------------------------------------------
def listed():
    return [
        # one decode step of 64 sequences appends its token to the cache (8 KV heads)
        dict(name="write_step", op="write", B=64, T=1, H_kv=8, d=128, N_cap=1024, ragged=False),
        # a padded batch of prompts of different lengths
        dict(name="write_ragged", op="write", B=12, T=1371, H_kv=2, d=64, N_cap=2050, ragged=True),
        # one long prompt, every row at once
        dict(name="write_prompt", op="write", B=1, T=131072, H_kv=8, d=128, N_cap=131072, ragged=False),
        # a few short ranges read back, at odd starts
        dict(name="read_ragged", op="read", B=7, T=333, H_kv=4, d=64, N_cap=1999, ragged=True),
        # whole caches read back (to rebuild the pyramid, to select in the prefill form)
        dict(name="read_caches", op="read", B=4, T=32768, H_kv=8, d=128, N_cap=32768, ragged=False),
        # one sequence, one token: latency
        dict(name="sparse_one", op="sparse", B=1, T=1, H_q=16, H_kv=1, d=128, K=16, N_cap=32768, ragged=False),
        # the batched decode step: 64 sequences, 32 query heads over 8 KV heads
        dict(name="sparse_step", op="sparse", B=64, T=1, H_q=32, H_kv=8, d=128, K=16, N_cap=32768, ragged=False),
        # drafted tokens, up to five a sequence, sequences of different lengths
        dict(name="sparse_drafts", op="sparse", B=24, T=5, H_q=32, H_kv=2, d=128, K=32, N_cap=9001, ragged=True),
        # three short answers after one short instruction: latency
        dict(name="prefix_few", op="prefix", P=1, R=3, H_q=4, H_kv=1, d=64, N_cap=1000, bits=8, joined=True),
        # 64 sequences after one system prompt, the prefix in 8 bits
        dict(name="prefix_step", op="prefix", P=1, R=64, H_q=32, H_kv=8, d=128, N_cap=32768, bits=8, joined=True),
        # five documents, each with its own group of sequences
        dict(name="prefix_groups", op="prefix", P=5, R=217, H_q=16, H_kv=4, d=128, N_cap=10007, bits=16, joined=True),
        # 64 sequences of four drafted tokens each over one long document
        dict(name="prefix_long", op="prefix", P=1, R=256, H_q=32, H_kv=2, d=128, N_cap=131072, bits=16, joined=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "sparse", "prefix"])
    d = rng.choice([64, 128])
    if op in ("write", "read"):
        B, H_kv = _log(rng, 1, 64), rng.choice([1, 2, 4, 8])
        most = (1 << 20) // (B * H_kv)
        T = _log(rng, 1, max(1, min(131072, most)))
        N_cap = T + _log(rng, 1, max(2, most - T)) if most > T else T
        return dict(op=op, B=B, T=T, H_kv=H_kv, d=d, N_cap=N_cap, ragged=rng.random() < 0.7)
    G = rng.choice([1, 2, 4, 8, 16])
    H_kv = rng.choice([1, 2, 4, 8])
    if op == "sparse":
        T = rng.choice([1, 1, 2, 3, 5, 8])
        B = _log(rng, 1, max(1, 512 // (H_kv * T)))
        N_cap = _log(rng, 64, max(64, min(65536, (1 << 24) // (B * H_kv))))
        return dict(op=op, B=B, T=min(T, N_cap), H_q=G * H_kv, H_kv=H_kv, d=d, K=rng.choice([4, 8, 16, 32]), N_cap=N_cap,
                    ragged=rng.random() < 0.5)
    P = rng.choice([1, 1, 2, 3, 6])
    R = _log(rng, P, 256)
    # at most the largest listed case's products
    N_cap = _log(rng, 100, max(100, min(131072, 256 * 32 * 131072 // (P * R * G * H_kv))))
    return dict(op=op, P=P, R=R, H_q=G * H_kv, H_kv=H_kv, d=d, N_cap=N_cap, bits=rng.choice([8, 16]),
                joined=rng.random() < 0.7)


# ---- inputs --------------------------------------------------------------------------------
def _normal(gen, shape, dev, scale=1.0):
    return (torch.randn(shape, generator=gen, device=dev) * scale).to(torch.bfloat16)


def _codes(x):
    """Plain quantiser: bf16 rows -> (int8 codes, fp32 scale a row).  127 |x| is exact in 32 bits and the
    quotient keeps ties exact, so the codes are those of the real quotient."""
    x = x.float()
    a = x.abs().amax(dim=-1)
    u = torch.floor(x.abs() * 127 / torch.where(a > 0, a, torch.ones_like(a))[..., None] + 0.5)
    return torch.copysign(u, x).to(torch.int8), a / 127


def _cache(gen, B, H_kv, N_cap, d, dev):
    """A filled 8-bit cache: every row quantised from normal K (with an offset a block) and V rows."""
    q = [torch.empty(B, H_kv, N_cap, d, dtype=torch.int8, device=dev) for _ in range(2)]
    s = [torch.empty(B, H_kv, N_cap, dtype=torch.float32, device=dev) for _ in range(2)]
    nb = -(-N_cap // C)
    for b in range(B):
        for i in range(2):
            x = torch.randn((H_kv, N_cap, d), generator=gen, device=dev)
            if i == 0:
                x += torch.randn((H_kv, nb, 1, d), generator=gen, device=dev).mul(0.5).expand(-1, -1, C, -1).reshape(
                    H_kv, nb * C, d)[:, :N_cap]
            q[i][b], s[i][b] = _codes(x.to(torch.bfloat16))
    return q[0], q[1], s[0], s[1]


def _ints(gen, lo, hi, n, dev):
    """n whole numbers, number i uniform in [lo, hi[i]]."""
    u = torch.rand(n, generator=gen, device=dev, dtype=torch.float64)
    return (lo + torch.floor(u * (hi - lo + 1))).to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    c, d = dict(case), case["d"]
    s = dict(case=c, op=c["op"])
    if c["op"] == "write":
        B, H, T, N = c["B"], c["H_kv"], c["T"], c["N_cap"]
        s["k"], s["v"] = _normal(gen, (B, H, T, d), dev), _normal(gen, (B, H, T, d), dev)
        s["new"] = None
        n = torch.full((B,), T, dtype=torch.int32, device=dev)
        if c["ragged"]:
            n = _ints(gen, min(1, T), n.double(), B, dev)
            n[-1] = T
            s["new"] = n
        s["len"] = _ints(gen, 0, N - n.double(), B, dev)  # rows already there
        s["Kq"], s["Vq"] = (torch.randint(-127, 128, (B, H, N, d), generator=gen, device=dev, dtype=torch.int8)
                            for _ in range(2))
        s["ks"], s["vs"] = (torch.rand((B, H, N), generator=gen, device=dev) * 0.01 + 0.015 for _ in range(2))
        s["k_out"], s["v_out"] = torch.zeros_like(s["k"]), torch.zeros_like(s["v"])
    elif c["op"] == "read":
        B, H, T, N = c["B"], c["H_kv"], c["T"], c["N_cap"]
        s["Kq"], s["Vq"], s["ks"], s["vs"] = _cache(gen, B, H, N, d, dev)
        s["start"] = s["n"] = None
        if c["ragged"]:
            s["n"] = _ints(gen, 0, torch.full((B,), T, device=dev).double(), B, dev)
            s["n"][0] = T
            s["start"] = _ints(gen, 0, N - s["n"].double(), B, dev)
        s["k_out"], s["v_out"] = (torch.zeros((B, H, T, d), dtype=torch.bfloat16, device=dev) for _ in range(2))
    elif c["op"] == "sparse":
        B, H, T, N, K = c["B"], c["H_kv"], c["T"], c["N_cap"], c["K"]
        s["q"] = _normal(gen, (B, T, c["H_q"], d), dev, 1.5)
        s["Kq"], s["Vq"], s["ks"], s["vs"] = _cache(gen, B, H, N, d, dev)
        s["len"] = torch.full((B,), N - T, dtype=torch.int32, device=dev)
        s["new"] = None
        if c["ragged"]:
            s["len"] = _ints(gen, 0, s["len"].double(), B, dev)
            s["new"] = _ints(gen, 1, torch.full((B,), T, device=dev).double(), B, dev)
        # K blocks a query: its own and K - 1 others that start at or before it, ascending, -1 behind
        M = -(-N // C)
        pos = s["len"][:, None].long() + torch.arange(T, device=dev)
        j = torch.arange(M, device=dev)
        r = torch.rand((B, H, T, M), generator=gen, device=dev)
        at = (pos // C)[:, None, :, None]
        r = torch.where(j == at, 2.0, torch.where(j < at, r, -1.0))
        top, idx = r.topk(min(K, M), dim=-1)
        idx = torch.where(top >= 0, idx, M).sort(dim=-1).values
        full = torch.full((B, H, T, K), -1, dtype=torch.int32, device=dev)
        full[..., : idx.shape[-1]] = torch.where(idx == M, -1, idx).int()
        s["idx"] = full
        s["o"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros((B, T, c["H_q"]), dtype=torch.float32, device=dev)
    else:
        P, R, H, N = c["P"], c["R"], c["H_kv"], c["N_cap"]
        s["q"] = _normal(gen, (R, c["H_q"], d), dev, 1.5)
        s["ks"] = s["vs"] = None
        if c["bits"] == 8:
            s["K"], s["V"], s["ks"], s["vs"] = _cache(gen, P, H, N, d, dev)
        else:
            s["K"], s["V"] = _normal(gen, (P, H, N, d), dev), _normal(gen, (P, H, N, d), dev)
        full = torch.full((P,), N, device=dev)
        s["len"] = full.int() if P == 1 else _ints(gen, max(1, N // 3), full.double(), P, dev)
        cuts = torch.sort(_ints(gen, 0, torch.full((P - 1,), R, device=dev).double(), P - 1, dev)).values if P > 1 else full[:0]
        zero = torch.zeros(1, dtype=torch.int32, device=dev)
        s["rows"] = torch.cat([zero, cuts.int(), zero + R])
        s["o_own"] = s["lse_own"] = None
        if c["joined"]:  # what a sequence's own few hundred tokens gave
            s["o_own"] = _normal(gen, (R, c["H_q"], d), dev, 0.1)
            s["lse_own"] = torch.rand((R, c["H_q"]), generator=gen, device=dev) * 4 + 7
    return s


# ---- one pass ------------------------------------------------------------------------------
def _spots(start, n, T, B, dev):
    """Cache rows [B, T] from starts (None: 0), and which of them are in use from counts (None: all)."""
    t = torch.arange(T, device=dev)
    rows = t.expand(B, T) if start is None else start.long()[:, None] + t
    return rows, None if n is None else t < n[:, None]


def _fill(out, live, x):
    """out = x where live [B, T] (None: everywhere); out [B, H, T, d]."""
    out.copy_(x if live is None else torch.where(live[:, None, :, None], x, out))


def _plain_write(s):
    B, H, T, d = s["k"].shape
    dev = s["k"].device
    rows, live = _spots(s["len"], s["new"], T, B, dev)
    b = torch.arange(B, device=dev)[:, None, None].expand(B, H, T)
    h = torch.arange(H, device=dev)[None, :, None].expand(B, H, T)
    at = rows[:, None, :].expand(B, H, T)
    pick = slice(None)
    if live is not None:
        pick = live[:, None, :].expand(B, H, T)
        b, h, at = b[pick], h[pick], at[pick]
    for x, q, sc, out in ((s["k"], s["Kq"], s["ks"], s["k_out"]), (s["v"], s["Vq"], s["vs"], s["v_out"])):
        code, scale = _codes(x)
        q[b, h, at] = code[pick]
        sc[b, h, at] = scale[pick]
        _fill(out, live, (code.float() * scale[..., None]).to(torch.bfloat16))
    return dict(k=s["k_out"], v=s["v_out"], k_code=s["Kq"], v_code=s["Vq"], k_scale=s["ks"], v_scale=s["vs"])


def _plain_read(s):
    B, H, T, d = s["k_out"].shape
    dev = s["k_out"].device
    rows, live = _spots(s["start"], s["n"], T, B, dev)
    at = rows if live is None else torch.where(live, rows, 0)
    at = at[:, None, :].expand(B, H, T)
    b = torch.arange(B, device=dev)[:, None, None]
    h = torch.arange(H, device=dev)[None, :, None]
    for q, sc, out in ((s["Kq"], s["ks"], s["k_out"]), (s["Vq"], s["vs"], s["v_out"])):
        _fill(out, live, (q[b, h, at].float() * sc[b, h, at][..., None]).to(torch.bfloat16))
    return dict(k=s["k_out"], v=s["v_out"])


def _softmax_sums(z):
    """z [..., keys], masked entries -inf: weights, their sum and the log-sum-exp (empty rows: 0, 0, -inf)."""
    m = z.amax(dim=-1, keepdim=True)
    w = torch.exp(z - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    l = w.sum(dim=-1)
    return w, l, m[..., 0] + torch.log(l)


def _plain_sparse(s):
    B, T, H_q, d = s["q"].shape
    H, N = s["Kq"].shape[1:3]
    G, dev = H_q // H, s["q"].device
    pos, live = _spots(s["len"], s["new"], T, B, dev)
    keys = (s["idx"].long()[..., None] * C + torch.arange(C, device=dev)).reshape(B, H, T, -1)
    seen = (keys >= 0) & (keys <= pos[:, None, :, None])
    at = torch.where(seen, keys, 0)
    b = torch.arange(B, device=dev)[:, None, None, None]
    h = torch.arange(H, device=dev)[None, :, None, None]
    k = s["Kq"][b, h, at].float() * s["ks"][b, h, at][..., None]
    v = s["Vq"][b, h, at].float() * s["vs"][b, h, at][..., None]
    q = s["q"].float().reshape(B, T, H, G, d).permute(0, 2, 1, 3, 4)
    z = torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    w, l, lse = _softmax_sums(torch.where(seen[..., None, :], z, -math.inf))
    o = torch.matmul(w, v) / torch.where(l > 0, l, torch.ones_like(l))[..., None]
    o = o.permute(0, 2, 1, 3, 4).reshape(B, T, H_q, d).to(torch.bfloat16)
    lse = lse.permute(0, 2, 1, 3).reshape(B, T, H_q)
    if live is not None:  # rows behind a sequence's last new token stay as they were
        o = torch.where(live[..., None, None], o, s["o"])
        lse = torch.where(live[..., None], lse, s["lse"])
    s["o"].copy_(o)
    s["lse"].copy_(lse)
    return dict(o=s["o"], lse=s["lse"])


def _plain_prefix(s):
    R, H_q, d = s["q"].shape
    P, H, N = s["K"].shape[:3]
    G, dev = H_q // H, s["q"].device
    k, v = s["K"].float(), s["V"].float()
    if s["ks"] is not None:
        k, v = k * s["ks"][..., None], v * s["vs"][..., None]
    # the rows of each group, padded to R a group (a single group: the rows as they are)
    first, last = s["rows"][:-1].long(), s["rows"][1:].long()
    most = R
    row = first[:, None] + torch.arange(most, device=dev)
    live = row < last[:, None]
    row = torch.where(live, row, 0)
    if P == 1:
        q = s["q"].float().reshape(1, R, H, G, d).permute(0, 2, 1, 3, 4).reshape(1, H, R * G, d)
    else:
        q = s["q"].float()[row].reshape(P, most, H, G, d).permute(0, 2, 1, 3, 4).reshape(P, H, most * G, d)
    z = torch.matmul(q, k.transpose(-1, -2))
    z *= 1.0 / math.sqrt(d)
    z = z.masked_fill_((torch.arange(N, device=dev) >= s["len"][:, None])[:, None, None, :], -math.inf)
    m = z.amax(dim=-1, keepdim=True)
    w = z.sub_(torch.where(torch.isinf(m), torch.zeros_like(m), m)).exp_()
    l = w.sum(dim=-1)
    lse = m[..., 0] + torch.log(l)
    o = torch.matmul(w, v) / torch.where(l > 0, l, torch.ones_like(l))[..., None]
    o = o.reshape(P, H, most, G, d).permute(0, 2, 1, 3, 4).reshape(P, most, H_q, d)
    lse = lse.reshape(P, H, most, G).permute(0, 2, 1, 3).reshape(P, most, H_q)
    if P == 1:
        o, lse = o[0], lse[0]
    else:
        o, lse = o[live], lse[live]  # the groups' rows in order: rows 0 .. R - 1
    if s["o_own"] is not None:
        m = torch.maximum(lse, s["lse_own"])
        a, b = torch.exp(lse - m), torch.exp(s["lse_own"] - m)
        o = (a[..., None] * o + b[..., None] * s["o_own"].float()) / (a + b)[..., None]
        lse = m + torch.log(a + b)
    return dict(o=o.to(torch.bfloat16), lse=lse)


def run(state):
    s = state
    if own:
        import hierarchical_top_block_gb300 as pisa

        if s["op"] == "write":
            pisa.pisa_cache_write(s["k"], s["v"], s["Kq"], s["Vq"], s["ks"], s["vs"], s["len"], new_len=s["new"],
                                  k_out=s["k_out"], v_out=s["v_out"])
            return dict(k=s["k_out"], v=s["v_out"], k_code=s["Kq"], v_code=s["Vq"], k_scale=s["ks"], v_scale=s["vs"])
        if s["op"] == "read":
            k, v = pisa.pisa_cache_read(s["Kq"], s["Vq"], s["ks"], s["vs"], s["k_out"].shape[2], start=s["start"],
                                        length=s["n"], k_out=s["k_out"], v_out=s["v_out"])
            return dict(k=k, v=v)
        if s["op"] == "sparse":
            o, lse = pisa.pisa_sparse_attn_cache(s["q"], s["Kq"], s["Vq"], s["ks"], s["vs"], s["idx"], s["len"],
                                                 new_len=s["new"], O=s["o"], LSE=s["lse"])
            return dict(o=o, lse=lse)
        o, lse = pisa.pisa_prefix_attn(s["q"], s["K"], s["V"], s["len"], row_start=s["rows"], k_scale=s["ks"],
                                       v_scale=s["vs"], o_own=s["o_own"], lse_own=s["lse_own"])
        return dict(o=o, lse=lse)
    return {"write": _plain_write, "read": _plain_read, "sparse": _plain_sparse, "prefix": _plain_prefix}[s["op"]](s)


# ---- the work a pass cannot do without -------------------------------------------------------
def work(case):
    c, d = case, case["d"]
    if c["op"] in ("write", "read"):
        # ragged: about half of the padded rows are in use
        rows = 2 * c["B"] * c["H_kv"] * c["T"] * (0.5 if c["ragged"] else 1.0)
        return dict(bytes=rows * (d * (5 if c["op"] == "write" else 3) + 4), flops=rows * d * 3)
    if c["op"] == "sparse":
        pairs = c["B"] * c["H_kv"] * c["T"] * (0.5 if c["ragged"] else 1.0)
        keys = min(c["K"] * C, c["N_cap"])
        # a sequence's new tokens may select the same blocks: no row is counted twice
        read = min(pairs * keys, c["B"] * c["H_kv"] * c["N_cap"])
        G = c["H_q"] // c["H_kv"]
        return dict(bytes=read * (2 * d + 8) + pairs * (G * (4 * d + 4) + 4 * c["K"]), flops=pairs * keys * G * d * 4)
    keys = c["N_cap"] * (1.0 if c["P"] == 1 else 2 / 3)
    kv = c["P"] * c["H_kv"] * keys * (2 * d + 8 if c["bits"] == 8 else 4 * d)
    io = c["R"] * c["H_q"] * (4 * d + 4 + (2 * d + 4 if c["joined"] else 0))
    return dict(bytes=kv + io, flops=c["R"] * c["H_q"] * keys * d * 4)


# ---- the definition in 64 bits ---------------------------------------------------------------
def _exact_codes(x):
    """(codes, scale) in float64 of one block of rows."""
    x = x.double()
    a = torch.max(x.abs(), -1).values
    u = (127 * x.abs() / a.clamp(min=1e-300).unsqueeze(-1) + 0.5).floor()
    return torch.where(x < 0, -u, u), a / 127


def _attend64(q, k, v, d):
    """One head group in float64: q [r, d], k and v [n, d] -> o [r, d], lse [r]."""
    z = q @ k.T / math.sqrt(d)
    m = z.max(dim=1, keepdim=True).values
    w = (z - m).exp()
    l = w.sum(1, keepdim=True)
    return (w @ v) / l, (m + l.log())[:, 0]


def exact(case, seed):
    c, s, d = case, prepare(case, seed), case["d"]
    if c["op"] == "write":
        if 2 * c["B"] * c["H_kv"] * c["T"] * d > 1 << 29:
            return None
        out = dict(k_code=None, v_code=None)
        ln = s["len"].tolist()
        nn = s["new"].tolist() if s["new"] is not None else [c["T"]] * c["B"]
        for name, x, sc in (("k", s["k"], s["ks"]), ("v", s["v"], s["vs"])):
            vals, scales = torch.zeros(x.shape, dtype=torch.float64, device=x.device), sc.double()
            for b in range(c["B"]):
                code, a = _exact_codes(x[b, :, : nn[b]])
                vals[b, :, : nn[b]] = code * a[..., None]
                scales[b, :, ln[b] : ln[b] + nn[b]] = a
            out[name], out[name + "_scale"] = vals, scales
        return out
    if c["op"] == "read":
        st = s["start"].tolist() if s["start"] is not None else [0] * c["B"]
        nn = s["n"].tolist() if s["n"] is not None else [c["T"]] * c["B"]
        out = {}
        for name, q, sc in (("k", s["Kq"], s["ks"]), ("v", s["Vq"], s["vs"])):
            vals = torch.zeros((c["B"], c["H_kv"], c["T"], d), dtype=torch.float64, device=q.device)
            for b in range(c["B"]):
                e = st[b] + nn[b]
                vals[b, :, : nn[b]] = q[b, :, st[b] : e].double() * sc[b, :, st[b] : e].double().unsqueeze(-1)
            out[name] = vals
        return out
    G = c["H_q"] // c["H_kv"]
    if c["op"] == "sparse":
        o = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
        lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=s["q"].device)
        ln = s["len"].tolist()
        nn = s["new"].tolist() if s["new"] is not None else [c["T"]] * c["B"]
        idx = s["idx"].cpu().numpy()
        for b in range(c["B"]):
            for h in range(c["H_kv"]):
                for t in range(nn[b]):
                    blocks = idx[b, h, t][idx[b, h, t] >= 0].astype(np.int64)
                    keys = (blocks[:, None] * C + np.arange(C)).reshape(-1)
                    keys = torch.from_numpy(keys[keys <= ln[b] + t]).to(o.device)
                    k = s["Kq"][b, h, keys].double() * s["ks"][b, h, keys].double()[:, None]
                    v = s["Vq"][b, h, keys].double() * s["vs"][b, h, keys].double()[:, None]
                    heads = slice(h * G, (h + 1) * G)
                    o[b, t, heads], lse[b, t, heads] = _attend64(s["q"][b, t, heads].double(), k, v, d)
        return dict(o=o, lse=lse)
    # the last case takes 4 * 256 * 32 * 131072 * 128 = 5.5e11 products: a second or so in 64 bits
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=s["q"].device)
    rows, lens = s["rows"].tolist(), s["len"].tolist()
    for p in range(c["P"]):
        for h in range(c["H_kv"]):
            n = lens[p]
            k, v = s["K"][p, h, :n].double(), s["V"][p, h, :n].double()
            if s["ks"] is not None:
                k, v = k * s["ks"][p, h, :n].double()[:, None], v * s["vs"][p, h, :n].double()[:, None]
            for r0 in range(rows[p], rows[p + 1], 64):
                r1 = min(r0 + 64, rows[p + 1])
                q = s["q"][r0:r1, h * G : (h + 1) * G].double().reshape(-1, d)
                a, b = _attend64(q, k, v, d)
                o[r0:r1, h * G : (h + 1) * G], lse[r0:r1, h * G : (h + 1) * G] = a.reshape(-1, G, d), b.reshape(-1, G)
    if s["o_own"] is not None:
        own_o, own_l = s["o_own"].double(), s["lse_own"].double()
        tot = torch.logaddexp(lse, own_l)
        o = (lse - tot).exp()[..., None] * o + (own_l - tot).exp()[..., None] * own_o
        lse = tot
    return dict(o=o, lse=lse)
