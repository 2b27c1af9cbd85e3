"""Workloads of the serving operators over a paged bf16 key/value cache.

Four operators, each in its plain form (elementary torch operations in 32 bits) and as the library's
call (``own``).  Keys and values lie in pages [P, H_kv, S, d] of S tokens; key c of sequence b is row
c mod S of page page_table[b, c // S].  Sequence b has seq_len[b] keys before its new tokens, whose rows
(of all sequences one after the other) are row_start[b] .. row_start[b + 1] - 1.

  write     put the new tokens' K and V rows into their pages and clear the weights kept beside them
  attn      attention of the new tokens (one, a few, a chunk, a whole prompt) over their sequences' pages:
            token t sees the keys up to its own, seq_len + t
  weights   the attention weight each key has got from the new tokens, summed over them and over the
            query heads that share the key:  w_c = sum exp(scale q . k_c - lse)
  evict     of every sequence and KV head, keep the keys of the largest weights (the first `sinks` and the
            last `recent` always; ties to the lower index) and put them, in their order, into new pages
"""
import math

import torch

own = False


# ---- cases ---------------------------------------------------------------------------------
def listed():
    return [
        # a decode step of 64 sequences puts one token each into its page
        dict(name="write_step", op="write", B=64, T=1, H_kv=8, d=128, S=64, L=4096, ragged=False),
        # a batch of chunks of prompts of different lengths
        dict(name="write_chunks", op="write", B=12, T=4999, H_kv=8, d=128, S=16, L=8000, ragged=True),
        # one short conversation, one token: latency
        dict(name="attn_one", op="attn", B=1, T=1, H_q=16, H_kv=1, d=128, S=64, L=1000, ragged=False),
        # a decode step of 64 sequences of different lengths
        dict(name="attn_step", op="attn", B=64, T=1, H_q=32, H_kv=8, d=128, S=64, L=16384, ragged=True),
        # up to five drafted tokens a sequence, small pages
        dict(name="attn_drafts", op="attn", B=24, T=5, H_q=32, H_kv=4, d=64, S=16, L=9001, ragged=True),
        # one chunk of a long prompt, half of it in the cache
        dict(name="attn_chunk", op="attn", B=1, T=4096, H_q=32, H_kv=8, d=128, S=64, L=28672, ragged=False),
        # whole prompts of different lengths, nothing before them
        dict(name="attn_prompts", op="attn", B=4, T=6001, H_q=16, H_kv=16, d=64, S=128, L=0, ragged=True),
        # the last chunk of a very long prompt
        dict(name="attn_long", op="attn", B=1, T=2048, H_q=32, H_kv=2, d=128, S=256, L=126976, ragged=False),
        # what each key got in a decode step of 64 sequences
        dict(name="weights_step", op="weights", B=64, T=1, H_q=32, H_kv=8, d=128, S=64, L=8192, ragged=True),
        # what each key got from a prompt's last chunk
        dict(name="weights_chunk", op="weights", B=1, T=2048, H_q=32, H_kv=8, d=128, S=64, L=30720, ragged=False),
        # a few small caches cut down
        dict(name="evict_small", op="evict", B=3, H_kv=2, d=64, S=16, L=1000, keep=257, sinks=4, recent=32, ragged=True),
        # eight long prompts cut down to a quarter
        dict(name="evict_prompts", op="evict", B=8, H_kv=8, d=128, S=64, L=32768, keep=8192, sinks=4, recent=512, ragged=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))))


def draw(rng):
    op = rng.choice(["write", "attn", "attn", "weights", "evict"])
    d, S, H_kv = rng.choice([64, 128]), rng.choice([16, 32, 64, 128, 256]), rng.choice([1, 2, 4, 8])
    B = _log(rng, 1, 64)
    ragged = rng.random() < 0.7
    if op == "write":
        T = _log(rng, 1, max(1, 400000 // (B * H_kv)))
        return dict(op=op, B=B, T=T, H_kv=H_kv, d=d, S=S, L=rng.choice([0, _log(rng, 1, 8000)]), ragged=ragged)
    if op == "evict":
        L = _log(rng, 64, min(65536, (1 << 21) // (B * H_kv)))
        keep = _log(rng, 1, L)
        sinks = rng.choice([0, min(4, keep)])
        return dict(op=op, B=B, H_kv=H_kv, d=d, S=S, L=L, keep=keep, sinks=sinks,
                    recent=rng.choice([0, (keep - sinks) // 16]), ragged=ragged)
    G = rng.choice([1, 2, 4, 8, 16])
    T = rng.choice([1, 1, 2, 5, 17, _log(rng, 1, 4096)])
    B = min(B, max(1, 8192 // T))
    # keys a sequence: at most the largest listed cases' products and keys
    most = min((1 << 31) // (B * T * G * H_kv), (1 << 22) // (B * H_kv), 131072)
    L = rng.choice([0, _log(rng, 1, max(1, most - T))]) if T > 5 else _log(rng, 1, max(1, most - T))
    return dict(op=op, B=B, T=T, H_q=G * H_kv, H_kv=H_kv, d=d, S=S, L=L, ragged=ragged)


# ---- inputs --------------------------------------------------------------------------------
def _normal(gen, shape, scale=1.0):
    return torch.empty(shape, dtype=torch.bfloat16, device=gen.device).normal_(0, scale, generator=gen)


def _spread(gen, lo, hi, n):
    """n whole numbers spread over lo .. hi, hi among them, in any order."""
    x = torch.arange(n, device=gen.device, dtype=torch.float64) * 0.6180339887498949
    x = lo + ((hi - lo) * (1 - (x - x.floor()))).int()
    return x[torch.randperm(n, generator=gen, device=gen.device)]


def _tables(gen, n_pages, sizes):
    """Page tables [B, M] of the given sizes, no page twice; entries behind a sequence's last page -1."""
    order = torch.randperm(n_pages, generator=gen, device=gen.device).int()
    tables, at = [], 0
    for counts, M in sizes:
        first = torch.cumsum(counts, 0) - counts + at
        j = torch.arange(M, device=gen.device)
        used = j < counts[:, None]
        tables.append(torch.where(used, order[torch.where(used, first[:, None] + j, 0).long()], -1).int())
        at += int(counts.sum())
    return tables


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    c = dict(case)
    op, B, H, d, S, L = c["op"], c["B"], c["H_kv"], c["d"], c["S"], c["L"]
    dev = gen.device
    s = dict(case=c, op=op)
    T = c.get("T", 0)
    # keys before the new tokens, and new tokens; ragged ones are the same numbers for every seed, in another order
    s["len"], n = (_spread(gen, lo, hi, B) if c["ragged"] else torch.full((B,), hi, dtype=torch.int32, device=dev)
                   for lo, hi in ((L // 2, L), (min(1, T), T)))
    s["rows"], s["R"] = None, int(n.sum())
    if c["ragged"] and T > 1:
        s["rows"] = torch.cat([n[:1] * 0, torch.cumsum(n, 0).int()])
    s["n"] = n
    # pages: those in use, those that an eviction fills, and others
    sizes = [(-(-(s["len"] + n) // S), -(-(L + T) // S))]
    if op == "evict":
        s["keep"], s["sinks"], s["recent"] = c["keep"], c["sinks"], c["recent"]
        sizes.append((-(-torch.clamp(s["len"], max=c["keep"]) // S), -(-c["keep"] // S)))
    P = sum(B * M for _, M in sizes) + 3
    tables = _tables(gen, P, sizes)
    s["table"] = tables[0]
    s["K"], s["V"] = _normal(gen, (P, H, S, d)), _normal(gen, (P, H, S, d))
    if op != "write":
        s["K"] += _normal(gen, (P, H, 1, d), 0.5)  # keys of a page lie together
    if op == "write":
        s["k"], s["v"] = _normal(gen, (s["R"], H, d)), _normal(gen, (s["R"], H, d))
        s["w"] = torch.rand((P, H, S), generator=gen, device=dev)
    elif op == "evict":
        s["new_table"] = tables[1]
        # long-tailed weights; some keys got none
        w = torch.randn((P, H, S), generator=gen, device=dev).mul_(2).exp_()
        s["w"] = torch.where(torch.rand((P, H, S), generator=gen, device=dev) < 0.05, 0.0, w)
        s["new_len"] = torch.zeros(B, dtype=torch.int32, device=dev)
        s["kept"] = torch.full((B, H, c["keep"]), -1, dtype=torch.int32, device=dev)
    else:
        s["q"] = _normal(gen, (s["R"], c["H_q"], d), 1.5)
        if op == "weights":
            s["lse"] = _plain_attn(s)["lse"]
            s["w"] = torch.zeros((P, H, S), device=dev)
    return s


# ---- one pass ------------------------------------------------------------------------------
def _slots(s):
    """Of every new row: its sequence, its key's page and row in the page."""
    R, S, B = s["R"], s["K"].shape[2], s["table"].shape[0]
    r = torch.arange(R, device=s["K"].device)
    if s["rows"] is None:
        b = r // (R // B)
        first = b * (R // B)
    else:
        b = torch.searchsorted(s["rows"][1:].long(), r, right=True)
        first = s["rows"].long()[b]
    at = s["len"].long()[b] + r - first
    return b, r - first, s["table"].long()[b, at // S], at % S


def _plain_write(s):
    _, _, page, at = _slots(s)
    s["K"][page, :, at] = s["k"]
    s["V"][page, :, at] = s["v"]
    s["w"][page, :, at] = 0
    return dict(k=s["K"], v=s["V"], w=s["w"])


def _gather(s, x):
    """The sequences' rows of x [P, H, S, ...] in 32 bits: [B, H, M S, ...]; rows of unused entries hold page 0's."""
    B, M = s["table"].shape
    rows = x[s["table"].clamp(min=0).long()].transpose(1, 2)
    return rows.reshape(B, x.shape[1], M * x.shape[2], *x.shape[3:]).float()


def _logits(s):
    """scale q . k of every sequence's rows, padded to the most of any: [B, H, G, T, keys], unseen keys -inf."""
    H_q, d = s["q"].shape[1:]
    B, H, T = s["table"].shape[0], s["K"].shape[1], s["case"]["T"]
    b, t, _, _ = _slots(s)
    q = s["q"].new_zeros((B, T, H_q, d))
    q[b, t] = s["q"]
    q = q.float().reshape(B, T, H, H_q // H, d).permute(0, 2, 3, 1, 4).reshape(B, H, -1, d)
    z = torch.matmul(q, _gather(s, s["K"]).transpose(-1, -2)).reshape(B, H, H_q // H, T, -1)
    z *= 1.0 / math.sqrt(d)
    last = s["len"][:, None].long() + torch.arange(T, device=z.device)
    unseen = torch.arange(z.shape[-1], device=z.device) > last[..., None]
    return z.masked_fill_(unseen[:, None, None], -math.inf), b, t


def _plain_attn(s):
    z, b, t = _logits(s)
    B, H, G, T, _ = z.shape
    m = z.amax(dim=-1, keepdim=True)
    z = z.sub_(m).exp_()
    l = z.sum(dim=-1)
    lse = (m[..., 0] + torch.log(l)).permute(0, 3, 1, 2).reshape(B, T, H * G)
    v = _gather(s, s["V"])
    o = torch.matmul(z.reshape(B, H, G * T, -1), v).reshape(B, H, G, T, -1) / l[..., None]
    o = o.permute(0, 3, 1, 2, 4).reshape(B, T, H * G, -1)
    return dict(o=o[b, t].to(torch.bfloat16), lse=lse[b, t].contiguous())


def _plain_weights(s):
    z, b, t = _logits(s)
    B, H, G, T, n = z.shape
    lse = torch.full((B, T, H * G), math.inf, device=z.device)  # rows that are not there weigh nothing
    lse[b, t] = s["lse"]
    z = z.sub_(lse.reshape(B, T, H, G).permute(0, 2, 3, 1)[..., None]).exp_()
    total = z.sum(dim=(2, 3))
    S = s["K"].shape[2]
    c = torch.arange(n, device=z.device).expand(B, n)
    live = c < (s["len"] + s["n"])[:, None]
    page = torch.gather(s["table"].long(), 1, c // S)[live]
    s["w"][page, :, (c % S)[live]] = total.transpose(1, 2)[live]
    return dict(w=s["w"])


def _plain_evict(s):
    B, H, keep = s["kept"].shape
    S, n = s["K"].shape[2], s["len"].long()
    w = _gather(s, s["w"])
    c = torch.arange(w.shape[-1], device=w.device)
    w = torch.where((c < s["sinks"]) | (c >= (n - s["recent"])[:, None])[:, None], math.inf, w)
    w = torch.where((c < n[:, None])[:, None], w, -1.0)
    best = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :keep]  # ties: the lower index first
    new_len = torch.clamp(n, max=keep)
    j = torch.arange(keep, device=w.device)
    live = (j < new_len[:, None])[:, None].expand(B, H, keep)[..., : best.shape[-1]]
    src = torch.where(live, best, w.shape[-1]).sort(dim=-1).values
    s["kept"].fill_(-1)
    s["kept"][..., : best.shape[-1]] = torch.where(live, src, -1).int()
    b, h, j = live.nonzero(as_tuple=True)
    src = src[b, h, j]
    page, to = s["table"].long()[b, src // S], s["new_table"].long()[b, j // S]
    for x in (s["K"], s["V"], s["w"]):
        x[to, h, j % S] = x[page, h, src % S]
    s["new_len"].copy_(new_len)
    return dict(k=s["K"], v=s["V"], w=s["w"], kept=s["kept"], n=s["new_len"])


def run(state):
    s = state
    if own:
        import hierarchical_top_block_gb300 as pisa

        if s["op"] == "write":
            pisa.pisa_paged_write(s["k"], s["v"], s["K"], s["V"], s["table"], s["len"], row_start=s["rows"], w=s["w"])
            return dict(k=s["K"], v=s["V"], w=s["w"])
        if s["op"] == "attn":
            o, lse = pisa.pisa_paged_attn(s["q"], s["K"], s["V"], s["table"], s["len"], row_start=s["rows"])
            return dict(o=o, lse=lse)
        if s["op"] == "weights":
            pisa.pisa_paged_weights(s["q"], s["lse"], s["K"], s["w"], s["table"], s["len"], row_start=s["rows"],
                                    accumulate=False)
            return dict(w=s["w"])
        pisa.pisa_paged_evict(s["K"], s["V"], s["w"], s["table"], s["len"], s["new_table"], s["keep"], sinks=s["sinks"],
                              recent=s["recent"], new_len=s["new_len"], kept=s["kept"])
        return dict(k=s["K"], v=s["V"], w=s["w"], kept=s["kept"], n=s["new_len"])
    return {"write": _plain_write, "attn": _plain_attn, "weights": _plain_weights, "evict": _plain_evict}[s["op"]](s)


# ---- the work a pass cannot do without -------------------------------------------------------
def work(case):
    c, B, H, d, L = case, case["B"], case["H_kv"], case["d"], case["L"]
    # ragged: all sequences but one have on average three quarters of the keys and half of the new tokens
    odd = (B - 1) if c["ragged"] else 0
    T = c.get("T", 0)
    keys, rows = (B - odd) * L + odd * 0.75 * L, (B - odd) * T + odd * (0.5 * (T + 1))
    if c["op"] == "write":
        return dict(bytes=rows * H * (8 * d + 4), flops=0)
    if c["op"] == "evict":
        kept = (B - odd) * min(L, c["keep"]) + odd * min(0.75 * L, c["keep"])
        return dict(bytes=H * (4 * keys + kept * (8 * d + 8)), flops=H * keys)
    G = c["H_q"] // H
    pairs = c["H_q"] * ((B - odd) * T * (L + 0.5 * (T + 1)) + odd * 0.5 * (T + 1) * (0.75 * L + 0.3 * (T + 1)))
    if c["op"] == "attn":
        return dict(bytes=(keys + rows) * H * 4 * d + rows * H * G * (4 * d + 4), flops=pairs * 4 * d)
    return dict(bytes=(keys + rows) * H * (2 * d + 4) + rows * H * G * (2 * d + 4), flops=pairs * 2 * d)


# ---- the definition in 64 bits ---------------------------------------------------------------
def exact(case, seed):
    c, s = case, prepare(case, seed)
    op, B, H, S, d = c["op"], c["B"], c["H_kv"], c["S"], c["d"]
    lens, table = s["len"].tolist(), s["table"]
    if op == "write":
        return None  # rows are moved, not computed
    if op == "evict":
        w, kept = s["w"].double(), torch.full(s["kept"].shape, -1, dtype=torch.int64, device=table.device)
        for b in range(B):
            n = lens[b]
            old = torch.arange(n, device=table.device)
            for h in range(H):
                mine = s["w"][table[b, old // S].long(), h, old % S].double()
                score = mine.clone()
                score[: c["sinks"]] = math.inf
                score[max(0, n - c["recent"]):] = math.inf
                if n > c["keep"]:
                    edge = score.sort().values[n - c["keep"]]
                    sure = score > edge
                    tied = (score == edge) & ((score == edge).cumsum(0) <= c["keep"] - int(sure.sum()))
                    idx = old[sure | tied]
                else:
                    idx = old
                new = torch.arange(len(idx), device=idx.device)
                kept[b, h, : len(idx)] = idx
                w[s["new_table"][b, new // S].long(), h, new % S] = mine[idx]
        return dict(k=None, v=None, w=w, kept=kept, n=torch.clamp(s["len"].long(), max=c["keep"]))
    if work(case)["flops"] > 8e12:
        return None
    G = c["H_q"] // H
    first = s["rows"].tolist() if s["rows"] is not None else [b * c["T"] for b in range(B + 1)]
    if op == "attn":
        o = torch.zeros(s["q"].shape, dtype=torch.float64, device=table.device)
        lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=table.device)
    else:
        w = s["w"].double()
    for b in range(B):
        n = first[b + 1] - first[b]
        total = lens[b] + n
        c_all = torch.arange(total, device=table.device)
        page, at = table[b, c_all // S].long(), c_all % S
        for h in range(H):
            k, v = s["K"][page, h, at].double(), s["V"][page, h, at].double()
            sums = torch.zeros(total, dtype=torch.float64, device=k.device)
            step = max(1, (1 << 27) // (G * total))
            for t0 in range(0, n, step):
                t1 = min(t0 + step, n)
                rows, heads = slice(first[b] + t0, first[b] + t1), slice(h * G, (h + 1) * G)
                e = lens[b] + t1  # no row of these sees further
                x = torch.einsum("tgd,cd->tgc", s["q"][rows, heads].double(), k[:e]) / math.sqrt(d)
                see = c_all[:e] <= lens[b] + torch.arange(t0, t1, device=k.device)[:, None]
                x = x.masked_fill(~see[:, None], -math.inf)
                if op == "attn":
                    lse[rows, heads] = torch.logsumexp(x, -1)
                    o[rows, heads] = torch.einsum("tgc,cd->tgd", torch.softmax(x, -1), v[:e])
                else:
                    sums[:e] += (x - s["lse"][rows, heads].double()[..., None]).exp().sum((0, 1))
            if op == "weights":
                w[page, h, at] = sums
    return dict(o=o, lse=lse) if op == "attn" else dict(w=w)
