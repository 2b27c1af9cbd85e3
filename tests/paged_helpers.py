"""Plain 64-bit forms of the paged cache's operators, with the error each result may have.

The attention's bounds are those of cache_helpers.attend64.  The weight of a key is a sum of n terms p = exp(z - lse)
that one row and head give each:
  z       off by E = (d + 8) 2^-23 scale |q| . |k| at most (d products summed in fp32, truncating)
  z - lse in log2 units: two factors and two products of half a step each, 2^-22 (|z| + |lse|) in all
  exp2    2^-22 of the term
  the sum n terms added one after the other at worst, n 2^-24 of the sum of them; joining parts, 2^-22
"""
import math

import torch

import cache_helpers as R

DEV = "cuda"


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Paged:
    """Sequences with lens[b] keys before their new[b] new tokens, in pages of S tokens in any order; rows of the pool
    that belong to nobody hold NaN."""

    def __init__(self, lens, new, H_kv, d, S, seed=0, M=None, spare=3, fill=math.nan, gap=0):
        g = self.g = torch.Generator(device=DEV).manual_seed(seed)
        self.lens, self.new, self.H_kv, self.d, self.S, self.B = list(lens), list(new), H_kv, d, S, len(lens)
        need = [-(-(a + b) // S) for a, b in zip(lens, new)]
        self.M = max(need + [1]) + 1 if M is None else M
        self.P = sum(need) + spare
        order = torch.randperm(self.P, generator=g, device=DEV).int()
        self.table = torch.full((self.B, self.M), self.P + 7, dtype=torch.int32, device=DEV)  # not read behind the last key
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.spare = order[at:]
        self.K = torch.full((self.P, H_kv, S, d), fill, dtype=torch.bfloat16, device=DEV)
        self.V = torch.full_like(self.K, fill)
        self.w = torch.full((self.P, H_kv, S), -7.0, device=DEV)
        self.len = i32(*lens)
        # `gap` rows before the first sequence's and behind the last's
        first = [gap]
        for n in new:
            first.append(first[-1] + n)
        self.first, self.R = first, first[-1] + gap
        self.rows = i32(*first)
        for b in range(self.B):
            n = lens[b] + new[b]
            if n:
                self.put(b, self.rand(n, H_kv, d), self.rand(n, H_kv, d))

    def rand(self, *shape, scale=1.0):
        return (torch.randn(shape, generator=self.g, device=DEV) * scale).to(torch.bfloat16)

    def at(self, b, n):
        c = torch.arange(n, device=DEV)
        return self.table[b, c // self.S].long(), c % self.S

    def put(self, b, k, v):
        page, row = self.at(b, k.shape[0])
        self.K[page, :, row], self.V[page, :, row] = k, v

    def get(self, x, b, n):
        """Rows 0 .. n - 1 of sequence b: [n, H_kv, ...]."""
        page, row = self.at(b, n)
        return x[page, :, row]


def attend(c, q, causal=True, scale=None, gone=()):
    """o, lse and their bounds, rows of no sequence NaN.  gone: (sequence, table entry) pairs that name no page."""
    H_q, d = q.shape[1:]
    G = H_q // c.H_kv
    o = torch.full(q.shape, math.nan, dtype=torch.float64, device=DEV)
    lse = torch.full(q.shape[:2], math.nan, dtype=torch.float64, device=DEV)
    bo, bl = o.clone(), lse.clone()
    for b in range(c.B):
        n = c.lens[b] + c.new[b]
        if n == 0:
            continue
        k, v = c.get(c.K, b, n).double(), c.get(c.V, b, n).double()
        there = torch.tensor([(b, i // c.S) not in gone for i in range(n)], device=DEV)
        for t in range(c.new[b]):
            e = c.lens[b] + t + 1 if causal else n
            see = there[:e].nonzero()[:, 0]
            for h in range(c.H_kv):
                r, heads = c.first[b] + t, slice(h * G, (h + 1) * G)
                o[r, heads], lse[r, heads], bo[r, heads], bl[r, heads] = R.attend64(q[r, heads].double(), k[see, h], v[see, h], scale)
    return o, lse, bo, bl


def attend_many(c, q):
    """attend's o, lse and bounds of causal rows, whole sequences at a time."""
    H_q, d = q.shape[1:]
    G, scale = H_q // c.H_kv, 1 / math.sqrt(d)
    o = torch.full(q.shape, math.nan, dtype=torch.float64, device=DEV)
    lse = torch.full(q.shape[:2], math.nan, dtype=torch.float64, device=DEV)
    bo, bl = o.clone(), lse.clone()
    for b in range(c.B):
        n, T = c.lens[b] + c.new[b], c.new[b]
        if T == 0:
            continue
        rows = slice(c.first[b], c.first[b] + T)
        k, v = (c.get(x, b, n).double().transpose(0, 1) for x in (c.K, c.V))  # [H, n, d]
        x = q[rows].double().reshape(T, c.H_kv, G, d).permute(1, 2, 0, 3)     # [H, G, T, d]
        z = scale * torch.einsum("hgtd,hcd->hgtc", x, k)
        see = torch.arange(n, device=DEV) <= c.lens[b] + torch.arange(T, device=DEV)[:, None]
        e = (d + 8) * R.F * scale * torch.einsum("hgtd,hcd->hgtc", x.abs(), k.abs()).masked_fill(~see, 0).amax(-1)
        z = z.masked_fill(~see, -math.inf)
        l = torch.logsumexp(z, -1)
        w = torch.exp(z - l[..., None])
        y, va = torch.einsum("hgtc,hcd->hgtd", w, v), torch.einsum("hgtc,hcd->hgtd", w, v.abs())
        flat = lambda t: t.permute(2, 0, 1, *range(3, t.dim())).reshape(T, H_q, *t.shape[3:])  # noqa: E731
        o[rows], lse[rows] = flat(y), flat(l)
        bo[rows] = flat((R.U + 4 * e[..., None] + 2.0 ** -16) * va + R.U * y.abs())
        bl[rows] = flat(2 * e + 2.0 ** -18 + 2.0 ** -22 * l.abs())
    return o, lse, bo, bl


def weights(c, q, lse, causal=True, scale=None, gone=()):
    """What the rows give to each key, and the bound: [P, H_kv, S], NaN where a key belongs to nobody (or is gone)."""
    H_q, d = q.shape[1:]
    G, scale = H_q // c.H_kv, 1 / math.sqrt(d) if scale is None else scale
    out = torch.full(c.w.shape, math.nan, dtype=torch.float64, device=DEV)
    bound = out.clone()
    for b in range(c.B):
        n, T = c.lens[b] + c.new[b], c.new[b]
        if n == 0:
            continue
        page, row = c.at(b, n)
        keep = torch.tensor([(b, i // c.S) not in gone for i in range(n)], device=DEV)
        rows = slice(c.first[b], c.first[b] + T)
        see = torch.arange(n, device=DEV) <= c.lens[b] + torch.arange(T, device=DEV)[:, None]
        if not causal:
            see = torch.ones_like(see)
        for h in range(c.H_kv):
            k = c.get(c.K, b, n)[:, h].double()
            x = q[rows, h * G:(h + 1) * G].double()
            l = lse[rows, h * G:(h + 1) * G].double()[..., None]
            z = scale * torch.einsum("tgd,cd->tgc", x, k)
            e = (d + 8) * R.F * scale * torch.einsum("tgd,cd->tgc", x.abs(), k.abs()) + 2.0 ** -22 * (z.abs() + l.abs()) + 2.0 ** -22
            p = torch.where(see[:, None] & (l > -math.inf), torch.exp(z - l), torch.zeros_like(z))
            p = torch.where(p.isnan() & ~see[:, None], torch.zeros_like(p), p)
            w = p.sum((0, 1))
            out[page[keep], h, row[keep]] = w[keep]
            bound[page[keep], h, row[keep]] = ((p * e.nan_to_num(0)).sum((0, 1)) + (T * G * 2.0 ** -24 + 2.0 ** -22) * w)[keep]
    return out, bound


def evict(c, w, n, keep, sinks, recent, gone=()):
    """The kept keys of each sequence and head: lists of indices, ascending."""
    out = []
    for b in range(c.B):
        page, row = c.at(b, n[b])
        for h in range(c.H_kv):
            x = w[page, h, row].double().cpu().tolist()
            rank = []
            for i, v in enumerate(x):
                if (b, i // c.S) in gone:
                    continue
                stays = i < sinks or i >= n[b] - recent
                rank.append((0 if stays else 1, 1 if v != v else 0, 0.0 if v != v else -v, i))
            out.append(sorted(i for *_, i in sorted(rank)[:keep]))
    return out
