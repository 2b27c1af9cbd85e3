"""How many bits of an attention weight the paged attention keeps.

With few query rows a weight is multiplied with its value as two bf16 operands, and 2^-17 of it is lost (bf16 keeps 8 bits: half a
step is 2^-8; what is left of a weight is at most 2^-8 of it and is rounded to 8 bits of its own, where half a step is 2^-17 of
the weight).  With many rows it is one operand: 2^-8.  Errors of one sign show this: values that have the sign of what the first rounding
does to their weight, so that a kernel that leaves the second operand out is off by the mean of |rounding|, about 2^-9.5, while the
output itself, whose rounding to bf16 would hide that, is near 0.

The bound, relative to sum w |v|:  the weight's own loss;  4 E for the logits (E of cache_helpers);  2^-16 for exp2 and the
factors;  F 2.4 n + 64 F for the sums of n weights and n products (each truncated, in two operands).  And U |o| for the output."""
import math

import pytest
import torch

import cache_helpers as R

TWO, ONE = 2.0 ** -17, R.U


def signed_case(n, d, heads, dev, seed):
    """q [heads, d], k and v [n, d], bf16: logits from 0 down (the key 0 has none above), values of the sign of the
    first head's rounding."""
    g = torch.Generator(device="cpu").manual_seed(seed)
    q, k = torch.zeros(heads, d), torch.zeros(n, d)
    q[:, 0] = 1 + 0.25 * torch.arange(heads)
    k[1:, 0] = -(torch.rand(n - 1, generator=g) * 4 * math.sqrt(d)).to(torch.bfloat16).float()
    p = torch.exp(k[:, 0].double() / math.sqrt(d))
    off = p.to(torch.float32).to(torch.bfloat16).double() / p - 1
    v = torch.where(off >= 0, 1.0, -1.0) * (0.5 + 0.5 * torch.rand(n, generator=g))
    v = v[:, None] * torch.ones(d)
    v[:, 1::2] *= -1
    # the heavier sign is made lighter, so that the outputs are near 0
    up, down = (p * v[:, 0])[v[:, 0] > 0].sum(), -(p * v[:, 0])[v[:, 0] < 0].sum()
    v[v[:, 0] > 0] *= min(1.0, float(down / up))
    v[v[:, 0] < 0] *= min(1.0, float(up / down))
    return [x.to(torch.bfloat16).to(dev) for x in (q, k, v)]


def bound(q, k, v, weight):
    """o and lse of rows that see every key, and the bound of o."""
    n, d = k.shape
    o, lse, _, bl = R.attend64(q, k, v)
    z = q @ k.T / math.sqrt(d)
    e = (d + 8) * R.F * (q.abs() @ k.abs().T).amax(1, keepdim=True) / math.sqrt(d)
    w = torch.softmax(z, -1)
    return o, lse, (weight + 4 * e + 2.0 ** -16 + R.F * (2.4 * n + 64)) * (w @ v.abs()) + R.U * o.abs(), bl


@pytest.mark.parametrize("n,d", [(60, 64), (250, 128), (600, 64), (600, 128)])
def test_bound_tells_one_operand_from_two(n, d):
    """The planted mistake: weights of one operand are outside the bound of two, inside that of one."""
    q, k, v = (x.double() for x in signed_case(n, d, 1, "cpu", n + d))
    o, _, two, _ = bound(q, k, v, TWO)
    one = bound(q, k, v, ONE)[2]
    p = torch.exp(q @ k.T / math.sqrt(d)).float()
    first = p.to(torch.bfloat16)
    second = (p - first.float()).to(torch.bfloat16)
    l = p.double().sum(1, keepdim=True)

    def off(w):
        return ((w @ v) / l).to(torch.bfloat16).double().sub(o).abs()

    assert (off(first.double() + second.double()) <= two).all()
    assert (off(first.double()) > 2 * two).all() and (off(first.double()) <= one).all()


@pytest.mark.gpu
@pytest.mark.parametrize("d,S", [(64, 16), (64, 64), (128, 16), (128, 64)])
@pytest.mark.parametrize("G,T", [(1, 1), (1, 8), (4, 1), (4, 3), (8, 2), (16, 1), (4, 5), (8, 16), (16, 10), (16, 20)])
@pytest.mark.parametrize("n", [60, 250, 600])
def test_bits_of_a_weight(d, S, G, T, n):
    """Up to 16 rows a sequence keep 2^-17 of a weight, more 2^-8; the last token's rows are looked at, which see every key."""
    import hierarchical_top_block_gb300 as pisa
    from paged_helpers import DEV, Paged

    H_kv = 2
    c = Paged([n - T, n - T], [T, T], H_kv, d, S, seed=n)
    q = c.rand(c.R, H_kv * G, d, scale=0.1)
    for b in range(2):
        k, v = torch.zeros(n, H_kv, d, device=DEV), torch.zeros(n, H_kv, d, device=DEV)
        for h in range(H_kv):
            qs, k[:, h], v[:, h] = signed_case(n, d, G, DEV, n + d + 2 * b + h)
            q[c.first[b + 1] - 1, h * G:(h + 1) * G] = qs
        c.put(b, k.to(torch.bfloat16), v.to(torch.bfloat16))
    o, lse = pisa.pisa_paged_attn(q, c.K, c.V, c.table, c.len, row_start=c.rows)
    for b in range(2):
        for h in range(H_kv):
            r, heads = c.first[b + 1] - 1, slice(h * G, (h + 1) * G)
            k, v = (c.get(x, b, n)[:, h].double() for x in (c.K, c.V))
            want, wl, most, bl = bound(q[r, heads].double(), k, v, TWO if T * G <= 16 else ONE)
            R.close(o[r, heads], want, most, "o")
            R.close(lse[r, heads], wl, bl, "lse")
    assert pisa.pisa_get_last_device_error() == 0
