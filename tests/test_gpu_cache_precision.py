"""What the attention over the 8-bit cache promises of its roundings, each at the size at which it shows: weights
in fp16 (2^-11 of each), the least weight that is not lost (2^-32 of the largest weight times value scale), sums
over many keys.

Bounds: U = 2^-8 is half a step of bf16, F = 2^-23.  With e the error of a logit (d products summed in fp32, and
three factors), w the softmax weights, vs the value scales and c the codes, o is off by at most
  (2^-11 + 4 e + 2^-16) sum w |v|     a weight's rounding to fp16, its logit and the sum's, exp2
  + sum min(2^-32 W, w vs) |c|        the least weight; W = max w max(vs, 2^-87)
  + 2 s sum w |v| + U |o|             the sums; the result's rounding
where s = N 2^-27: of N weights a lane adds N / 8 at most, a half step (2^-24) each, and the products are added up
16 keys at a time, a step each.  The log-sum-exp is off by s, 2 e and its own rounding.
"""
import math

import pytest
import torch

import cache_helpers as R
import hierarchical_top_block_gb300 as pisa

pytestmark = pytest.mark.gpu
DEV = "cuda"
# query rows of 4 heads that take each kernel: 8 and 16 rows on mma.sync, one and two streams' rows on tcgen05
ROWS = [2, 6, 20, 50]


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(torch.bfloat16)


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def no_error():
    assert pisa.pisa_get_last_device_error() == 0


def attend(q, kc, ks, vc, vs):
    """q [r, d], codes [n, d], scales [n] -> o, lse in 64 bits and the bounds on both."""
    q, kc, ks, vc, vs = (x.double() for x in (q, kc, ks, vc, vs))
    d = q.shape[1]
    scale = 1 / math.sqrt(d)
    z = scale * (q @ kc.T) * ks
    e = (d + 8) * R.F * scale * ((q.abs() @ kc.abs().T) * ks.abs()).amax(1)
    m = z.amax(1, keepdim=True)
    w = torch.exp(z - m)
    l = w.sum(1, keepdim=True)
    w = w / l
    wv = w * vs
    o, mag = wv @ vc, wv.abs() @ vc.abs()
    top = (w * vs.abs().clamp(min=2.0 ** -87)).amax(1, keepdim=True)
    least = torch.minimum(2.0 ** -32 * top, wv.abs()) @ vc.abs()
    lse, s = (m + l.log())[:, 0], kc.shape[0] * 2.0 ** -27
    bound = (2.0 ** -11 + 4 * e[:, None] + 2.0 ** -16 + 2 * s) * mag + least + R.U * o.abs()
    return o, lse, bound, 2 * e + s + 2.0 ** -18 + 2.0 ** -22 * lse.abs()


def both(q, kc, ks, vc, vs):
    """[R, 4, d] queries over one KV head's codes [n, d]: the prefix's answer and the definition's."""
    n, d = kc.shape
    o, lse = pisa.pisa_prefix_attn(q, kc[None, None], vc[None, None], i32(n), k_scale=ks[None, None], v_scale=vs[None, None])
    want, l, to, tl = attend(q.reshape(-1, d), kc, ks, vc, vs)
    return o.reshape(-1, d), lse.reshape(-1), want, l, to, tl


def dominant(N, at, value, d=64):
    """A key 17.5 nats above N - 1 equal ones of value +-1; its own values are `value` and 0 in turn."""
    kc, vc = (torch.zeros((N, d), dtype=torch.int8, device=DEV) for _ in range(2))
    ks, vs = (torch.full((N,), 1 / 127, device=DEV) for _ in range(2))
    vc[:] = 127
    vc[:, 1::4] = -127
    kc[at] = 127
    ks[at] = 17.5 * math.sqrt(d) / (127 * d)
    vc[at], vc[at, 1::2] = 127, 0
    vs[at] = value / 127
    if value == 0:
        vc[at] = 0
    return kc, ks, vc, vs


@pytest.mark.parametrize("value", [1.0, 0.01, 0.0])
@pytest.mark.parametrize("Rn,H_q,H,N", [
    *((r, 4, 1, 131072) for r in ROWS),
    # as many jobs as blocks and more: a block takes all keys of a job
    (2, 608, 608, 32768), (12, 304, 304, 32768), (40, 152, 152, 65536), (2432, 16, 1, 131072)])
@pytest.mark.parametrize("middle", [False, True])
def test_many_keys_under_a_dominant_one(middle, Rn, H_q, H, N, value):
    """The many lie near fp16's least number below the one, and are as much as the one or more in some columns."""
    d = 64
    kc, ks, vc, vs = dominant(N, N // 2 + 4321 if middle else 0, value)
    q = torch.ones((Rn, H_q, d), dtype=torch.bfloat16, device=DEV)
    Kp, Vp = (x.expand(1, H, N, d).contiguous() for x in (kc, vc))
    sk, sv = (x.expand(1, H, N).contiguous() for x in (ks, vs))
    o, lse = pisa.pisa_prefix_attn(q, Kp, Vp, i32(N), k_scale=sk, v_scale=sv)
    want, l, to, tl = attend(q[0, :1], kc, ks, vc, vs)  # (all rows are alike)
    R.close(lse, l.expand(Rn, H_q), tl.expand(Rn, H_q), "lse")
    R.close(o, want.expand(Rn, H_q, d), to.expand(Rn, H_q, d), "o")
    no_error()


@pytest.mark.parametrize("value", [1.0, 0.01, 0.0])
@pytest.mark.parametrize("H_q", [4, 16])
def test_selected_keys_under_a_dominant_one(H_q, value):
    N, d, K = 2048, 64, 32
    kc, ks, vc, vs = dominant(N, 77, value)
    q = torch.ones((1, H_q, d), dtype=torch.bfloat16, device=DEV)
    idx = torch.arange(K, dtype=torch.int32, device=DEV).reshape(1, 1, K)
    O, L = pisa.pisa_sparse_attn_cache(q, kc[None, None], vc[None, None], ks[None, None], vs[None, None], idx, i32(N - 1))
    o, l, to, tl = attend(q[0], kc, ks, vc, vs)
    R.close(L[0], l, tl, "LSE")
    R.close(O[0], o, to, "O")
    no_error()


@pytest.mark.parametrize("N", [2, 3, 5, 17, 100, 700])
@pytest.mark.parametrize("Rn", ROWS)
@pytest.mark.parametrize("d", [64, 128])
def test_weights_of_few_keys(d, Rn, N):
    """Few keys: a weight's rounding is not averaged away, and values of both signs leave it in the result."""
    g = gen(N + Rn + d)
    kc, ks, _ = R.quantise64(normal(g, N, d))
    vc, vs, _ = R.quantise64(normal(g, N, d))
    o, lse, want, l, to, tl = both(normal(g, Rn, 4, d, scale=1.5), kc, ks, vc, vs)
    R.close(lse, l, tl, "lse")
    R.close(o, want, to, "o")
    no_error()


@pytest.mark.parametrize("N", [2, 3, 5, 17, 100, 700])
@pytest.mark.parametrize("H_q", [4, 16])
@pytest.mark.parametrize("d", [64, 128])
def test_weights_of_few_selected_keys(d, H_q, N):
    g = gen(N + H_q + d)
    kc, ks, _ = R.quantise64(normal(g, N, d))
    vc, vs, _ = R.quantise64(normal(g, N, d))
    q = normal(g, 1, H_q, d, scale=1.5)
    K = -(-N // 64)
    idx = torch.arange(K, dtype=torch.int32, device=DEV).reshape(1, 1, K)
    O, L = pisa.pisa_sparse_attn_cache(q, kc[None, None], vc[None, None], ks[None, None], vs[None, None], idx, i32(N - 1))
    o, l, to, tl = attend(q[0], kc, ks, vc, vs)
    R.close(L[0], l, tl, "LSE")
    R.close(O[0], o, to, "O")
    no_error()


@pytest.mark.parametrize("Rn", ROWS)
def test_values_of_zero_over_many_keys(Rn):
    """Weights are large where value scales are small (or 0): their sum over 2^22 keys is no infinity."""
    N, d = (1 << 22) + 3, 64
    c = torch.zeros((1, 1, N, d), dtype=torch.int8, device=DEV)
    s = torch.zeros((1, 1, N), device=DEV)
    q = normal(gen(5), Rn, 4, d)
    o, lse = pisa.pisa_prefix_attn(q, c, c, i32(N), k_scale=s, v_scale=s)
    assert (o == 0).all()
    # equal weights, powers of two: the sum of fewer than 2^24 of them is exact.  It is below 2^128, its logarithm a
    # number below 128 whose last place is 2^-17: that place once, and a rounding of the result
    want = math.log(N)
    assert (lse.double() - want).abs().max() <= 2.0 ** -17 + 2.0 ** -24 * want
    no_error()


@pytest.mark.parametrize("e", [-60, -87, -95, -105, -115])
@pytest.mark.parametrize("Rn", ROWS)
def test_tiny_values(Rn, e):
    """Value scales down to where they are less than the least that the reference follows."""
    N, d = 300, 64
    g = gen(Rn)
    kc, ks, _ = R.quantise64(normal(g, N, d))
    vc, vs, _ = R.quantise64(normal(g, N, d))
    vs *= 2.0 ** e
    o, lse, want, l, to, tl = both(normal(g, Rn, 4, d, scale=1.5), kc, ks, vc, vs)
    R.close(lse, l, tl + 2.0 ** -17, "lse")  # a logarithm of a sum up to 2^127: its last place
    up = 2.0 ** -e
    # the output itself is a normal bf16 number or off by half of bf16's least, 2^-134
    R.close(o.double() * up, want * up, (to + 2.0 ** -134) * up, "o")
    no_error()
