"""Plain 64-bit forms of the 8-bit cache's operators and of the attention over a shared prefix, with
the error each result may have.

The error bounds count roundings (U = half a step of bf16, 2^-8 relative; F = a step of fp32, 2^-23,
a truncating sum's error a term):
  logit   d products summed in fp32, then three fp32 factors:  E = (d + 8) F max_c scale |q| . |k_c|
  lse     an average of the logits' errors, exp2 / log2 and the sums: 2 E + 2^-18 + 2^-22 |lse|
  o       each weight is off by 2 E (its logit, the sum) and rounded to bf16 once (U), the result is
          rounded to bf16 (U):  (U + 4 E + 2^-16) sum_c w_c |v_c| + U |o|, w the softmax weights
  o, codes   the weight times its value's scale vs_c is held in fp16: 2^-12 of it, within U, or where it is
          below fp16's normal range half a step there, 2^-25, of numbers p_c vs_c with p_c = w_c l.  The
          reference n of p_c = 2^(z_c - n) is at most z_top + log2(2 vs_max), so p_top >= 1 / (2 vs_max)
          and l = p_top / w_top >= 1 / (2 vs_max w_top): 2^-25 of p_c vs_c is at most 2^-24 vs_max w_top of
          w_c vs_c.  No error exceeds the weight itself (rounded to 0):
          + sum_c min(2^-24 w_top vs_max / vs_c, w_c) |v_c|
"""
import math

import torch

U = 2.0 ** -8
F = 2.0 ** -23


def quantise64(x):
    """bf16 rows -> (codes int8, fp32 scales, bf16 values), from the definition in 64 bits."""
    x = x.double()
    a = x.abs().amax(-1)
    bad = ~torch.isfinite(a)
    safe = torch.where((a > 0) & ~bad, a, torch.ones_like(a))
    u = torch.floor(127 * x.abs() / safe[..., None] + 0.5)
    code = torch.where(x < 0, -u, u)
    code[bad] = 0
    scale = (a / 127).float()
    scale[bad] = math.nan
    # code * scale is rounded to fp32, then to bf16, as documented
    return code.to(torch.int8), scale, (code.float() * scale[..., None]).to(torch.bfloat16)


def attend64(q, k, v, scale=None, vs=None):
    """q [r, d], k and v [n, d] in float64 -> o [r, d], lse [r], and the bounds on both.  vs [n]: the scales of the
    values, where they are codes."""
    d = q.shape[-1]
    scale = 1 / math.sqrt(d) if scale is None else scale
    if k.shape[0] == 0:
        z = q.new_zeros(q.shape[0])
        return q.new_zeros(q.shape), z - math.inf, q.new_zeros(q.shape), z
    z = scale * q @ k.T
    e = (d + 8) * F * scale * (q.abs() @ k.abs().T).amax(1)
    m = z.amax(1, keepdim=True)
    w = torch.exp(z - m)
    l = w.sum(1, keepdim=True)
    w = w / l
    o, lse = w @ v, (m + l.log())[:, 0]
    floor = 0.0
    if vs is not None:
        ratio = vs.max() / vs.clamp(min=1e-300)
        floor = torch.minimum(2.0 ** -24 * w.amax(1, keepdim=True) * ratio, w) @ v.abs()
    return o, lse, (U + 4 * e[:, None] + 2.0 ** -16) * (w @ v.abs()) + U * o.abs() + floor, 2 * e + 2.0 ** -18 + 2.0 ** -22 * lse.abs()


def join64(o, lse, to, tl, o_own, lse_own):
    """The joined result of a prefix part and an own part, with its bounds."""
    tot = torch.logaddexp(lse, lse_own)
    none = torch.isinf(tot)
    a = torch.where(none, 0.0, torch.exp(lse - tot))[:, None]
    b = torch.where(none, 0.0, torch.exp(lse_own - tot))[:, None]
    own = torch.where(b > 0, o_own, torch.zeros_like(o_own))
    joined = a * o + b * own
    # the part's own bound holds a rounding of its result; the joined result has that rounding instead.
    # the two factors are off by the error of the lse and of exp2 (2^-18)
    e = (tl + 2.0 ** -18)[:, None]
    bound = a * to + e * (a * o.abs() + b * own.abs()) + U * joined.abs()
    return joined, tot, bound, tl + 2.0 ** -18 + 2.0 ** -22 * torch.where(none, torch.zeros_like(tot), tot).abs()


def close(got, want, bound, what):
    got, want, bound = got.double().cpu(), want.double().cpu(), bound.double().cpu()
    fin = torch.isfinite(want)
    assert torch.equal(got[~fin].nan_to_num(7), want[~fin].nan_to_num(7)), f"{what}: not finite where the definition is"
    err = (got - want).abs()[fin]
    over = err - bound[fin]
    assert not err.isnan().any() and (over <= 1e-30).all(), \
        f"{what}: off by {float(err.max()):.3g}, {float((err / bound[fin].clamp(min=1e-30)).max()):.2f} of its bound"
