"""Refusals of the 8-bit cache's and the prefix attention's entry points: no GPU is touched."""
import math

import pytest
import torch

import hierarchical_top_block_gb300 as pisa

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 6
A = 0x1000  # an aligned address that nothing reads: every call made with it is refused


def shape(**kw):
    s = dict(B=1, N=2, H_q=4, H_kv=2, d=64, N_cap=128)
    s.update(kw)
    return pisa.make_shape(**s)


def par(**kw):
    p = dict(K=4)
    p.update(kw)
    return pisa.make_params(**p)


CALLS = {  # arguments before the shape, which of them may be NULL, whether parameters follow
    "pisa_cache_write": (10, {7, 8, 9}, False),
    "pisa_cache_read": (8, {0, 1, 2, 3, 4, 5, 6, 7}, False),
    "pisa_sparse_attn_cache": (10, {7, 9}, True),
    "pisa_prefix_attn": (13, {6, 10}, True),
}


def call(name, args, s, p):
    fn = getattr(pisa.lib(), name)
    return fn(*args, s, p, None) if CALLS[name][2] else fn(*args, s, None)


def params(name, **kw):
    return par(causal=name != "pisa_prefix_attn", **kw)


def args(name):
    a = [A + 0x1000 * i for i in range(CALLS[name][0])]
    if name == "pisa_prefix_attn":
        a[12] = 1 << 40  # ws_bytes
    return a


@pytest.mark.parametrize("name", CALLS)
def test_nothing_to_do(name):
    none = [None] * CALLS[name][0]
    if name == "pisa_prefix_attn":
        none[12] = 0
    assert call(name, none, shape(B=0), params(name)) == OK
    assert call(name, none, shape(N=0), params(name)) == OK


@pytest.mark.parametrize("name", CALLS)
def test_null_and_misaligned(name):
    n, may, _ = CALLS[name]
    for i in range(n):
        if name == "pisa_prefix_attn" and i == 12:
            continue
        a = args(name)
        a[i] = None
        if i not in may:
            assert call(name, a, shape(), params(name)) == INVALID, i
        a[i] = A + 2
        assert call(name, a, shape(), params(name)) == INVALID, i


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("bad,rc", [(dict(d=96), UNSUPPORTED), (dict(d=0), INVALID), (dict(B=-1), INVALID),
                                    (dict(N=-1), INVALID), (dict(H_kv=0), INVALID), (dict(N_cap=1 << 25), UNSUPPORTED),
                                    (dict(B=1 << 20, N_cap=1 << 14), UNSUPPORTED)])
def test_shapes(name, bad, rc):
    assert call(name, args(name), shape(**bad), params(name)) == rc


@pytest.mark.parametrize("name", ["pisa_cache_write", "pisa_cache_read", "pisa_sparse_attn_cache"])
def test_more_rows_than_the_cache_holds(name):
    assert call(name, args(name), shape(N=129), params(name)) == INVALID


@pytest.mark.parametrize("name", ["pisa_sparse_attn_cache", "pisa_prefix_attn"])
def test_heads_and_parameters(name):
    assert call(name, args(name), shape(H_q=3), params(name)) == INVALID
    assert call(name, args(name), shape(H_q=6), params(name)) == UNSUPPORTED     # G_Q = 3
    assert call(name, args(name), shape(H_q=64), params(name)) == UNSUPPORTED    # G_Q = 32
    assert call(name, args(name), shape(), params(name, K=0)) == UNSUPPORTED
    assert call(name, args(name), shape(), params(name, K=33)) == UNSUPPORTED
    assert call(name, args(name), shape(), params(name, scale=math.nan)) == INVALID
    assert call(name, args(name), shape(), par(causal=name == "pisa_prefix_attn")) == UNSUPPORTED


def test_read_sides():
    for gone in ((6, 7), (0,), (2,), (1,), (3,)):  # no output; an output without its cache or scales
        a = args("pisa_cache_read")
        for i in gone:
            a[i] = None
        assert call("pisa_cache_read", a, shape(), None) == INVALID


def test_prefix_pairs_and_scratch():
    name = "pisa_prefix_attn"
    for i in (3, 4, 7, 8):  # one scale without the other, one own result without the other
        a = args(name)
        a[i] = None
        assert call(name, a, shape(), params(name)) == INVALID
    a = args(name)
    a[6] = None
    assert call(name, a, shape(B=2), params(name)) == INVALID  # several groups without their bounds
    need = pisa.pisa_prefix_attn_workspace_bytes(shape(), params(name))
    assert need > 0
    a = args(name)
    a[12] = need - 1
    assert call(name, a, shape(), params(name)) == WORKSPACE
    a[12] = need
    a[11] = A + 16
    assert call(name, a, shape(), params(name)) == INVALID
    assert call(name, args(name), shape(N=1 << 30), params(name)) == UNSUPPORTED
    assert call(name, args(name), shape(N_cap=0), params(name)) == INVALID
    assert pisa.pisa_prefix_attn_workspace_bytes(shape(d=96), params(name)) == 0
    assert pisa.pisa_prefix_attn_workspace_bytes(shape(), par(causal=True)) == 0


def test_binding_refuses_cpu_tensors_and_wrong_ranks():
    k = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    c = torch.zeros(1, 2, 8, 64, dtype=torch.int8)
    s = torch.zeros(1, 2, 8)
    n = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        pisa.pisa_cache_write(k, k, c, c, s, s, n)
    with pytest.raises(ValueError):
        pisa.pisa_cache_read(c, c, s, s, 4)
    with pytest.raises(ValueError):
        pisa.pisa_cache_read(None, None, None, None, 4)
    with pytest.raises(ValueError):
        pisa.pisa_sparse_attn_cache(k, c, c, s, s, torch.zeros(1, 2, 1, dtype=torch.int32), n)
    with pytest.raises(ValueError):
        pisa.pisa_prefix_attn(k, c, c, n, k_scale=s, v_scale=s)


@pytest.mark.gpu
def test_binding_refuses_what_does_not_match():
    dev = "cuda"
    k = torch.zeros(2, 2, 3, 64, dtype=torch.bfloat16, device=dev)
    c = torch.zeros(2, 2, 8, 64, dtype=torch.int8, device=dev)
    s = torch.zeros(2, 2, 8, device=dev)
    n = torch.zeros(2, dtype=torch.int32, device=dev)
    q = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16, device=dev)
    idx = torch.zeros(2, 2, 3, 1, dtype=torch.int32, device=dev)

    def write(**kw):
        a = dict(k=k, v=k, Kq=c, Vq=c, k_scale=s, v_scale=s, seq_len=n)
        a.update(kw)
        pisa.pisa_cache_write(**a)

    for kw in (dict(k=k.float()), dict(v=k[:, :, :2]), dict(k=k.transpose(2, 3)), dict(Kq=c.float()), dict(Vq=c[:1]),
               dict(k_scale=s.double()), dict(v_scale=s[..., :7]), dict(v_scale=None), dict(seq_len=n.long()),
               dict(seq_len=n[:1]), dict(seq_len=None), dict(new_len=n.cpu()), dict(k_out=k[..., :32]), dict(Kq=c[0])):
        with pytest.raises(ValueError):
            write(**kw)
    for kw in (dict(idx=idx[..., 0]), dict(idx=idx.long()), dict(q=q[:, :2]), dict(seq_len=None), dict(O=q.float()),
               dict(LSE=s), dict(q=q.reshape(2, 12, 64))):
        a = dict(q=q, Kq=c, Vq=c, k_scale=s, v_scale=s, idx=idx, seq_len=n)
        a.update(kw)
        with pytest.raises(ValueError):
            pisa.pisa_sparse_attn_cache(**a)
    rows = torch.zeros(3, dtype=torch.int32, device=dev)
    p = q.reshape(6, 4, 64)
    for kw in (dict(k_scale=None), dict(Kp=c.to(torch.bfloat16)), dict(prefix_len=None), dict(row_start=rows[:2]),
               dict(o_own=q), dict(q=q), dict(o=p[:2]), dict(lse=s)):
        a = dict(q=p, Kp=c, Vp=c, prefix_len=n, row_start=rows, k_scale=s, v_scale=s)
        a.update(kw)
        with pytest.raises(ValueError):
            pisa.pisa_prefix_attn(**a)
    for kw in (dict(v_scale=None), dict(row_start=None), dict(o_own=p)):
        a = dict(q=p, Kp=c, Vp=c, prefix_len=n, row_start=rows, k_scale=s, v_scale=s)
        a.update(kw)
        with pytest.raises((pisa.PisaError, ValueError)):
            pisa.pisa_prefix_attn(**a)
    with pytest.raises(pisa.PisaError):
        pisa.pisa_cache_read(c, c, s, s, 9)
