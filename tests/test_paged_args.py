"""Refusals of the paged cache's entry points: no GPU is touched."""
import math

import pytest
import torch

import hierarchical_top_block_gb300 as pisa

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 6
A = 0x1000  # an aligned address that nothing reads: every call made with it is refused

# tensors, which of them may be NULL, whether parameters follow
CALLS = {"pisa_paged_write": (8, {4, 7}, False), "pisa_paged_attn": (9, {5, 7}, True),
         "pisa_paged_weights": (8, {6}, True), "pisa_paged_evict": (9, {7, 8}, False)}


def shape(**kw):
    s = dict(B=1, N=2, H_q=4, H_kv=2, d=64, N_cap=0)
    s.update(kw)
    return pisa.make_shape(**s)


def par(**kw):
    p = dict(K=4)
    p.update(kw)
    return pisa.make_params(**p)


def call(name, null=(), odd=(), ws_bytes=1 << 40, s=None, p=None, pages=(10, 16, 4), extra=None):
    a = [None if i in null else A + 0x1000 * i + (2 if i in odd else 0) for i in range(CALLS[name][0])]
    s, p = s or shape(), p or par()
    if name == "pisa_paged_write":
        a += extra or [0, 0]
    elif name == "pisa_paged_attn":
        a += [ws_bytes] + (extra or [0])
    elif name == "pisa_paged_weights":
        a += [ws_bytes] + (extra or [1, 0])
    else:
        a += [ws_bytes] + (extra or [8, 1, 2, 1])
    a += [s] + ([p] if CALLS[name][2] else []) + [pisa.pisa_pages(*pages), None]
    return getattr(pisa.lib(), name)(*a)


@pytest.mark.parametrize("name", CALLS)
def test_nothing_to_do(name):
    every = set(range(CALLS[name][0]))
    assert call(name, null=every, s=shape(B=0)) == OK
    if name != "pisa_paged_evict":
        assert call(name, null=every, s=shape(N=0)) == OK


@pytest.mark.parametrize("name", CALLS)
def test_null_and_misaligned(name):
    n, may, _ = CALLS[name]
    for i in range(n):
        if i not in may:
            assert call(name, null={i}) == INVALID, i
        assert call(name, odd={i}) == INVALID, i
    if name == "pisa_paged_evict":
        assert call(name, null={7, 8}) == INVALID


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("bad,rc", [(dict(d=96), UNSUPPORTED), (dict(d=0), INVALID), (dict(B=-1), INVALID),
                                    (dict(H_kv=0), INVALID), (dict(N_cap=64), INVALID), (dict(B=1 << 15), UNSUPPORTED)])
def test_shapes(name, bad, rc):
    assert call(name, s=shape(**bad)) == rc


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("pages,rc", [((0, 16, 4), INVALID), ((4, 0, 4), INVALID), ((4, 16, 0), INVALID), ((4, 8, 4), UNSUPPORTED),
                                      ((4, 48, 4), UNSUPPORTED), ((4, 16, 1 << 21), UNSUPPORTED), ((4, 1 << 25, 1), UNSUPPORTED)])
def test_pages(name, pages, rc):
    assert call(name, pages=pages) == rc


@pytest.mark.parametrize("name", ["pisa_paged_write", "pisa_paged_attn", "pisa_paged_weights"])
def test_rows(name):
    assert call(name, s=shape(N=-1)) == INVALID
    assert call(name, s=shape(N=1 << 30)) == UNSUPPORTED
    row_start = {"pisa_paged_write": 7, "pisa_paged_attn": 5, "pisa_paged_weights": 6}[name]
    assert call(name, null={row_start}, s=shape(B=3, N=4)) == INVALID  # not the same number each


@pytest.mark.parametrize("name", ["pisa_paged_attn", "pisa_paged_weights"])
def test_heads_and_parameters(name):
    assert call(name, s=shape(H_q=3)) == INVALID
    assert call(name, s=shape(H_q=6)) == UNSUPPORTED   # G_Q = 3
    assert call(name, s=shape(H_q=64)) == UNSUPPORTED  # G_Q = 32
    assert call(name, p=par(scale=math.nan)) == INVALID
    p = par()
    p.causal = 2
    assert call(name, p=p) == INVALID


def test_strides():
    for bad in (127, 120, -256, 1 << 31):
        assert call("pisa_paged_write", extra=[bad, 0]) == INVALID
        assert call("pisa_paged_write", extra=[0, bad]) == INVALID
    for bad in (255, 248, 260, -256, 1 << 31):
        assert call("pisa_paged_attn", extra=[bad]) == INVALID
        assert call("pisa_paged_weights", extra=[1, bad]) == INVALID
    assert call("pisa_paged_weights", extra=[2, 0]) == INVALID


def test_scratch():
    pages = pisa.pisa_pages(10, 16, 4)
    need = pisa.pisa_paged_attn_workspace_bytes(shape(), par(), pages)
    assert need > 0
    assert call("pisa_paged_attn", ws_bytes=need - 1) == WORKSPACE
    assert pisa.pisa_paged_attn_workspace_bytes(shape(d=96), par(), pages) == 0
    assert pisa.pisa_paged_attn_workspace_bytes(shape(B=0), par(), pages) == 0
    need = pisa.pisa_paged_weights_workspace_bytes(shape(), par(), pages)
    assert need > 0
    assert call("pisa_paged_weights", ws_bytes=need - 1) == WORKSPACE
    assert pisa.pisa_paged_weights_workspace_bytes(shape(d=96), par(), pages) == 0
    need = pisa.pisa_paged_evict_workspace_bytes(shape(), pages, 8)
    assert need >= 2 * 8 * 4
    assert call("pisa_paged_evict", null={7}, ws_bytes=need - 1) == WORKSPACE
    assert pisa.pisa_paged_evict_workspace_bytes(shape(), pages, 0) == 0


@pytest.mark.parametrize("keep,sinks,recent,m,rc", [(0, 0, 0, 1, INVALID), (-1, 0, 0, 1, INVALID), (8, -1, 0, 1, INVALID),
                                                    (8, 0, -1, 1, INVALID), (8, 5, 4, 1, INVALID), (17, 0, 0, 1, INVALID),
                                                    (8, 0, 0, 0, INVALID), (8, 1, 2147483647, 1, INVALID),
                                                    (1 << 25, 0, 0, 1 << 21, UNSUPPORTED)])
def test_evict_arguments(keep, sinks, recent, m, rc):
    assert call("pisa_paged_evict", extra=[keep, sinks, recent, m]) == rc


def test_binding_refuses_cpu_tensors():
    k = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    pool, w = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(4, 2, 16)
    table, n = torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for f in (lambda: pisa.pisa_paged_write(k, k, pool, pool, table, n), lambda: pisa.pisa_paged_attn(k, pool, pool, table, n),
              lambda: pisa.pisa_paged_weights(k, w, pool, w, table, n), lambda: pisa.pisa_paged_evict(pool, pool, w, table, n, table, 4)):
        with pytest.raises(ValueError):
            f()


@pytest.mark.gpu
def test_binding_refuses_what_does_not_match():
    dev = "cuda"
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device=dev)
    k = q[:, :2].contiguous()
    pool, w = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16, device=dev), torch.zeros(4, 2, 16, device=dev)
    table, n = torch.zeros(2, 1, dtype=torch.int32, device=dev), torch.zeros(2, dtype=torch.int32, device=dev)
    rows, lse = torch.zeros(3, dtype=torch.int32, device=dev), torch.zeros(2, 4, device=dev)
    wide = torch.zeros(2, 4, 68, dtype=torch.bfloat16, device=dev)[..., :64]
    common = [dict(Kp=pool[0]), dict(Kp=pool.float()), dict(Kp=None), dict(page_table=table.long()), dict(page_table=table[0]),
              dict(page_table=None), dict(seq_len=None), dict(seq_len=n[:1]), dict(row_start=rows[:2]), dict(row_start=rows.cpu())]
    calls = [
        (pisa.pisa_paged_write, dict(k=k, v=k, Kp=pool, Vp=pool, page_table=table, seq_len=n, row_start=rows, w=w),
         [dict(k=k.float()), dict(v=None), dict(v=k[:1]), dict(k=q), dict(w=w[:2]), dict(w=w.double()), dict(Vp=None), dict(Vp=pool[:2]),
          dict(k=wide[:, :2]), dict(k=q[:, ::2]), dict(k=q.transpose(1, 2)), dict(k=None), dict(k=k[0])]),
        (pisa.pisa_paged_attn, dict(q=q, Kp=pool, Vp=pool, page_table=table, seq_len=n, row_start=rows),
         [dict(q=q[0]), dict(q=q.float()), dict(q=wide), dict(q=q[..., :32]), dict(o=q[:1]), dict(o=q.float()), dict(lse=lse[:1]),
          dict(lse=lse.double()), dict(Vp=None), dict(ws=w), dict(o=wide)]),
        (pisa.pisa_paged_weights, dict(q=q, lse=lse, Kp=pool, w=w, page_table=table, seq_len=n, row_start=rows),
         [dict(q=q[0]), dict(q=wide), dict(lse=None), dict(lse=lse[:, :2]), dict(w=None), dict(w=w[..., :8]), dict(lse=lse.bfloat16())]),
        (pisa.pisa_paged_evict, dict(Kp=pool, Vp=pool, w=w, page_table=table, seq_len=n, new_table=table, keep=4),
         [dict(w=None), dict(Vp=None), dict(new_table=None), dict(new_table=table[0]), dict(new_table=table.long()),
          dict(new_len=n[:1]), dict(kept=table), dict(Vp=pool[:1]), dict(new_table=table[:1])])]
    for fn, good, bad in calls:
        for kw in bad + [x for x in common if next(iter(x)) in good]:
            with pytest.raises(ValueError):
                fn(**{**good, **kw})
    for kw in (dict(keep=0), dict(keep=17), dict(sinks=3, recent=2)):
        with pytest.raises(pisa.PisaError):
            pisa.pisa_paged_evict(**{**calls[3][1], **kw})
    with pytest.raises(pisa.PisaError):  # three heads over two
        pisa.pisa_paged_attn(q[:, :3], pool, pool, table, n)
