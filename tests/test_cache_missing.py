"""The binding refuses a missing tensor of the 8-bit cache's and the prefix's calls by name, before any launch."""
import inspect

import pytest
import torch

import hierarchical_top_block_gb300 as pisa

WANTED = {
    "pisa_cache_write": ("k", "v", "Kq", "Vq", "k_scale", "v_scale", "seq_len"),
    "pisa_sparse_attn_cache": ("q", "Kq", "Vq", "k_scale", "v_scale", "idx", "seq_len"),
    "pisa_prefix_attn": ("q", "Kp", "Vp", "prefix_len"),
}


@pytest.mark.gpu
@pytest.mark.parametrize("call,name", [(c, n) for c, names in WANTED.items() for n in names])
def test_missing(call, name):
    dev = "cuda"
    k = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16, device=dev)
    code = torch.zeros(1, 2, 8, 64, dtype=torch.int8, device=dev)
    scale = torch.zeros(1, 2, 8, device=dev)
    n = torch.zeros(1, dtype=torch.int32, device=dev)
    given = dict(k=k, v=k, Kq=code, Vq=code, Kp=code, Vp=code, k_scale=scale, v_scale=scale, seq_len=n, prefix_len=n,
                 q=torch.zeros(1, 3, 4, 64, dtype=torch.bfloat16, device=dev),
                 idx=torch.zeros(1, 2, 3, 1, dtype=torch.int32, device=dev))
    if call == "pisa_prefix_attn":
        given["q"] = given["q"][0]
    fn = getattr(pisa, call)
    args = {a: x for a, x in given.items() if a in inspect.signature(fn).parameters}
    fn(**args)
    args[name] = None
    with pytest.raises(ValueError, match=name):
        fn(**args)
    assert pisa.pisa_get_last_device_error() == 0


@pytest.mark.parametrize("call", WANTED)
def test_missing_first(call):
    """Without a device at hand: the tensor that names the device, and the cache whose shape counts."""
    fn = getattr(pisa, call)
    none = {a: None for a in WANTED[call]}
    with pytest.raises(ValueError, match=WANTED[call][0]):
        fn(**none)
