"""The handle of a paged cache holds its tensors' addresses, so neither they nor
what follows from them can be exchanged under it, and a copy of it is a handle
of its own."""
import copy
import pickle

import pytest
import torch

NAMES = ["k", "v", "k_scale", "v_scale", "num_pages", "page_size", "H_kv", "d", "format", "dtype", "device"]


@pytest.mark.parametrize("name", NAMES)
def test_parts_of_a_handle_cannot_be_assigned(name):
    import quantized_attention_08_b200 as sage
    handle = object.__new__(sage.SageKVCache)  # a whole one needs a GPU
    with pytest.raises(AttributeError):
        setattr(handle, name, torch.zeros(4, 2, 16, 64, dtype=torch.float16))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["16", "B", "8+8"])
def test_handle_names_what_it_was_made_of(fmt):
    import quantized_attention_08_b200 as sage
    c = sage.SageKVCache.allocate(5, 2, 32, 64, fmt, torch.bfloat16)
    assert [c.num_pages, c.H_kv, c.page_size, c.d, c.format, c.dtype] == [5, 2, 32, 64, fmt, torch.bfloat16]
    assert c.device == c.k.device and c.k.shape == c.v.shape == (5, 2, 32, 64)
    assert (c.k_scale is None) == (fmt == "16") and (c.v_scale is None) == (fmt != "8+8")


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["16", "B", "8+8"])
@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, lambda c: pickle.loads(pickle.dumps(c))],
                         ids=["copy", "deepcopy", "pickle"])
def test_copied_handles(fmt, how):
    """What is appended through a copy lands in the copy's own tensors, those of
    the first handle if it shares them."""
    import quantized_attention_08_b200 as sage
    c = sage.SageKVCache.allocate(3, 2, 16, 64, fmt, torch.bfloat16)
    other = how(c)
    shares = how is copy.copy
    assert (other.k.data_ptr() == c.k.data_ptr()) == shares and other.format == fmt and other.dtype == torch.bfloat16
    x = torch.ones(2, 1, 64, dtype=torch.bfloat16, device="cuda")
    sage.sage_kv_append(x, x, torch.tensor([17], dtype=torch.int32, device="cuda"), other)
    assert bool((other.k[1, :, 1] != 0).all()) and bool((other.v[1, :, 1] != 0).all())
    assert bool((c.k[1, :, 1] != 0).all()) == shares and bool((c.v[1, :, 1] != 0).all()) == shares
