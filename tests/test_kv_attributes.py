"""What a KVCache says and what its calls use stay the same (no GPU): the calls pass addresses
taken at construction, so tensors cannot be exchanged under them."""
import pytest
import torch

import bit_linear_moe_b200 as nv

FIXED = ("data", "k_gs", "v_gs", "num_pages", "page_size", "heads", "head_dim", "format", "device")


def made(**kw):
    """A cache object as the constructor leaves it, without a device."""
    c = nv.KVCache.__new__(nv.KVCache)
    for n in FIXED:
        setattr(c, n, kw.get(n, 1))
    return c


@pytest.mark.parametrize("name", FIXED)
def test_attributes_are_set_once(name):
    old = torch.zeros(1)
    c = made(**{name: old})
    with pytest.raises(AttributeError, match="KVCache"):
        setattr(c, name, torch.ones(1))
    with pytest.raises(AttributeError, match="KVCache"):
        delattr(c, name)
    assert getattr(c, name) is old


def test_other_attributes_are_free():
    c = made()
    c.layer = 3
    c.layer = 4
    del c.layer
