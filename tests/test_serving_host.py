"""Host side of the serving operators, next to test_serving_cpu.py: the cache's tensors, the build, sizes and strides."""

import pytest
import torch


def test_cache_tensors_change_in_place_only():
    """`cache.lens += 1` counts once and does not raise; another tensor is refused before anything has changed."""
    from linear_attention_nats_gb300.paged import PagedCache

    names = ("k_pages", "v_pages", "table", "lens", "weight", "err")
    c = PagedCache.__new__(PagedCache)
    c._t = tuple(torch.zeros(2, dtype=torch.int32) for _ in names)
    for name, t in zip(names, c._t):
        assert getattr(c, name) is t
        setattr(c, name, t)
        with pytest.raises(AttributeError):
            setattr(c, name, t.clone())
    c.lens += 1
    assert c.lens is c._t[3] and c.lens.tolist() == [1, 1]
    with pytest.raises(AttributeError):
        c.lens = c.lens + 1
    assert c.lens.tolist() == [1, 1]
