"""More of the key/value cache calls' host side (no GPU, no kernel)."""
import pytest
import torch

import nvfp4_block_scaled_amd as nv


def _held(pages=2, heads=3, page=4, dim=64):
    return {n + part: torch.zeros(pages, heads, page, dim // per, dtype=torch.uint8)
            for n in ("k_", "v_") for part, per in (("codes", 2), ("scales", 16))}


def _points_at(c):
    s = c._struct
    for n in ("k_codes", "k_scales", "v_codes", "v_scales", "global_scale_k", "global_scale_v"):
        t = getattr(c, n)
        assert getattr(s, n) == (None if t is None else t.data_ptr()), n
    assert (s.pages, s.heads, s.page_size, s.dim) == (c.pages, c.heads, c.page_size, c.dim)


def test_cache_attributes_assigned_anew():
    """What calls get always points at the tensors that the cache holds now."""
    c = nv.KVCache(**_held())
    _points_at(c)
    for n in ("global_scale_k", "global_scale_v"):
        for g in (torch.ones(1), torch.full((), 2.0), None):
            setattr(c, n, g)
            assert getattr(c, n) is g
            _points_at(c)
    for n, t in _held().items():
        setattr(c, n, t)
        assert getattr(c, n) is t
        _points_at(c)


def test_cache_attributes_refused():
    """An unfit tensor is refused and nothing changes; sizes are not assigned and nothing is deleted."""
    c = nv.KVCache(**_held())
    before = {n: getattr(c, n) for n in (*_held(), "global_scale_k", "global_scale_v")}
    for n, bad in (("k_codes", torch.zeros(2, 3, 5, 32, dtype=torch.uint8)), ("v_scales", torch.zeros(2, 3, 4, 4)),
                   ("k_scales", torch.zeros(2, 3, 4, 8, dtype=torch.uint8)[..., ::2]), ("global_scale_k", torch.ones(2)),
                   ("global_scale_v", torch.ones(1, dtype=torch.float16))):
        with pytest.raises(ValueError):
            setattr(c, n, bad)
    for n, value in (("pages", 3), ("heads", 1), ("page_size", 8), ("dim", 128), ("device", "cuda:0"), ("_struct", None)):
        with pytest.raises(AttributeError):
            setattr(c, n, value)
    for n in ("k_codes", "global_scale_k", "pages", "_struct"):
        with pytest.raises(AttributeError):
            delattr(c, n)
    assert all(getattr(c, n) is t for n, t in before.items())
    _points_at(c)
    c.owner = "anything else may be kept on it"
