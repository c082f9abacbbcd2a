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


UNSUP = nv.NVFP4_ERR_UNSUPPORTED
BF16 = 2
A, B, C, D, E = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000  # fake aligned addresses


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(nv.LIB_PATH):
        from nvfp4_block_scaled_amd import build
        build.build()
    lib = nv.load_library()
    lib.nvfp4_debug_set_arch_override(b"gfx942")  # nothing reaches a device
    yield lib
    lib.nvfp4_debug_set_arch_override(None)


def _struct(heads, dim, pages=10, page=16):
    return nv._KVCacheStruct(A, B, C, D, None, None, pages, page, heads, dim)


def _says(L, status, text):
    assert status == UNSUP and text in L.nvfp4_last_error().decode(), L.nvfp4_last_error()


@pytest.mark.parametrize("heads,dim", [(2, 128), (8, 128), (1, 16), (32767, 256), (5, 80), (64, 240)])
def test_codec_limits(L, heads, dim):
    """Writes and reads take the tokens that the header states, and no more."""
    # (t dim / 4096 + 1) heads < 2^23, rounded down: t dim / 4096 <= (2^23 - 1) / heads - 1
    most = min((2 ** 31 - 4097) // (dim // 8), (((2 ** 23 - 1) // heads) * 512 - 1) // (dim // 8))
    c = _struct(heads, dim)
    for tokens, text in ((most, "gfx950"), (most + 1, "too large")):
        _says(L, L.nvfp4_kv_write(c, A, B, BF16, tokens, dim, dim, dim, dim, C, None), text)
        _says(L, L.nvfp4_kv_read(c, A, tokens, B, C, BF16, None), text)


def _attend(L, c, tokens, query_heads, seqs, max_queries, max_context, pages=8, window=0):
    need = L.nvfp4_kv_attention_workspace_size(c, tokens, query_heads, seqs, max_queries, max_context, window)
    return L.nvfp4_kv_attention(c, A, BF16, tokens, query_heads, 1, 1, B, seqs, pages, C, D, max_queries, max_context,
                                0.1, 1, window, E, None, E, need, None)


def test_attention_limits(L):
    """Attention's limits are its own: not those of writes, and every launch fits a grid."""
    _says(L, _attend(L, _struct(8, 128), 2 ** 26, 8, 4, 5, 100), "gfx950")  # more tokens than a write takes
    _says(L, _attend(L, _struct(8, 128), 2 ** 28, 8, 4, 5, 100), "too large")
    one = _struct(1, 16)
    _says(L, _attend(L, one, 2 ** 31 - 1, 1, 1, (2 ** 24 - 1) * 128, 100), "gfx950")
    _says(L, _attend(L, one, 2 ** 31 - 1, 1, 1, (2 ** 24 - 1) * 128 + 1, 100), "too large")
    far = _struct(1, 16, page=2 ** 22)
    _says(L, _attend(L, far, 1, 1, 1, 1, 2 ** 31 - 4096, pages=512), "gfx950")
    _says(L, _attend(L, far, 1, 1, 1, 1, 2 ** 31 - 4095, pages=512), "too large")


def test_workspace_sizes(L):
    """A long context is shared out and needs a workspace; one workgroup a pair needs none, and is no choice where
    there are 2^24 pairs."""
    size = L.nvfp4_kv_attention_workspace_size
    need = size(_struct(2, 128, pages=1 << 16), 1, 8, 1, 1, 1 << 20, 0)
    assert need > 0
    many = _struct(16384, 16)
    assert size(many, 1023, 16384, 1023, 1, 100, 0) == 0 and size(many, 1024, 16384, 1024, 1, 100, 0) > 0
    for window in (1 << 20, 1 << 40):  # as good as none
        assert size(_struct(2, 128, pages=1 << 16), 1, 8, 1, 1, 1 << 20, window) == need


class _Devices:
    """Two GPUs as torch shows them: the current one, and the changes to it."""

    def __init__(self, monkeypatch):
        self.current, self.entered = 0, []
        devices = self

        class device:
            def __init__(self, which):
                self.index = which if isinstance(which, int) else which.index

            def __enter__(self):
                self.before, devices.current = devices.current, self.index
                devices.entered.append(self.index)

            def __exit__(self, *_):
                devices.current = self.before

        monkeypatch.setattr(torch.cuda, "device", device)
        monkeypatch.setattr(nv, "_current_device", lambda: devices.current)


def test_calls_run_on_the_device_of_their_cache(monkeypatch):
    """A cache on another GPU than the current one: every call makes that current, and leaves the current one after."""
    import types
    devices = _Devices(monkeypatch)
    seen = []

    def stream(index):
        seen.append((index, devices.current))
        raise InterruptedError

    monkeypatch.setattr(nv, "_raw_stream", stream)
    cache = types.SimpleNamespace(device=torch.device("cuda:1"), _gpu=1, pages=2, heads=1, page_size=4, dim=16)
    for call in (lambda: nv.nvfp4_kv_write(cache, None, None, None), lambda: nv.nvfp4_kv_read(cache, None),
                 lambda: nv.nvfp4_kv_attention(None, cache, None, None)):
        with pytest.raises(InterruptedError):
            call()
        assert seen.pop() == (1, 1) and devices.entered.pop() == 1 and devices.current == 0
    cache.device, cache._gpu = torch.device("cuda:0"), 0
    with pytest.raises(InterruptedError):
        nv.nvfp4_kv_read(cache, None)
    assert seen.pop() == (0, 0) and not devices.entered


def test_workspace_bytes_are_of_a_device(monkeypatch):
    """GPUs may differ in compute units: the bytes of one are not remembered for the other."""
    import types
    devices = _Devices(monkeypatch)
    library = types.SimpleNamespace(nvfp4_kv_attention_workspace_size=lambda *_: (100, 300)[devices.current])
    monkeypatch.setattr(nv, "load_library", lambda: library)
    nv._kv_attention_bytes.cache_clear()
    sizes = (2, 4, 1, 16, 1, 1, 1, 1, 8, 0)
    assert [nv._kv_attention_bytes(d, *sizes) for d in (0, 1, 0, 1)] == [100, 300, 100, 300]
    assert devices.entered == [0, 1]
    nv._kv_attention_bytes.cache_clear()


def test_cache_declarations_keep_to_their_header():
    """bench.py reports measured traffic only for the sources and the two shared headers that it was measured on:
    the cache's declarations stand in a header of their own, so that they do not void those figures."""
    import os
    csrc = os.path.join(os.path.dirname(nv.LIB_PATH), "csrc")
    for shared in ("nvfp4_internal.h", "nvfp4_device.h"):
        with open(os.path.join(csrc, shared)) as f:
            text = f.read()
        assert "kv_" not in text and "Kv" not in text, shared
