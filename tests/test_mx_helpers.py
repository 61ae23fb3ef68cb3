"""The torch helpers of the microscaled 4-bit operators on host memory: refused before any call."""
import pytest
import torch

from hadamard_rotated_precision_amd import tensors as T


def test_tensors_on_the_host_are_refused():
    q = T.MxTensor(8, 64, device="cpu")
    x = torch.zeros(8, 64)
    with pytest.raises(ValueError, match="GPU"):
        q.quantize(x)
    with pytest.raises(ValueError, match="GPU"):
        q.dequantize(x)
    with pytest.raises(ValueError, match="GPU"):
        T.mx_gemm(q, q, torch.zeros(8, 8), ws=torch.zeros(16, dtype=torch.uint8))
    layer = T.MxLayer(8, 64, 32, device="cpu")
    with pytest.raises(ValueError, match="GPU"):
        layer.set_weight(torch.zeros(32, 64))
    with pytest.raises(ValueError, match="GPU"):
        layer.fwd(x, torch.zeros(8, 32))
    cache = T.KVCache(4, 16, 2, 64, device="cpu")
    k, slots = torch.zeros(3, 2, 64), torch.arange(3)
    with pytest.raises(ValueError, match="GPU"):
        cache.append(k, k, slots)
    with pytest.raises(ValueError, match="GPU"):
        cache.read(slots, k=k)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        cache.attend(k, k.clone(), i, i[:1], i[:1].view(1, 1), max_q=3, max_len=5, ws=torch.zeros(1 << 20, dtype=torch.uint8))


def test_buffers_stay():
    q = T.MxTensor(8, 64, device="cpu")
    with pytest.raises(AttributeError):
        q.codes = q.codes.clone()
    cache = T.KVCache(4, 16, 2, 64, device="cpu")
    with pytest.raises(AttributeError):
        cache.k_codes = cache.k_codes.clone()


def test_layouts():
    q = T.MxTensor(70, 100, device="cpu")
    assert q.codes.shape == (70, 64) and q.scales.shape == (70, 16)
    assert q.codes_t.shape == (100, 48) and q.scales_t.shape == (100, 16)
    assert T.MxTensor(70, 100, codes=False, device="cpu").codes is None
    with pytest.raises(ValueError, match="holds"):
        T.MxTensor(8, 8, codes=False, codes_t=False, device="cpu")
    cache = T.KVCache(3, 32, 2, 256, rotate=False, device="cpu")
    assert cache.k_codes.shape == (3, 2, 32, 128) and cache.v_scales.shape == (3, 2, 32, 8)
    assert cache.st.rot == 1 and T.KVCache(3, 32, 2, 256, device="cpu").st.rot == 256


def test_bounds_past_32_bits_are_refused():
    """The library's struct holds 32-bit bounds, and ctypes would cut longer ones: 2^32 + 5 to 5."""
    cache = T.KVCache(4, 16, 2, 64, device="cpu")
    q, i = torch.zeros(3, 2, 64), torch.zeros(2, dtype=torch.int32)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    for name in ("max_q", "max_len", "window"):
        for value in (1 << 31, (1 << 32) + 5, 1 << 63):
            kw = dict(dict(max_q=3, max_len=5, window=0), **{name: value})
            with pytest.raises(ValueError, match=name):
                cache.attend(q, q.clone(), i, i[:1], i[:1].view(1, 1), ws=ws, **kw)
    for kw in (dict(max_q=(1 << 32) + 1, max_len=5), dict(max_q=1, max_len=(1 << 32) + 5)):
        with pytest.raises(ValueError, match="32 bits"):
            cache.attention_workspace(1, 2, **kw)
    with pytest.raises(ValueError, match="seqs"):
        cache.attention_workspace((1 << 32) + 1, 2, max_q=1, max_len=5)


def test_wrapped_codes_need_their_scales():
    q = T.MxTensor(8, 64, device="cpu")
    for t in (q.codes, q.scales, q.codes_t, q.scales_t):
        t.zero_()
    assert T.MxTensor.wrap(q.codes, q.scales, 8, 64).scales is q.scales
    for args, kw in (((q.codes, None, 8, 64), {}), ((None, q.scales, 8, 64), {}),
                     ((q.codes, q.scales, 8, 64), dict(codes_t=q.codes_t)),
                     ((q.codes, q.scales, 8, 64), dict(scales_t=q.scales_t))):
        with pytest.raises(ValueError, match="needed"):
            T.MxTensor.wrap(*args, **kw)
