"""The key/value cache entry points refuse bad arguments on the host (CPU only:
no compute call is made here), and the format's plain definition holds together."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from row_normalization_gb300 import binding
from row_normalization_gb300.binding import (RN_ERR_ALIGN, RN_ERR_ARG, RN_ERR_NULL, RN_ERR_SHAPE,
                                             RN_KV_INT4, RN_KV_INT8, RN_OK)
from row_normalization_gb300.build import build
from tests import kv_ref

P = 0x10000  # well-formed pointers that nothing dereferences


@pytest.fixture(scope="module")
def lib():
    build()
    return binding.load()


def write(lib, qkv=P, slots=P, T=4, Hq=4, Hkv=2, D=128, fmt=RN_KV_INT4, page=16, pages=8, codes=P,
          scales=P):
    return lib.kv_cache_write(qkv, slots, T, Hq, Hkv, D, fmt, page, pages, codes, scales, None)


def read(lib, codes=P, scales=P, fmt=RN_KV_INT4, Hkv=2, D=128, page=16, pages=8, table=P, B=2,
         width=4, cu=P, starts=None, total=5, k=P, v=P + 4096):
    return lib.kv_cache_read(codes, scales, fmt, Hkv, D, page, pages, table, B, width, cu, starts,
                             total, k, v, None)


def attend(lib, q=P, stride=512, codes=P, scales=P, fmt=RN_KV_INT4, Hq=4, Hkv=2, D=128, page=16,
           pages=8, table=P, B=2, width=4, lens=P, cu=P, T=5, max_q=3, scale=0.1, window=0, sinks=0,
           out=P, lse=P, ws=P, ws_bytes=1 << 40):
    return lib.kv_attention_fwd(q, stride, codes, scales, fmt, Hq, Hkv, D, page, pages, table, B,
                                width, lens, cu, T, max_q, scale, window, sinks, out, lse, ws,
                                ws_bytes, None)


@pytest.mark.parametrize("call", [write, read, attend])
@pytest.mark.parametrize("kw,expect", [
    ({"fmt": 5}, RN_ERR_ARG), ({"fmt": 0}, RN_ERR_ARG),
    ({"D": 96}, RN_ERR_SHAPE), ({"D": 512}, RN_ERR_SHAPE),
    ({"page": 8}, RN_ERR_SHAPE), ({"page": 48}, RN_ERR_SHAPE), ({"page": 512}, RN_ERR_SHAPE),
    ({"Hkv": 0}, RN_ERR_SHAPE), ({"Hkv": -1}, RN_ERR_SHAPE), ({"pages": 0}, RN_ERR_SHAPE),
    ({"pages": 1 << 31}, RN_ERR_SHAPE),
    ({"codes": None}, RN_ERR_NULL), ({"scales": None}, RN_ERR_NULL),
    ({"codes": P + 8}, RN_ERR_ALIGN), ({"scales": P + 8}, RN_ERR_ALIGN),
])
def test_cache_arguments(lib, call, kw, expect):
    assert call(lib, **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    ({"T": -1}, RN_ERR_SHAPE), ({"T": 1 << 30}, RN_ERR_SHAPE), ({"Hq": -1}, RN_ERR_SHAPE),
    ({"T": 0}, RN_OK), ({"qkv": None}, RN_ERR_NULL), ({"slots": None}, RN_ERR_NULL),
    ({"qkv": P + 2}, RN_ERR_ALIGN), ({"slots": P + 4}, RN_ERR_ALIGN),
])
def test_write_arguments(lib, kw, expect):
    assert write(lib, **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    ({"total": -1}, RN_ERR_SHAPE), ({"total": 1 << 30}, RN_ERR_SHAPE), ({"B": -1}, RN_ERR_SHAPE),
    ({"width": -1}, RN_ERR_SHAPE), ({"total": 0}, RN_OK), ({"B": 0}, RN_OK),
    ({"cu": None}, RN_ERR_NULL), ({"k": None}, RN_ERR_NULL), ({"v": None}, RN_ERR_NULL),
    ({"table": None}, RN_ERR_NULL), ({"cu": P + 4}, RN_ERR_ALIGN), ({"starts": P + 2}, RN_ERR_ALIGN),
    ({"table": P + 1}, RN_ERR_ALIGN), ({"k": P + 8}, RN_ERR_ALIGN), ({"v": P}, RN_ERR_ARG),
])
def test_read_arguments(lib, kw, expect):
    assert read(lib, **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    ({"Hq": 5}, RN_ERR_SHAPE), ({"Hq": 0}, RN_ERR_SHAPE), ({"T": -1}, RN_ERR_SHAPE),
    ({"T": 1 << 30}, RN_ERR_SHAPE), ({"B": -1}, RN_ERR_SHAPE), ({"B": 1 << 30}, RN_ERR_SHAPE),
    ({"width": 1 << 28}, RN_ERR_SHAPE), ({"max_q": -1}, RN_ERR_SHAPE),
    ({"cu": None}, RN_ERR_SHAPE),                       # T != B
    ({"stride": 504}, RN_ERR_SHAPE), ({"stride": 516}, RN_ERR_SHAPE),
    ({"window": -1}, RN_ERR_ARG), ({"sinks": -1}, RN_ERR_ARG),
    ({"scale": float("nan")}, RN_ERR_ARG), ({"scale": float("inf")}, RN_ERR_ARG),
    ({"T": 0}, RN_OK), ({"B": 0}, RN_OK), ({"max_q": 0}, RN_OK),
    ({"q": None}, RN_ERR_NULL), ({"lens": None}, RN_ERR_NULL), ({"out": None}, RN_ERR_NULL),
    ({"ws": None}, RN_ERR_NULL), ({"table": None}, RN_ERR_NULL),
    ({"q": P + 8}, RN_ERR_ALIGN), ({"out": P + 8}, RN_ERR_ALIGN), ({"ws": P + 8}, RN_ERR_ALIGN),
    ({"lse": P + 2}, RN_ERR_ALIGN), ({"lens": P + 2}, RN_ERR_ALIGN), ({"cu": P + 4}, RN_ERR_ALIGN),
])
def test_attention_arguments(lib, kw, expect):
    assert attend(lib, **kw) == expect


def test_attention_workspace_sizes_refused(lib):
    for args in [(5, 1, 4, 2, 128, 1), (4, 1, 5, 2, 128, 1), (4, -1, 4, 2, 128, 1),
                 (4, 1, 4, 2, 100, 1), (4, 1, 4, 2, 128, -1)]:
        assert lib.kv_attention_workspace_bytes(*args) in (RN_ERR_ARG, RN_ERR_SHAPE)


def test_binding_refuses_host_tensors_and_wrong_shapes():
    cache = binding.new_kv_cache(2, 2, 64, page_size=16, device="cpu")
    assert (cache.num_pages, cache.num_kv_heads, cache.head_dim, cache.page_size) == (2, 2, 64, 16)
    assert cache.format == RN_KV_INT4
    assert binding.new_kv_cache(1, 1, 256, format=RN_KV_INT8, device="cpu").format == RN_KV_INT8
    with pytest.raises(ValueError):
        binding.kv_cache_write(torch.zeros(1, 8 * 64), torch.zeros(1), cache, 4, 2, 64)
    with pytest.raises(ValueError):
        binding.kv_cache_read(cache, torch.zeros(1, 1), torch.zeros(2), 1)
    with pytest.raises(ValueError):
        binding.kv_attention_fwd(torch.zeros(1, 256), cache, torch.zeros(1, 1), torch.zeros(1), 4)
    for kw in ({"D": 96}, {"page_size": 20}, {"format": 3}, {"num_pages": 0}):
        args = {"num_pages": 2, "Hkv": 2, "D": 64, "device": "cpu", **kw}
        with pytest.raises(binding.RowNormError):
            binding.new_kv_cache(**args)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_stored_orders_are_permutations_inside_groups(D):
    for value in (False, True):
        assert sorted(kv_ref.stored_order(D, value)) == list(range(D))


@pytest.mark.parametrize("bits", [4, 8])
def test_plain_quantiser_is_within_half_a_step(bits):
    g = torch.Generator().manual_seed(7)
    x = (torch.randn(300, 128, generator=g) * torch.exp(4 * torch.randn(300, 1, generator=g)))
    x = x.to(torch.bfloat16)
    c, s = kv_ref.quantise(x, bits)
    step = s.double().repeat_interleave(32, -1)
    # s is max|x| / Q rounded to fp16: off by half a step of fp16, 2^-11 s at most, or 2^-25
    # where s is subnormal.  The clamp to Q codes then takes up to Q times that.  (Beyond
    # 65504 Q the largest scale's clamp decides, as documented.)
    room = 0.5 * step + kv_ref.QMAX[bits] * torch.clamp(step * 2.0 ** -11, min=2.0 ** -25)
    near = x.double().abs() <= 65504.0 * kv_ref.QMAX[bits]
    assert ((kv_ref.values(c, s) - x.double()).abs() <= room)[near].all()
    assert (kv_ref.values(c, s).abs() == 65504.0 * kv_ref.QMAX[bits])[~near].all()


def test_quotient_is_a_tie_or_far_from_one():
    """x / s for 8-bit x and 11-bit s: exactly k + 1/2, or 2^-12 away from every
    such value (what the kernel's two roundings rely on).  All significand pairs,
    quotients up to the 8-bit codes' 127.5."""
    X = np.arange(128, 256, dtype=np.int64)[:, None]
    S = np.arange(1024, 2048, dtype=np.int64)[None, :]
    for e in range(-1, 12):  # x / s = X / S * 2^(e + 3): 0.5 .. 127.5 and above
        num, den = (X << (e + 4)), S << 1
        k2 = np.round(num / S).astype(np.int64)          # 2 x / s to the nearest integer
        for near in (k2 - 1, k2, k2 + 1):
            odd = (near % 2) != 0
            gap = np.abs(num - near * S)                  # |2 x / s - near| * S
            use = odd & (near > 0) & (near <= 255) & (gap != 0)
            assert (gap[use] * 2 ** 11 >= np.broadcast_to(S, gap.shape)[use]).all()
        assert den.shape == S.shape
