"""Writing the quantised key/value cache and reading it back (GPU): stored bytes
and scales must equal the 64-bit definition exactly, values read back are its
values rounded once to bf16, and nothing else is touched."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from row_normalization_gb300 import binding
from tests import kv_ref
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    binding.device_status()


def rows(T, Hq, Hkv, D, seed):
    """Packed QKV with rows of very different size, exact ties, zeros and tiny groups."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, Hq + 2 * Hkv, D, generator=g)
    x *= torch.exp(3 * torch.randn(T, Hq + 2 * Hkv, 1, generator=g))
    x = x.to(torch.bfloat16)
    for i in range(0, T, 3):      # multiples of a half: every quotient a code or a tie
        x[i] = (torch.randint(-14, 15, (Hq + 2 * Hkv, D), generator=g).to(torch.bfloat16)) / 2
        x[i, :, ::32] = 7.0
    x[0, :, 32:64] = 0
    if T > 1:
        x[1] *= 2.0 ** -26        # scales among fp16's subnormals, and below them
    return x.reshape(T, -1)


def to_gpu(ref):
    return binding.KVCache(ref.codes.cuda(), ref.scales.cuda())


def same(cache, ref):
    assert torch.equal(cache.codes.cpu(), ref.codes)
    got = cache.scales.cpu().view(torch.int16).numpy().view(np.uint16)
    assert np.array_equal(got, ref.scales.contiguous().view(torch.int16).numpy().view(np.uint16))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,Hq,Hkv,D,P", [
    (1, 4, 1, 64, 16), (7, 3, 3, 128, 32), (33, 8, 2, 256, 64), (65, 0, 5, 128, 16),
    (130, 32, 8, 128, 256), (257, 1, 1, 64, 128),
])
def test_write_stores_exactly_the_definition(bits, T, Hq, Hkv, D, P):
    pages = 2 * T // P + 2
    ref = kv_ref.Cache(pages, Hkv, D, P, bits)
    cache = to_gpu(ref)
    qkv = rows(T, Hq, Hkv, D, seed=T + D)
    g = torch.Generator().manual_seed(T)
    slots = torch.randperm(pages * P, generator=g)[:T]
    slots[T // 2] = -1                                     # padding
    ref.write(qkv.view(T, Hq + 2 * Hkv, D)[:, Hq:].unflatten(1, (2, Hkv)), slots)
    before = qkv.cuda()
    got = binding.kv_cache_write(before, slots.cuda(), cache, Hq, Hkv, D)
    assert got is cache
    torch.cuda.synchronize()
    assert torch.equal(before.cpu(), qkv)
    same(cache, ref)                                        # rows no slot names included
    assert binding.device_status() == 0


@pytest.mark.parametrize("bits", [4, 8])
def test_non_finite_and_huge_groups(bits):
    T, Hkv, D, P = 6, 1, 64, 16
    ref = kv_ref.Cache(1, Hkv, D, P, bits)
    cache = to_gpu(ref)
    qkv = rows(T, 0, Hkv, D, seed=5)
    qkv[0, 3] = float("nan")
    qkv[1, 40] = float("inf")
    qkv[2, 70] = -float("inf")
    qkv[3, :32] = 3.3e38                                    # clamped to the largest scale
    qkv[4, 33] = -1e30
    slots = torch.tensor([5, 0, 9, 3, 15, 1])
    ref.write(qkv.view(T, 2, Hkv, D), slots)
    binding.kv_cache_write(qkv.cuda(), slots.cuda(), cache, 0, Hkv, D)
    torch.cuda.synchronize()
    same(cache, ref)
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    k, v = binding.kv_cache_read(cache, table, torch.tensor([0, P], device="cuda"), P)
    assert torch.isnan(k[5, 0, :32].float()).all() and not torch.isnan(k[5, 0, 32:].float()).any()
    assert torch.isnan(v[9, 0, :32].float()).all()
    assert torch.isfinite(k[3].float()).all()


def test_bad_slots_are_skipped_and_reported():
    T, Hkv, D, P, pages = 5, 2, 128, 16, 2
    ref = kv_ref.Cache(pages, Hkv, D, P, 4)
    cache = to_gpu(ref)
    qkv = rows(T, 0, Hkv, D, seed=9)
    slots = torch.tensor([pages * P, 3, -7, 2 ** 62, 31])
    ref.write(qkv.view(T, 2, Hkv, D), slots)
    binding.kv_cache_write(qkv.cuda(), slots.cuda(), cache, 0, Hkv, D)
    assert binding.device_status() == binding.RN_STATUS_BAD_INDEX
    assert binding.device_status() == 0
    same(cache, ref)


def filled(bits, Hkv, D, P, lens, seed):
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // P) for n in lens]
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=g)
    table = torch.full((len(lens), max(max(need), 1) + 1), -1, dtype=torch.int32)
    ref = kv_ref.Cache(pages, Hkv, D, P, bits)
    at = 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]].int()
        at += need[b]
        if n:
            pos = torch.arange(n)
            ref.write(rows(n, 0, Hkv, D, seed + b).view(n, 2, Hkv, D),
                      table[b, pos // P].long() * P + pos % P)
    return ref, table


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("Hkv,D,P", [(1, 64, 16), (3, 128, 32), (2, 256, 128), (8, 128, 64)])
def test_read_returns_the_values_rounded_once(bits, Hkv, D, P):
    lens = [1, 0, 40, 17, 0, 129, 0]
    starts = [0, 0, 3, 16, 0, 100, 0]
    ref, table = filled(bits, Hkv, D, P, lens, seed=11)
    cu = [4]                                                # four rows before the first sequence
    for n, s in zip(lens, starts):
        cu.append(cu[-1] + n - s)
    total = cu[-1] + 5
    canary = torch.full((total, Hkv, D), 7.5, dtype=torch.bfloat16)
    k, v = canary.cuda(), canary.cuda()
    binding.kv_cache_read(to_gpu(ref), table.cuda(), torch.tensor(cu).cuda(), total,
                          torch.tensor(starts, dtype=torch.int32).cuda(), k, v)
    assert binding.device_status() == 0
    for which, got in ((0, k.cpu()), (1, v.cpu())):
        want = canary.clone()
        for b, (n, s) in enumerate(zip(lens, starts)):
            want[cu[b]:cu[b + 1]] = ref.tokens(table[b], which, s, n).float().to(torch.bfloat16)
        assert torch.equal(got, want)


def test_read_of_bad_pages_gives_zeros_and_reports():
    Hkv, D, P = 2, 64, 16
    ref, table = filled(8, Hkv, D, P, [64], seed=3)
    pages = ref.codes.shape[0]
    table = torch.tensor([[int(table[0, 0]), -1, pages, int(table[0, 3])]], dtype=torch.int32)
    cache = to_gpu(ref)
    cu = torch.tensor([0, 80])
    k, v = binding.kv_cache_read(cache, table.cuda(), cu.cuda(), 80)
    assert binding.device_status() == binding.RN_STATUS_BAD_INDEX
    for which, got in ((0, k.cpu()), (1, v.cpu())):
        want = torch.cat((ref.tokens(table[0], which, 0, 64), torch.zeros(16, Hkv, D).double()))
        assert torch.equal(got, want.float().to(torch.bfloat16))
    # negative starts
    binding.kv_cache_read(cache, table[:, :1].contiguous().cuda(), torch.tensor([0, 2]).cuda(), 2,
                          torch.tensor([-2], dtype=torch.int32).cuda())
    assert binding.device_status() == binding.RN_STATUS_BAD_INDEX


def test_empty_calls():
    cache = binding.new_kv_cache(1, 1, 64, page_size=16)
    binding.kv_cache_write(torch.empty(0, 128, dtype=torch.bfloat16, device="cuda"),
                           torch.empty(0, dtype=torch.int64, device="cuda"), cache, 0, 1, 64)
    k, v = binding.kv_cache_read(cache, torch.empty(0, 0, dtype=torch.int32, device="cuda"),
                                 torch.zeros(1, dtype=torch.int64, device="cuda"), 0)
    assert k.shape == (0, 1, 64) and v.shape == k.shape


def test_offsets_beyond_32_bits():
    """A cache whose codes pass 4 GiB: first and last rows, written and read back."""
    Hkv, D, P = 8, 256, 256
    pages = 2 ** 32 // (2 * Hkv * P * D) + 2
    codes = torch.empty(pages, 2, Hkv, P, D, dtype=torch.uint8, device="cuda")
    scales = torch.empty(pages, 2, Hkv, P, D // 32, dtype=torch.float16, device="cuda")
    cache = binding.KVCache(codes, scales)
    T = 4
    qkv = rows(T, 0, Hkv, D, seed=1)
    slots = torch.tensor([0, pages * P - 1, (pages - 1) * P, 255])
    binding.kv_cache_write(qkv.cuda(), slots.cuda(), cache, 0, Hkv, D)
    table = torch.tensor([[0, pages - 1]], dtype=torch.int32, device="cuda")
    k, v = binding.kv_cache_read(cache, table, torch.tensor([0, 2 * P], device="cuda"), 2 * P)
    c, s = kv_ref.quantise(qkv.view(T, 2, Hkv, D), 8)
    want = kv_ref.values(c, s).float().to(torch.bfloat16)
    at = [0, 2 * P - 1, P, 255]
    assert torch.equal(k.cpu()[at], want[:, 0]) and torch.equal(v.cpu()[at], want[:, 1])
    assert binding.device_status() == 0


def test_another_stream():
    Hkv, D, P, T = 2, 128, 32, 50
    ref = kv_ref.Cache(3, Hkv, D, P, 4)
    cache = to_gpu(ref)
    qkv = rows(T, 2, Hkv, D, seed=21)
    slots = torch.randperm(96)[:T]
    ref.write(qkv.view(T, 2 + 2 * Hkv, D)[:, 2:].unflatten(1, (2, Hkv)), slots)
    x, sl = qkv.cuda(), slots.cuda()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    binding.kv_cache_write(x, sl, cache, 2, Hkv, D, stream=st)
    st.synchronize()
    same(cache, ref)
