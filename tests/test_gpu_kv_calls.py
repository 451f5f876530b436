"""Key/value cache calls as programs make them (GPU): results and workspaces on a stream
other than the caller's, one workspace for calls of several sizes, lengths and row offsets
that do not fit."""
from __future__ import annotations

import pytest
import torch

from row_normalization_gb300 import binding
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    binding.device_status()


def plain_cache(pages, Hkv, D, P, format, seed=0):
    """A cache of arbitrary codes and scales of ordinary size."""
    g = torch.Generator().manual_seed(seed)
    cache = binding.new_kv_cache(pages, Hkv, D, page_size=P, format=format)
    cache.codes.copy_(torch.randint(0, 256, cache.codes.shape, generator=g, dtype=torch.uint8))
    cache.scales.copy_((0.1 + torch.rand(cache.scales.shape, generator=g)).half())
    return cache


def side_streams():
    return [torch.cuda.Stream(), torch.cuda.Stream().cuda_stream]


def late(x):
    """x as the current stream reads it some milliseconds from now."""
    torch.cuda._sleep(20_000_000)
    return x.clone()


def calls(cache, B, Hq, stream):
    Hkv, D, P = cache.num_kv_heads, cache.head_dim, cache.page_size
    L = cache.num_pages // B * P
    table = torch.arange(cache.num_pages, dtype=torch.int32, device="cuda").view(B, -1)
    cu = torch.arange(B + 1, device="cuda") * L
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    q = torch.randn(B, Hq, D, device="cuda").bfloat16()
    torch.cuda.synchronize()
    return {"read": lambda: binding.kv_cache_read(cache, table, cu, B * L, stream=stream),
            "attend": lambda: binding.kv_attention_fwd(q, cache, table, lens, Hq, stream=stream)}


@pytest.mark.parametrize("which", ["read", "attend"])
@pytest.mark.parametrize("kind", [0, 1])
def test_new_results_do_not_take_memory_the_caller_still_reads(which, kind):
    """Blocks that the current stream reads late and the program has dropped are not
    handed to a call on another stream."""
    stream = side_streams()[kind]
    cache = plain_cache(80, 4, 128, 64, binding.RN_KV_INT4)
    call = calls(cache, 2, 32, stream)[which]
    n_ws = binding.kv_attention_workspace(cache, 2, 32).numel()
    sizes = ([80 * 64 * 4 * 128 * 2] * 2 if which == "read" else
             [2 * 32 * 128 * 2, 2 * 32 * 4, n_ws])
    call()                                                   # (loads the kernels)
    torch.cuda.synchronize()
    olds = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda.synchronize()
    copies = [late(x) for x in olds]
    olds.clear()
    results = call()
    torch.cuda.synchronize()
    assert len(results) == 2
    for x in copies:
        assert (x == 7).all()


@pytest.mark.parametrize("which", ["read", "attend"])
@pytest.mark.parametrize("kind", [0, 1])
def test_results_the_caller_still_reads_are_not_written_again(which, kind):
    """A result used on the current stream and dropped there is not handed to the next
    call on its own stream before that use."""
    stream = side_streams()[kind]
    one, two = (calls(plain_cache(80, 4, 128, 64, binding.RN_KV_INT4, seed), 2, 32, stream)[which]
                for seed in (0, 5))
    want = [x.clone() for x in (one(), torch.cuda.synchronize())[0]]
    first = one()
    torch.cuda.synchronize()
    copies = [late(x) for x in first]
    del first
    again = two()
    torch.cuda.synchronize()
    for x, y, z in zip(copies, want, again):
        assert torch.equal(x, y) and not torch.equal(z, y)


@pytest.mark.parametrize("format", [binding.RN_KV_INT4, binding.RN_KV_INT8])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_workspaces_never_shrink_as_calls_grow(format, D):
    query = binding.load().kv_attention_workspace_bytes
    Hkv = 2
    for group in (1, 2, 3, 4, 5, 8, 16, 20, 70, 130):
        last = 0
        for n in [*range(0, 140), 255, 256, 257, 5000]:
            now = query(format, 3, group * Hkv, Hkv, D, n)
            assert now >= last, (group, n)
            last = now
    for n in (1, 2, 7, 20, 100):
        last = 0
        for group in range(1, 200):
            now = query(format, 3, group * Hkv, Hkv, D, n)
            assert now >= last, (group, n)
            last = now
        assert query(format, 500, 8, Hkv, D, n) >= query(format, 3, 8, Hkv, D, n)


@pytest.mark.parametrize("format", [binding.RN_KV_INT4, binding.RN_KV_INT8])
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 32, 8), (128, 32, 8), (256, 16, 4)])
def test_one_workspace_for_calls_of_up_to_its_sizes(format, D, Hq, Hkv):
    """A server's workspace for its longest draft, used by shorter ones."""
    B, P, L, longest = 3, 64, 2048, 40
    cache = plain_cache(B * L // P, Hkv, D, P, format)
    table = torch.arange(B * L // P, dtype=torch.int32, device="cuda").view(B, -1)
    lens = torch.tensor([L, 900, 77], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(1)
    ws = {n: binding.kv_attention_workspace(cache, B, Hq, max_q_len=n) for n in (16, longest)}
    for n in (1, 2, 3, 4, 5, 16, 17, 32, 33, longest):
        q = torch.randn(B * n, Hq, D, generator=g).bfloat16().cuda()
        cu = torch.arange(B + 1, device="cuda") * n
        want = binding.kv_attention_fwd(q, cache, table, lens, Hq, cu_q=cu, max_q_len=n)
        for most, w in ws.items():
            if n <= most:
                w.fill_(0xFF)
                got = binding.kv_attention_fwd(q, cache, table, lens, Hq, cu_q=cu, max_q_len=n,
                                               workspace=w)
                assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert binding.device_status() == 0


@pytest.mark.parametrize("cu,total,bad", [([0, 40, 60], 60, False), ([5, 40, 60], 64, False),
                                          ([0, 40, 60], 59, True), ([0, 40, 60], 7, True),
                                          ([-3, 40, 60], 60, True), ([0, 0, 0], 4, False),
                                          ([100, 140, 160], 60, True)])
def test_reads_that_have_more_rows_than_their_results_say_so(cu, total, bad):
    cache = plain_cache(8, 3, 64, 16, binding.RN_KV_INT8)
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    k, v = (torch.full((total, 3, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    binding.kv_cache_read(cache, table, torch.tensor(cu).cuda(), total, k=k, v=v)
    assert binding.device_status() == (binding.RN_STATUS_BAD_INDEX if bad else 0)
    want, _ = binding.kv_cache_read(cache, table, torch.tensor([0, 64, 128]).cuda(), 128)
    for row in range(total):
        b = 0 if row < cu[1] else 1
        if cu[0] <= row < cu[2]:
            assert torch.equal(k[row], want[64 * b + row - cu[b]])
        else:
            assert (k[row] == 7).all() and (v[row] == 7).all()
