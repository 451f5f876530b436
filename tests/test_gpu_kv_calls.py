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
