"""Every layout that rows of logits are given, clusters that take several rows among them (GPU).

Each test asks which layout its rows get, so that another choice of layouts cannot leave one
of them without a test."""
from __future__ import annotations

import pytest
import torch

from row_normalization_gb300 import binding
from row_normalization_gb300.binding import RowNormError
from tests.gpu_util import require_gpu
from tests.test_gpu_logprobs_equal_largest import apart
from tests.test_gpu_token_logprobs import BF, DTYPES, F32, HALF, INF, check, logits

pytestmark = pytest.mark.gpu

# threads of a block, blocks of a row, rows, columns in 16 bits (in 32 bits half of them)
LAYOUTS = [(64, 1, 2048, 8003), (96, 1, 1500, 9001), (128, 1, 1000, 30000), (192, 1, 700, 20001),
           (256, 1, 350, 20000), (320, 1, 333, 50000), (512, 1, 150, 60001),
           (128, 8, 1, 50021), (128, 8, 20, 50021), (128, 8, 100, 131072), (256, 4, 110, 262144),
           (256, 8, 7, 131073), (256, 8, 40, 131072)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    binding.device_status()


def varied(T, V, dtype, offset=0):
    """Rows that differ: plain ones, nearly sure ones, banned, few values, all equal, and rows whose
    largest lie in the last share of a cluster's, or two of them in one thread's elements."""
    x, targets = logits(T, V, dtype, T, offset, spread=2.0)
    g = torch.Generator(device="cuda").manual_seed(V)
    kinds = torch.arange(T, device="cuda") % 7
    lift = torch.where(kinds == 1, 24.0, 0.0)[:, None].to(dtype)
    x.scatter_(1, targets[:, None], x.gather(1, targets[:, None]) + lift)
    for t in range(2, T, 7):
        x[t].masked_fill_(torch.rand(V, generator=g, device="cuda") < 0.999, -INF)
        x[t, int(targets[t])] = 1.0
    x[3::7] = x[3::7].float().round().to(dtype)
    x[4::7] = -1.5
    x[5::7, V - V // 9:] += 6.0
    gaps = apart(dtype, V)
    for n, t in enumerate(range(6, T, 7)):
        gap = gaps[n % len(gaps)]
        x[t] = -40.0
        x[t, :gap + 1:gap] = 3.7
    targets[::5] = -1
    return x, targets


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("threads,blocks,T,V", LAYOUTS)
def test_layouts(threads, blocks, T, V, dtype):
    if dtype is F32:
        V //= 2
    assert binding.token_logprobs_select_layout(dtype, T, V) == (threads, blocks)
    x, targets = varied(T, V, dtype, offset=V % 3)
    for k in (0, 5, 32):
        check(x, targets, k, what=f"k {k}", grad=k == 0)


@pytest.mark.parametrize("dtype,T,V", [(BF, 165, 2400001), (HALF, 160, 2400007), (F32, 158, 1200005)])
def test_clusters_that_take_several_rows(dtype, T, V):
    """No more than 152 clusters of 8 blocks of 256 threads fit on 152 SMs (2048 threads each), so
    some take a second row, into the other place for what a cluster knows; and a third
    (the first place again) where an SM holds half of that.  The same bits again."""
    assert binding.token_logprobs_select_layout(dtype, T, V) == (256, 8)
    x, targets = varied(T, V, dtype, offset=1)
    for k in (0, 20):
        got = check(x, targets, k, what=f"k {k}", grad=False)
        for _ in range(3):
            again = binding.token_logprobs_fwd(x, targets, top_k=k)
            assert all(torch.equal(a, b) for a, b in zip(got, again) if a is not None)


def test_query_refuses():
    for T, V in ((0, 100), (-1, 100), (5, 0), (1 << 28, 100), (5, (1 << 31) - 1)):
        with pytest.raises(RowNormError, match="sizes"):
            binding.token_logprobs_select_layout(BF, T, V)
    with pytest.raises(TypeError, match="logits"):
        binding.token_logprobs_select_layout(torch.float64, 5, 100)
