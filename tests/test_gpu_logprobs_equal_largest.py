"""Rows of logits whose two largest are equal and hold all of the probability (GPU)."""
from __future__ import annotations

import pytest
import torch

from row_normalization_gb300 import binding
from tests.axes_ref import U, assert_near
from tests.gpu_util import require_gpu
from tests.test_gpu_token_logprobs import DTYPES, INF, check

pytestmark = pytest.mark.gpu

THREADS = (64, 96, 128, 192, 256, 320, 512)  # of the blocks that rows are given


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    binding.device_status()


def apart(dtype, V):
    """Distances of two columns: in one granule of 16 bytes, and in granules that one thread
    of a block reads, of one batch (four granules of each thread), of the next and of the last."""
    per = 128 // torch.finfo(dtype).bits
    far = [1, per - 1] + [per * n * j for n in THREADS for j in (1, 3, 4, V // (per * n) - 1)]
    return [d for d in far if 0 < d < V]


def two_equal(T, V, dtype, scale, below, offset, seed):
    """x [T, V], `offset` elements from a 16-byte boundary: rows of two equal logits, others
    `below` under them; and their columns [T, 2]."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def pick(n):
        return torch.randint(0, n, (T,), generator=g, device="cuda")

    gap = torch.tensor(apart(dtype, V), device="cuda")
    gap = gap[pick(len(gap))]
    # anywhere, or with the second in the row's last columns, or the first in its first
    where, last = pick(4), V - 1 - gap
    first = torch.where(where == 0, last - pick(4).clamp(max=V - 2),
                        torch.where(where == 1, pick(4), pick(1 << 30) % (last + 1)))
    first = first.clamp(min=0).minimum(last)
    most = (torch.rand(T, generator=g, device="cuda") * 60 - 30).to(dtype)
    room = torch.zeros(T * V + offset, dtype=dtype, device="cuda")
    x = room[offset:].view(T, V)
    x.copy_((most.float() - below / scale)[:, None].expand(T, V))
    columns = torch.stack((first, first + gap), 1)
    x.scatter_(1, columns, most[:, None].expand(T, 2).contiguous())
    return x, columns


@pytest.mark.parametrize("below", [INF, 40.0])
@pytest.mark.parametrize("scale", [0.7, 1.0, 1.6])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,V", [(1, 2), (500, 2), (300, 9), (1, 50021), (20, 50021), (64, 131072), (100, 131072),
                                 (150, 50021), (333, 50000), (700, 20001), (1000, 7777), (1500, 9001), (2048, 8003),
                                 (4096, 515)])
def test_two_equal_logits_share_the_row(T, V, dtype, scale, below):
    """Each has probability 1/2: nothing is lost of the second, wherever the two lie."""
    for seed in range(max(1, 24 // T)):
        x, columns = two_equal(T, V, dtype, scale, below, seed % 2, seed)
        targets = columns[:, seed % 2].contiguous()
        got = check(x, targets, 2, scale, f"seed {seed}")
        assert torch.equal(got.top_ids, columns)
        # the gradient of the log probability is +-1/2 on the two.  p = e^(s - lse) with lse
        # rounded, and s - lse once more: (|lse| + 16) U of itself each
        dp = torch.linspace(0.5, 2.0, T, device="cuda")
        d = binding.token_logprobs_bwd(x, targets, got, dp, scale=scale).gather(1, columns)
        want = scale * dp.double()[:, None] * torch.where(columns == targets[:, None], 0.5, -0.5)
        assert_near(d, want, want.abs() * (2 * got.lse.abs().double()[:, None] + 32) * U, f"seed {seed} gradient")
