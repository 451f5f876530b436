"""Rows masked by the format's lowest value instead of -infinity (GPU)."""
from __future__ import annotations

import math

import pytest
import torch

from row_normalization_gb300 import binding
from tests import axes_ref
from tests.axes_ref import U, assert_near
from tests.gpu_util import require_gpu
from tests.test_gpu_token_logprobs import DTYPES, INF, logits, upstream

pytestmark = pytest.mark.gpu

SCALES = [0.25, 0.7, 1.0, 1.6, 2.0, 3.7]  # above 1 the lowest values leave fp32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    binding.device_status()


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,V,offset", [(3, 5001, 0), (40, 20011, 1), (1300, 700, 0)])
def test_rows_of_nothing_else(T, V, offset, dtype, scale):
    """A padded row whose mask leaves nothing: uniform, and a finite gradient; none where
    nothing comes back for it.

    A thread adds 40 equal terms at most in each of its sums, joins and the power that they
    share add 20: Z is off by 60 U, and ln V is 6 or more."""
    x, targets = logits(T, V, dtype, 1, offset)
    x.fill_(torch.finfo(dtype).min)
    targets[::3] = -1
    got = binding.token_logprobs_fwd(x, targets, scale=scale, top_k=2)
    want = torch.full((T,), -math.log(V), device="cuda", dtype=torch.float64).masked_fill(targets < 0, 0.0)
    assert_near(got.logprobs, want, 64 * U * math.log(V), "logprobs")
    assert_near(got.entropy, torch.full_like(want, math.log(V)), 64 * U * math.log(V), "entropy")
    assert (got.top_ids == torch.arange(2, device="cuda")).all()
    s = float(torch.tensor(scale, dtype=torch.float32)) * torch.finfo(dtype).min
    if s < torch.finfo(torch.float32).min:
        assert (got.lse == -INF).all()
    else:
        assert_near(got.lse, torch.full_like(want, s + math.log(V)), 2 * U * abs(s), "lse")
    ups = upstream(T)
    d = binding.token_logprobs_bwd(x, targets, got, *ups, scale=scale)
    # p is between 0 and 1, l = ln p below 0, p |l| at most 1/e; one rounding, and 64 U of each part
    dp, dh, dl = (v.abs().double() for v in ups)
    most = scale * (dp + dl + dh * (math.log(V) + 1 / math.e)) * (1 + axes_ref.half(dtype) + 64 * U)
    assert d.isfinite().all() and (d.double().abs() <= most[:, None]).all()
    d = binding.token_logprobs_bwd(x, targets, got, ups[0], scale=scale)
    assert (d[::3] == 0).all() and d.isfinite().all()
    assert binding.device_status() == 0


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,V,offset", [(3, 5001, 0), (40, 20011, 1), (1300, 700, 0)])
def test_rows_that_are_masked_in_part(T, V, offset, dtype, scale):
    """The lowest value beside others: probability 0, as -infinity."""
    x, targets = logits(T, V, dtype, 2, offset)
    g = torch.Generator(device="cuda").manual_seed(3)
    mask = torch.rand(T, V, generator=g, device="cuda") < 0.9
    mask.scatter_(1, targets[:, None], False)
    scale = float(torch.tensor(scale, dtype=torch.float32))
    banned = x.masked_fill(mask, -INF)
    x.masked_fill_(mask, torch.finfo(dtype).min)
    got = binding.token_logprobs_fwd(x, targets, scale=scale)
    ups = upstream(T)
    d = binding.token_logprobs_bwd(x, targets, got, *ups, scale=scale)
    want, slack = axes_ref.logprobs(banned, targets, scale, 0)
    for a, b, s in zip(got[:3], want, slack):
        assert_near(a, b, s, "forward")
    want, slack = axes_ref.logprobs_grad(banned, targets, *got[:3], *ups, scale)
    assert_near(d, want, slack, "dlogits")
    assert (d[mask] == 0).all()
