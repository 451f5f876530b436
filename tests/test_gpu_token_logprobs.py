"""Log probabilities of given tokens and their gradient against the 64-bit definitions (GPU)."""
from __future__ import annotations

import math

import pytest
import torch

from row_normalization_gb300 import binding
from row_normalization_gb300.binding import RN_STATUS_BAD_INDEX, RowNormError, TokenLogprobs
from tests import axes_ref
from tests.axes_ref import U, assert_near
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu

BF, HALF, F32 = torch.bfloat16, torch.float16, torch.float32
DTYPES = [BF, HALF, F32]
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    binding.device_status()


def logits(T, V, dtype, seed=0, offset=0, pad=0, spread=2.0):
    """[T, V] in a wider buffer, `offset` elements from a 16-byte boundary."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    room = torch.full((T * (V + pad) + offset + 8,), 55.0, dtype=dtype, device="cuda")
    x = room[offset:offset + T * (V + pad)].view(T, V + pad)[:, :V]
    x.copy_(torch.randn(T, V, generator=g, device="cuda") * spread)
    return x, torch.randint(0, V, (T,), generator=g, device="cuda")


def upstream(T, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 100)
    return [torch.randn(T, generator=g, device="cuda") for _ in range(3)]


def check(x, targets, k=0, scale=1.0, what="", grad=True):
    got = binding.token_logprobs_fwd(x, targets, scale=scale, top_k=k)
    want, slack = axes_ref.logprobs(x, targets, scale, k)
    for name, a, b, s in zip(("logprobs", "lse", "entropy", "top_logprobs"), got, want, slack):
        if a is not None:
            assert_near(a, b, s, f"{what} {name}")
    if k:
        assert torch.equal(got.top_ids, want[4]), f"{what}: top_ids"
    else:
        assert got.top_ids is None and got.top_logprobs is None
    if grad:
        check_grad(x, targets, got, scale, what)
    assert binding.device_status() == 0
    return got


def check_grad(x, targets, forward, scale, what, ups=None):
    dp, dh, dl = upstream(x.shape[0]) if ups is None else ups
    want, slack = axes_ref.logprobs_grad(x, targets, *forward[:3], dp, dh, dl, scale)
    got = binding.token_logprobs_bwd(x, targets, forward, dp, dh, dl, scale=scale)
    assert got.dtype == x.dtype and got.shape == x.shape
    assert_near(got, want, slack, f"{what} dlogits")
    return got


@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 31, 33, 511, 4095, 4096, 4097, 8200, 50021])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,offset,pad", [(1, 0, 0), (3, 1, 0), (5, 3, 5)])
def test_sizes_and_alignments(V, dtype, T, offset, pad):
    x, targets = logits(T, V, dtype, V, offset, pad)
    check(x, targets, min(V, 20), what=f"V {V}")


@pytest.mark.parametrize("T,V", [(17, 131072), (64, 32768), (128, 131072), (200, 40003), (200, 131072), (300, 9001),
                                 (333, 50000), (500, 30011), (700, 4096), (1000, 7777), (1300, 20001), (2000, 1000),
                                 (3000, 2000), (5000, 515)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_row_counts(T, V, dtype):
    """Rows shared by clusters of every size, rows of blocks of every size, and blocks that
    take several rows one after another."""
    x, targets = logits(T, V, dtype, 1, pad=V % 8)
    check(x, targets, 8, what=f"T {T} V {V}")


@pytest.mark.parametrize("k", [0, 1, 2, 31, 32])
@pytest.mark.parametrize("scale", [0.25, 1.0, 3.7])
def test_alternatives_and_temperatures(k, scale):
    x, targets = logits(40, 12345, BF, 2)
    check(x, targets, k, scale, f"k {k} scale {scale}")


@pytest.mark.parametrize("T", [1, 400, 1500])
def test_rows_of_equal_logits(T):
    """All equal: a uniform distribution, the lowest columns first."""
    x = torch.full((T, 10007), -3.25, dtype=BF, device="cuda")
    got = check(x, torch.full((T,), 9999, device="cuda"), 32, what="equal")
    assert (got.top_ids == torch.arange(32, device="cuda")).all()


@pytest.mark.parametrize("T", [2, 1500])
@pytest.mark.parametrize("dtype", DTYPES)
def test_few_values_and_signed_zeros(T, dtype):
    """Ties everywhere; -0 equals 0."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randint(0, 3, (T, 9000), generator=g, device="cuda").to(dtype) - 2
    flip = torch.rand(T, 9000, generator=g, device="cuda") < 0.5
    x = torch.where((x == 0) & flip, torch.tensor(-0.0, dtype=dtype, device="cuda"), x)
    targets = torch.randint(0, 9000, (T,), generator=g, device="cuda")
    got = check(x, targets, 20, what="few values")
    first = torch.sort((x == 0).int(), dim=1, descending=True, stable=True).indices[:, :20]
    assert torch.equal(got.top_ids, first)


# rows, and the threads of a block that so many rows of concentrated()'s length are given
LAYOUTS = [(1, 256), (20, 256), (150, 512), (333, 320), (700, 192), (1000, 128), (1500, 96), (2048, 64)]


def concentrated(T, threads, dtype):
    """[T, V] and its view by the groups of 16 bytes that a block's threads take in turn, 48
    each (so that one thread may have more candidates than are listed)."""
    per = 128 // torch.finfo(dtype).bits
    x = torch.zeros(T, per * threads * 48, dtype=dtype, device="cuda")
    return x, x.view(T, -1, threads, per), torch.Generator(device="cuda").manual_seed(4)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,threads", LAYOUTS)
def test_large_logits_that_one_thread_meets(T, threads, dtype):
    """More candidates than the list holds, in the columns that a single thread of the
    block reads, in all orders."""
    x, view, g = concentrated(T, threads, dtype)
    view[:, :, 3] = (torch.rand(T, view.shape[1], view.shape[3], generator=g, device="cuda") * 8 + 1).to(dtype)
    targets = torch.randint(0, x.shape[1], (T,), generator=g, device="cuda")
    check(x, targets, 32, what="one thread", grad=T < 100)
    check(x, targets, 1, what="one thread, one alternative", grad=False)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,threads", LAYOUTS)
def test_many_equal_and_a_few_threads_with_more(T, threads, dtype):
    """Fewer threads than k above a value that many threads share, some with many columns
    above it, and one with more than the list holds."""
    x, view, _ = concentrated(T, threads, dtype)
    x.fill_(-1.0)
    view[:, ::9, 50, 2] = 2.0
    view[:, 5, 7, 0] = 3.0
    targets = torch.full((T,), 5, device="cuda")
    check(x, targets, 32, what="many equal", grad=False)
    view[:, :, 9] = 0.5
    check(x, targets, 32, what="many equal, a full list", grad=False)
    x[:, ::2] = -INF
    check(x, targets.fill_(1), 32, what="many equal, half banned", grad=False)


@pytest.mark.parametrize("k", [1, 31, 32])
@pytest.mark.parametrize("T,V", [(1, 131072), (1000, 32000), (2048, 32000), (3000, 5000)])
def test_more_runs_reach_than_are_listed(T, V, k):
    """Values that fall along the row, so that every thread's first are near the largest."""
    x = (-torch.arange(V, device="cuda") / 64).bfloat16().repeat(T, 1)
    check(x, torch.full((T,), V // 2, device="cuda"), k, what="falling slowly", grad=False)


@pytest.mark.parametrize("rising", [True, False])
@pytest.mark.parametrize("dtype", DTYPES)
def test_rising_and_falling_rows(rising, dtype):
    """Every granule raises the running maximum, or none does."""
    x = torch.linspace(-20, 20, 30011, device="cuda").to(dtype).repeat(3, 1)
    if not rising:
        x = x.flip(1).contiguous()
    check(x, torch.tensor([0, 15000, 30010], device="cuda"), 20, what="rising" if rising else "falling")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,V", [(4, 33333), (1200, 5003)])
def test_tokens_that_are_nearly_sure(T, V, dtype):
    """1 - p keeps its precision: logprobs, entropy and gradient down to 2^-24 and below."""
    x, targets = logits(T, V, dtype, 5, spread=1.0)
    lift = torch.linspace(8, 40, T, device="cuda")[:, None]
    x.scatter_(1, targets[:, None], lift.to(dtype))
    got = check(x, targets, 3, what="sure")
    assert (got.logprobs < 0).all() and (got.entropy > 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,V,left", [(3, 20000, 5), (3, 131072, 200), (1300, 4001, 1), (40, 9000, 31)])
def test_banned_tokens(T, V, dtype, left):
    """-infinity in all but `left` columns, fewer of them than alternatives wanted."""
    x, _ = logits(T, V, dtype, 6, offset=1)
    g = torch.Generator(device="cuda").manual_seed(7)
    kept = torch.stack([torch.randperm(V, generator=g, device="cuda")[:left] for _ in range(T)])
    mask = torch.ones(T, V, dtype=torch.bool, device="cuda").scatter_(1, kept, False)
    x.masked_fill_(mask, -INF)
    targets = kept[:, 0].contiguous()
    targets[0] = int(mask[0].int().argmax())              # a banned one
    got = check(x, targets, 32, what="banned")
    assert got.logprobs[0] == -INF and (got.logprobs[1:] > -INF).all()
    dp, dh, dl = upstream(T)
    d = binding.token_logprobs_bwd(x, targets, got, dp, dh, dl)
    mask.scatter_(1, targets[:, None], False)
    assert (d[mask] == 0).all() and d.isfinite().all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,V", [(2, 30000), (1300, 700)])
def test_rows_of_banned_tokens_alone(T, V, dtype):
    x = torch.full((T, V), -INF, dtype=dtype, device="cuda")
    x[1:, 3] = 1.0
    targets = torch.zeros(T, dtype=torch.int64, device="cuda") + 3
    got = binding.token_logprobs_fwd(x, targets, top_k=4)
    assert got.lse[0] == -INF and got.logprobs[0] == -INF and got.entropy[0] == 0
    assert (got.top_logprobs[0] == -INF).all() and got.top_ids[0].tolist() == [0, 1, 2, 3]
    assert (got.lse[1:] == 1).all() and (got.logprobs[1:] == 0).all() and (got.entropy[1:] == 0).all()
    assert got.top_ids[1].tolist() == [3, 0, 1, 2]
    d = binding.token_logprobs_bwd(x, targets, got, *upstream(T))
    assert (d[0] == 0).all() and d.isfinite().all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("at", [0, 7777, 9998])
@pytest.mark.parametrize("T", [4, 1300])
def test_infinities_and_nan(T, at, dtype):
    x, _ = logits(T, 9999, dtype, 8, offset=1)
    targets = torch.full((T,), at, device="cuda")
    x[1, at], x[2, at] = INF, NAN
    got = binding.token_logprobs_fwd(x, targets, top_k=3)
    assert got.lse[1] == INF and got.logprobs[1].isnan() and got.entropy[1].isnan()
    assert got.top_ids[1, 0] == at and got.top_logprobs[1, 0].isnan() and (got.top_logprobs[1, 1:] == -INF).all()
    assert got.lse[2].isnan() and got.logprobs[2].isnan() and got.entropy[2].isnan()
    assert got.top_ids[2, 0] == at and got.top_logprobs[2].isnan().all()
    rest = [0, 3] + list(range(4, T))
    want, slack = axes_ref.logprobs(x[rest], targets[rest], 1.0, 3)
    for a, b, s in zip(got, want, slack):
        assert_near(a[rest], b, s, "beside")
    assert torch.equal(got.top_ids[rest], want[4])
    # the other columns of a row with +infinity are impossible
    other = binding.token_logprobs_fwd(x, targets * 0 + 5)
    assert other.logprobs[1] == -INF and other.logprobs[2].isnan()
    for ups in (upstream(T), [upstream(T)[0], None, None]):
        d = binding.token_logprobs_bwd(x, targets, got, *ups)
        assert d[1].isnan().all() and d[2].isnan().all() and d[rest].isfinite().all()


def test_targets_that_are_ignored_or_outside():
    x, targets = logits(6, 3001, BF, 9)
    targets[1], targets[2] = -1, -100
    got = check(x, targets, what="ignored")
    assert (got.logprobs[1:3] == 0).all() and (got.lse[1:3] > 0).all()
    targets[4], targets[5] = 3001, 1 << 40
    got = binding.token_logprobs_fwd(x, targets)
    assert got.logprobs[4:].isnan().all() and got.logprobs[:4].isfinite().all() and got.lse.isfinite().all()
    assert binding.device_status() == RN_STATUS_BAD_INDEX
    dp, dh, dl = upstream(6)
    d = binding.token_logprobs_bwd(x, targets, got, dp, dh, dl)
    assert d[4:].isnan().all() and d[:4].isfinite().all()
    assert binding.device_status() == RN_STATUS_BAD_INDEX
    # without a gradient of log probabilities targets are not looked at
    assert binding.token_logprobs_bwd(x, targets, got, None, dh, dl).isfinite().all()
    assert binding.device_status() == 0


@pytest.mark.parametrize("dtype", DTYPES)
def test_logits_far_from_zero(dtype):
    """Differences count, not sizes: up to the ends of the format."""
    big = {BF: 1e38, HALF: 3e4, F32: 3e38}[dtype]
    x, targets = logits(4, 5000, dtype, 10)
    x[0] += 96
    x[1] -= 1000
    x[2, ::2] = big
    x[2, 1::2] = -big
    x[3] = -big
    check(x, targets, 5, what="far")


@pytest.mark.parametrize("dtype", DTYPES)
def test_gradients_alone_expanded_strided_and_none(dtype):
    x, targets = logits(7, 2999, dtype, 11)
    fwd = binding.token_logprobs_fwd(x, targets)
    dp, dh, dl = upstream(7)
    one = torch.tensor(-0.25, device="cuda").expand(7)
    wide = torch.randn(7, 3, device="cuda")[:, 1]
    for ups in ([dp, None, None], [None, dh, None], [None, None, dl], [one, wide, one], [None, None, None]):
        got = check_grad(x, targets, fwd, 1.0, "alone", ups)
        assert ups != [None] * 3 or (got == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("offset,pad,out_offset,out_pad", [(0, 0, 0, 0), (1, 0, 1, 0), (1, 2, 3, 0), (0, 3, 2, 6)])
def test_gradient_in_place_and_into_other_layouts(dtype, offset, pad, out_offset, out_pad):
    T, V = 9, 5001
    x, targets = logits(T, V, dtype, 12, offset, pad)
    fwd = binding.token_logprobs_fwd(x, targets)
    ups = upstream(T)
    want = binding.token_logprobs_bwd(x, targets, fwd, *ups)
    room = torch.full((T * (V + out_pad) + out_offset + 8,), 55.0, dtype=dtype, device="cuda")
    out = room[out_offset:out_offset + T * (V + out_pad)].view(T, V + out_pad)[:, :V]
    assert binding.token_logprobs_bwd(x, targets, fwd, *ups, dlogits=out) is out
    assert torch.equal(out, want)
    assert int((room != 55.0).sum()) <= T * V
    rest = torch.ones_like(room, dtype=torch.bool)
    rest[out_offset:out_offset + T * (V + out_pad)].view(T, V + out_pad)[:, :V] = False
    assert (room[rest] == 55.0).all()
    assert binding.token_logprobs_bwd(x, targets, fwd, *ups, dlogits=x) is x
    assert torch.equal(x, want)


def test_rows_behind_the_last_stay_as_they_were():
    x, targets = logits(5, 1000, BF, 13)
    full = [torch.full((9,), 5.0, device="cuda") for _ in range(3)]
    top, ids = torch.full((9, 4), 5.0, device="cuda"), torch.full((9, 4), 5, device="cuda")
    binding.token_logprobs_fwd(x, targets, top_k=4, logprobs=full[0][:5], lse=full[1][:5], entropy=full[2][:5],
                               top_logprobs=top[:5], top_ids=ids[:5])
    torch.cuda.synchronize()
    for t in (*full, top, ids):
        assert (t[5:] == 5).all() and not (t[:5] == 5).all()


def test_rows_beyond_32_bits():
    """Row offsets past 2^32 elements, and a row of 2^31 - 65 columns."""
    if torch.cuda.get_device_properties(0).total_memory < 100e9:
        pytest.skip("needs 100 GB")
    stride = (1 << 31) + 5
    far = torch.empty(2 * stride + 5000, dtype=BF, device="cuda").as_strided((3, 4097), (stride, 1))
    near, targets = logits(3, 4097, BF, 14)
    far.copy_(near)
    check(far, targets, 5, what="far rows")
    del far
    V = (1 << 31) - 65
    x = torch.zeros(1, V, dtype=BF, device="cuda")
    x[0, V - 1], x[0, 12345] = 20.0, 21.0
    targets = torch.tensor([V - 1], device="cuda")
    got = binding.token_logprobs_fwd(x, targets, top_k=4)
    assert got.top_ids[0].tolist() == [12345, V - 1, 0, 1]
    z = (V - 2) * math.exp(-21.0) + math.exp(-1.0) + 1.0
    # a thread adds 2^19 terms of one size (in fp32 sums of 2^-30 each: at most half of a
    # sum's unit, so 2^-5 of it if every rounding went one way)
    assert abs(float(got.lse[0]) - (21.0 + math.log(z))) <= 2.0 ** -5
    d = binding.token_logprobs_bwd(x, targets, got, dlogprobs=torch.ones(1, device="cuda"), dlogits=x)
    assert abs(float(d[0, V - 1]) - (1 - math.exp(-1.0) / z)) <= 2.0 ** -6
    assert float(d[0, 77]) < 0


def test_two_calls_at_once():
    """Calls on two streams share nothing."""
    a, ta = logits(1500, 30000, BF, 20)
    b, tb = logits(900, 50001, HALF, 21)
    want = [binding.token_logprobs_fwd(a, ta, top_k=5), binding.token_logprobs_fwd(b, tb, top_k=20)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(4):
        got = [binding.token_logprobs_fwd(x, t, top_k=k, stream=s)
               for (x, t, k), s in zip(((a, ta, 5), (b, tb, 20)), streams)]
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            for p, q in zip(w, g):
                assert torch.equal(p, q)


def test_scales_whose_powers_leave_the_format():
    """Temperatures so high that no fp16 or bf16 logit is out of reach of the largest, and so
    low that all but the largest are."""
    for dtype in DTYPES:
        x, targets = logits(5, 9000, dtype, 22)
        for scale in (1e-30, 1e-6, 1e-3, 0.003, 300.0, 1e20):
            check(x, targets, 7, scale, f"scale {scale}", grad=scale < 1e3)
        x[:, ::3] = -INF
        targets = targets // 3 * 3 + 1
        for scale in (1e-30, 1e-3, 300.0):
            check(x, targets, 7, scale, f"banned, scale {scale}")


def test_same_bits_again_and_beside_other_work():
    x, targets = logits(500, 30000, BF, 15)
    first = binding.token_logprobs_fwd(x, targets, top_k=20)
    side = torch.cuda.Stream()
    noise = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(side):
            noise = noise @ noise * 1e-3
        again = binding.token_logprobs_fwd(x, targets, top_k=20)
        for a, b in zip(first, again):
            assert torch.equal(a, b)
    torch.cuda.synchronize()


def test_captured_and_replayed():
    x, targets = logits(40, 20000, BF, 16)
    dp, dh, dl = upstream(40)
    d = torch.empty_like(x)

    def step(out=None):
        f = binding.token_logprobs_fwd(x, targets, top_k=5, **(out or {}))
        return f, binding.token_logprobs_bwd(x, targets, f, dp, dh, dl, dlogits=d)

    f, _ = step()
    out = dict(f._asdict())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(out)
    y, t2 = logits(40, 20000, BF, 17)
    x.copy_(y)
    targets.copy_(t2)
    graph.replay()
    torch.cuda.synchronize()
    kept = [v.clone() for v in out.values()] + [d.clone()]
    f, _ = step()
    for a, b in zip(kept, [*f, d]):
        assert torch.equal(a, b)


def test_on_another_stream_with_results_made_for_it():
    x, targets = logits(300, 30000, BF, 18)
    want = binding.token_logprobs_fwd(x, targets, top_k=7)
    dwant = binding.token_logprobs_bwd(x, targets, want, *upstream(300))
    side = torch.cuda.Stream()
    ups = upstream(300)
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        got = binding.token_logprobs_fwd(x, targets, top_k=7, stream=stream)
        d = binding.token_logprobs_bwd(x, targets, got, *ups, stream=stream)
        side.synchronize()
        for a, b in zip((*want, dwant), (*got, d)):
            assert torch.equal(a, b)


def test_one_column_of_any_stride():
    x = torch.randn(1, 5, device="cuda", dtype=F32).t()  # [5, 1]
    assert x.stride() == (1, 5)
    got = check(x, torch.zeros(5, dtype=torch.int64, device="cuda"), k=1, what="one column")
    assert (got.logprobs == 0).all() and (got.entropy == 0).all() and (got.top_ids == 0).all()


def test_no_rows():
    x = torch.empty(0, 100, dtype=BF, device="cuda")
    t = torch.empty(0, dtype=torch.int64, device="cuda")
    got = binding.token_logprobs_fwd(x, t, top_k=3)
    assert got.logprobs.shape == (0,) and got.top_ids.shape == (0, 3)
    assert binding.token_logprobs_bwd(x, t, got, *upstream(0)).shape == (0, 100)


def test_refusals_of_the_binding():
    x, targets = logits(3, 100, BF)
    got = binding.token_logprobs_fwd(x, targets)
    with pytest.raises(TypeError, match="logits"):
        binding.token_logprobs_fwd(x.double(), targets)
    with pytest.raises(ValueError, match="logits"):
        binding.token_logprobs_fwd(x[0], targets)
    with pytest.raises(ValueError, match="contiguous rows"):
        binding.token_logprobs_fwd(x.t(), torch.zeros(100, dtype=torch.int64, device="cuda"))
    with pytest.raises(TypeError, match="targets"):
        binding.token_logprobs_fwd(x, targets.int())
    with pytest.raises(ValueError, match="targets"):
        binding.token_logprobs_fwd(x, targets[:2])
    with pytest.raises(ValueError, match="top_k"):
        binding.token_logprobs_fwd(x, targets, top_ids=targets)
    for kw in ({"top_k": 33}, {"top_k": -1}, {"scale": 0.0}, {"scale": -2.0}, {"scale": float("nan")}):
        with pytest.raises(RowNormError):
            binding.token_logprobs_fwd(x, targets, **kw)
    with pytest.raises(RowNormError, match="sizes"):
        binding.token_logprobs_fwd(x[:, :3], targets, top_k=4)
    with pytest.raises(ValueError, match="dentropy"):
        binding.token_logprobs_bwd(x, targets, got, None, torch.zeros(4, device="cuda"))
    with pytest.raises(ValueError, match="dlogprobs"):
        binding.token_logprobs_bwd(x, targets, got, torch.zeros(3, device="cuda").double())
    with pytest.raises(TypeError, match="dlogits"):
        binding.token_logprobs_bwd(x, targets, got, dlogits=x.float())
    with pytest.raises(RowNormError, match="sizes"):
        binding.token_logprobs_bwd(x, targets, got, dlogits=x[:1].expand(3, 100))


def test_the_gradient_is_the_kernel_forward_s_differences():
    """fp32 logits, steps of 2^-5: third derivatives of log probability and entropy are
    below 4, so differences are within 2^-11 of the derivative; results of order 4 off by
    2^-20 at most each leave 2^-14 of a difference."""
    x, targets = logits(3, 200, F32, 19)
    dp, dh, dl = upstream(3)
    got = binding.token_logprobs_bwd(x, targets, binding.token_logprobs_fwd(x, targets), dp, dh, dl)
    h = 2.0 ** -5
    for v in list(range(0, 200, 17)) + targets.tolist():
        f = []
        for sign in (1, -1):
            y = x.clone()
            y[:, v] += sign * h
            r = binding.token_logprobs_fwd(y, targets)
            f.append((r.logprobs * dp + r.entropy * dh + r.lse * dl).double())
        moved = ((x[:, v] + h) - (x[:, v] - h)).double()
        d = (f[0] - f[1]) / moved
        scale = dp.abs() + dh.abs() + dl.abs()
        assert ((d - got[:, v].double()).abs() <= scale * (2.0 ** -11 + 2.0 ** -13)).all()
