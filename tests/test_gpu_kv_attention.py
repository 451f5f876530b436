"""Attention over the quantised key/value cache (GPU) against its 64-bit definition.

Tolerance of an output element (derived, nothing fitted):
  * the result is rounded once to bf16: eps/2 * |out|;
  * a weight p and its product with a value scale are each rounded to fp16, whose
    half step is 2^-11 relative (11 significant bits): together (1 + 2^-11)^2 - 1,
    2^-10 * sum w |v| with the factor 1.01 below.  What falls below fp16's normal
    range, 2^-28 of the largest weight, is off by 2^-39 of it at most: n * 2^-39
    of the value's range, nothing beside the first term for the lengths here;
  * the second product sums stored codes 0 .. 2z (z = 8 or 128, the codes' offset),
    whose offset is taken off at the end, so the rounding of its fp32 sums goes by
    2z * sum w s.  One instruction adds 17 numbers, each cut to the largest one's 24
    bits (17 * 2^-24); the caches here have fewer than 4 * 4 * 304 tiles, so a warp
    takes two tiles of two instructions at most, and fewer than 200 partial sums are
    joined by fused multiply-adds: together under 300 * 2^-24;
  * a logit's group sum takes two such instructions over q * code, with z * sum q
    taken off: 34 * 2^-24 * s * max(2z max|q|, z |sum q|) a group, then D / 32 fused
    multiply-adds and two roundings: 10 * 2^-24 * sum |q k|, all times the scale.  A
    logit moves a weight by that fraction and the weights' sum by the same: twice it;
  * exp2 and the running sums: 2^-20.
More than 64 columns (queries times heads of a group) run on restored fp16 values,
rounded once (2^-11), and weights rounded once: the output's 2^-10 is the same.  Keys
are restored as fp16 and the rest, itself fp16: off by 2^-22 |k| or, where the rest is
subnormal, 2^-25 an element; their products are summed D / 8 instructions long, 17 *
2^-24 of the largest partial sum each, sum |q k| at most.  Where a scale exceeds 255 the
32 tokens around it are restored at 2^-8 of their size, so that small scales among them
are rounded as subnormal numbers: 2^-25 * 2^8 a unit of the code, z a unit at most.
lse: the logit's error plus 2^-20 plus 2^-22 |lse|.
"""
from __future__ import annotations

import copy
import math

import pytest
import torch

from row_normalization_gb300 import binding
from row_normalization_gb300.inputs import qkv_inputs
from tests import kv_ref
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu

EPS = torch.finfo(torch.bfloat16).eps / 2
EXTRA_TOKENS = 0  # room in the page tables behind the longest sequence


@pytest.fixture(params=["direct", "line"])
def both_layouts(request, monkeypatch):
    """Short page tables give every head a CTA of its own; longer ones (here by entries
    that are no pages) the line of units and the joining kernel."""
    monkeypatch.setattr("tests.test_gpu_kv_attention.EXTRA_TOKENS",
                        2560 if request.param == "line" else 0)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    binding.device_status()


def to_gpu(ref):
    return binding.KVCache(ref.codes.cuda(), ref.scales.cuda())


def filled(bits, Hkv, D, P, lens, seed, spread=1.0, spare=2):
    """A cache holding `lens` tokens a sequence on shuffled pages; what no token
    wrote is NaN, and the table's unused entries are no pages."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // P) for n in lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g)
    table = torch.full((len(lens), max(need + [1]) + 1 + EXTRA_TOKENS // P), -1, dtype=torch.int32)
    ref = kv_ref.Cache(pages, Hkv, D, P, bits)
    at = 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]].int()
        at += need[b]
        if n:
            x = torch.randn(n, 2, Hkv, D, generator=g)
            x *= torch.exp(math.log(spread) * torch.randn(n, 2, Hkv, 1, generator=g))
            pos = torch.arange(n)
            ref.write(x.to(torch.bfloat16), table[b, pos // P].long() * P + pos % P)
    return ref, table


def queries(T, Hq, D, seed, size=1.5):
    g = torch.Generator().manual_seed(seed + 1000)
    return (size * torch.randn(T, Hq, D, generator=g)).to(torch.bfloat16)


def check(got, lse, q, ref, table, lens, cu, scale, window=0, sinks=0, wide=None):
    D = q.shape[-1]
    for b, n in enumerate(lens):
        lo, hi = cu[b], cu[b + 1]
        if lo == hi:
            continue
        K, V = (ref.tokens(table[b], w, 0, n) for w in (0, 1))
        # tokens no query sees may sit on pages that are gone
        o, l, weights = kv_ref.attention(q[lo:hi], K, V, n, scale, window, sinks)
        SK, SV = (ref.token_scales(table[b], w, 0, n) for w in (0, 1))
        z = 8 if ref.bits == 4 else 128
        G = q.shape[1] // K.shape[1]
        if wide is None:  # the arithmetic of more than 64 columns
            wide = max(y - x for x, y in zip(cu, cu[1:])) * G > 64
        low_k, low_v = (z * 2.0 ** -17 * float((x > 255).any()) * wide for x in (SK, SV))
        low_k += 2.0 ** -25 * wide
        tol, dl = torch.full_like(o, 2.0 ** -40), torch.zeros_like(l)
        for i in range(hi - lo):
            for h in range(q.shape[1]):
                if weights[i][h] is None:
                    continue
                js, w = weights[i][h]
                x = q[lo + i, h].double()
                k, sk = K[js, h // G], SK[js, h // G]
                grp = x.view(-1, 32)
                per = torch.maximum(2 * z * grp.abs().amax(1), z * grp.sum(1).abs())
                e = 34 * (sk[:, ::32] @ per) + 10 * (k.abs() @ x.abs())
                if wide:
                    e = (17 * D / 8 + 10) * (k.abs() @ x.abs())
                e = e * 2.0 ** -24 + wide * 2.0 ** -22 * (k.abs() @ x.abs())
                dlogit = float(e.max() + low_k * x.abs().sum()) * abs(scale)
                dl[i, h] = dlogit
                tol[i, h] += (2.0 ** -10 + 2 * dlogit + 2.0 ** -20) * 1.01 * (w @ V[js, h // G].abs())
                tol[i, h] += 300 * 2.0 ** -24 * 2 * z * (w @ SV[js, h // G]) + low_v
        tol += EPS * o.abs()
        err = (got[lo:hi].double() - o).abs()
        assert (err <= tol).all(), (b, n, float((err / tol).max()))
        g = lse[lo:hi].double()
        assert torch.equal(torch.isinf(g), torch.isinf(l))
        ok = ~torch.isinf(l)
        assert ((g - l)[ok].abs() <= dl[ok] + 2.0 ** -20 + 2.0 ** -22 * l[ok].abs()).all()


def attend(ref, table, lens, q, n_q, Hq, scale=None, **kw):
    T = sum(n_q)
    cu = [0]
    for n in n_q:
        cu.append(cu[-1] + n)
    out, lse = binding.kv_attention_fwd(
        q.cuda(), to_gpu(ref), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), Hq,
        cu_q=torch.tensor(cu).cuda(), max_q_len=max(n_q + [1]), scale=scale, **kw)
    assert out.shape == (q.shape[0], Hq, ref.D) and T <= q.shape[0]
    return out.cpu(), lse.cpu(), cu


LAYOUTS = [(4, 1, 64, 16), (6, 2, 128, 32), (8, 8, 64, 64), (32, 8, 128, 64), (5, 1, 256, 16),
           (16, 2, 256, 128), (9, 1, 128, 256), (48, 1, 64, 32), (20, 1, 128, 16)]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("Hq,Hkv,D,P", LAYOUTS)
@pytest.mark.usefixtures("both_layouts")
def test_one_token_ragged_lengths(bits, Hq, Hkv, D, P):
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 64, 127, 130, 257]
    ref, table = filled(bits, Hkv, D, P, lens, seed=D + P)
    q = queries(len(lens), Hq, D, seed=Hq)
    out, lse = binding.kv_attention_fwd(q.cuda(), to_gpu(ref), table.cuda(),
                                        torch.tensor(lens, dtype=torch.int32).cuda(), Hq)
    check(out.cpu(), lse.cpu(), q, ref, table, lens, list(range(len(lens) + 1)), D ** -0.5)
    assert binding.device_status() == 0


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("Hq,Hkv,D,P", LAYOUTS)
@pytest.mark.usefixtures("both_layouts")
def test_several_queries_a_sequence(bits, Hq, Hkv, D, P):
    lens, n_q = [5, 40, 33, 100, 64, 7], [5, 3, 0, 17, 1, 2]
    ref, table = filled(bits, Hkv, D, P, lens, seed=D + P + 1)
    q = queries(sum(n_q), Hq, D, seed=Hq)
    out, lse, cu = attend(ref, table, lens, q, n_q, Hq)
    check(out, lse, q, ref, table, lens, cu, D ** -0.5)
    assert binding.device_status() == 0


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (33, 0), (64, 40), (100, 3),
                                          (10 ** 6, 2)])
@pytest.mark.parametrize("Hq,Hkv,D,P,bits", [(8, 2, 128, 16, 4), (4, 4, 64, 64, 8),
                                             (12, 1, 256, 32, 4)])
@pytest.mark.usefixtures("both_layouts")
def test_window_and_sinks(window, sinks, Hq, Hkv, D, P, bits):
    lens, n_q = [1, 20, 90, 200, 333], [1, 7, 1, 30, 2]
    ref, table = filled(bits, Hkv, D, P, lens, seed=window + sinks)
    q = queries(sum(n_q), Hq, D, seed=3)
    out, lse, cu = attend(ref, table, lens, q, n_q, Hq, window=window, sinks=sinks)
    check(out, lse, q, ref, table, lens, cu, D ** -0.5, window, sinks)
    assert binding.device_status() == 0


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.usefixtures("both_layouts")
def test_tokens_behind_the_window_are_never_used(bits):
    """Their pages hold NaN scales or are gone from the table: nothing changes."""
    Hq, Hkv, D, P, window, sinks = 8, 2, 128, 16, 50, 3
    lens, n_q = [300], [9]
    ref, table = filled(bits, Hkv, D, P, lens, seed=8)
    q = queries(9, Hq, D, seed=4)
    out, lse, cu = attend(ref, table, lens, q, n_q, Hq, window=window, sinks=sinks)
    check(out, lse, q, ref, table, lens, cu, D ** -0.5, window, sinks)
    first = lens[0] - n_q[0] - window + 1                   # the first token a window reaches
    for j in range(sinks, first):
        pg, off = int(table[0, j // P]), j % P
        ref.scales[pg, :, :, off] = float("nan")
        ref.codes[pg, :, :, off] = 0xFF
    gone = table.clone()
    gone[0, 1:first // P] = -5
    again, lse2, _ = attend(ref, gone, lens, q, n_q, Hq, window=window, sinks=sinks)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    assert binding.device_status() == 0


@pytest.mark.usefixtures("both_layouts")
def test_rows_that_see_nothing():
    """More queries than cached tokens, and an empty cache: 0 and -inf."""
    Hq, Hkv, D, P = 4, 2, 128, 16
    lens, n_q = [0, 3, 0, 20], [1, 6, 4, 20]
    ref, table = filled(4, Hkv, D, P, lens, seed=2)
    q = queries(sum(n_q), Hq, D, seed=5)
    out, lse, cu = attend(ref, table, lens, q, n_q, Hq)
    check(out, lse, q, ref, table, lens, cu, D ** -0.5)
    assert (out[:4] == 0).all() and torch.isneginf(lse[:4]).all()
    assert binding.device_status() == 0
    one, l1 = binding.kv_attention_fwd(q[:1].cuda(), to_gpu(ref), table[:1].cuda(),
                                       torch.zeros(1, dtype=torch.int32).cuda(), Hq)
    assert (one == 0).all() and torch.isneginf(l1).all()


@pytest.mark.usefixtures("both_layouts")
def test_rows_outside_the_sequences_keep_their_content():
    Hq, Hkv, D, P = 8, 2, 64, 32
    lens = [50, 7]
    ref, table = filled(8, Hkv, D, P, lens, seed=6)
    T = 12
    q = queries(T, Hq, D, seed=6)
    out = torch.full((T, Hq, D), 3.25, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, Hq), 9.0, device="cuda")
    cu = [2, 5, 9]
    binding.kv_attention_fwd(q.cuda(), to_gpu(ref), table.cuda(),
                             torch.tensor(lens, dtype=torch.int32).cuda(), Hq,
                             cu_q=torch.tensor(cu).cuda(), max_q_len=4, out=out, lse=lse)
    out, lse = out.cpu(), lse.cpu()
    for sl in (slice(0, 2), slice(9, 12)):
        assert (out[sl] == 3.25).all() and (lse[sl] == 9.0).all()
    check(out, lse, q, ref, table, lens, cu, D ** -0.5)


@pytest.mark.usefixtures("both_layouts")
def test_packed_rows_and_strides():
    """The packed QKV tensor and a view with a wider row give the same bits."""
    Hq, Hkv, D, P = 8, 2, 128, 32
    lens = [40, 90, 3]
    ref, table = filled(4, Hkv, D, P, lens, seed=12)
    q = queries(3, Hq, D, seed=12)
    args = (to_gpu(ref), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), Hq)
    want, wl = binding.kv_attention_fwd(q.cuda(), *args)
    packed = torch.full((3, (Hq + 2 * Hkv) * D), float("nan"), dtype=torch.bfloat16)
    packed[:, :Hq * D] = q.view(3, -1)
    wide = torch.full((3, 4000), float("inf"), dtype=torch.bfloat16)
    wide[:, 8:8 + Hq * D] = q.view(3, -1)
    for x in (packed.cuda(), wide.cuda()[:, 8:8 + Hq * D], wide.cuda()[:, 8:]):
        got, gl = binding.kv_attention_fwd(x, *args)
        assert torch.equal(got, want) and torch.equal(gl, wl)
    heads = wide.cuda()[:, 8:8 + Hq * D].unflatten(1, (Hq, D))
    got, gl = binding.kv_attention_fwd(heads, *args)
    assert torch.equal(got, want) and torch.equal(gl, wl)


@pytest.mark.parametrize("size,spread,scale", [(40.0, 1.0, None), (1e-20, 1.0, None), (1e18, 1.0, 1e-18),
                                               (1.5, 30.0, None), (1.5, 1.0, 0.0), (1.5, 1.0, -0.2),
                                               (0.0, 1.0, None)])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.usefixtures("both_layouts")
def test_sizes_of_queries_and_values(size, spread, scale, bits):
    """One-hot and flat softmaxes, queries far outside fp16, values whose scales
    span fp16's range, zero and negative softmax scales."""
    Hq, Hkv, D, P = 4, 1, 128, 32
    lens, n_q = [200, 77], [1, 3]
    ref, table = filled(bits, Hkv, D, P, lens, seed=31, spread=spread)
    if spread > 1:  # keys of plain size: the logits stay ordinary, the values do not
        plain, _ = filled(bits, Hkv, D, P, lens, seed=31)
        ref.codes[:, 0], ref.scales[:, 0] = plain.codes[:, 0], plain.scales[:, 0]
        ref.vals[:, 0] = plain.vals[:, 0]
    q = queries(4, Hq, D, seed=31, size=size)
    out, lse, cu = attend(ref, table, lens, q, n_q, Hq, scale=scale)
    check(out, lse, q, ref, table, lens, cu, D ** -0.5 if scale is None else scale)


@pytest.mark.usefixtures("both_layouts")
def test_nan_stays_where_the_formula_has_it():
    Hq, Hkv, D, P = 8, 2, 128, 16
    lens, n_q = [60, 60], [3, 1]
    ref, table = filled(8, Hkv, D, P, lens, seed=13)
    q = queries(4, Hq, D, seed=13)
    q[3, 2, 5] = float("nan")                    # one head of sequence 1
    q[3, 5, 0] = float("inf")
    # sequence 0: a value group of the newest token, which only the last query sees
    pg, off = int(table[0, 59 // P]), 59 % P
    ref.scales[pg, 1, 1, off, 2] = float("nan")
    ref.vals[pg, 1, 1, off, 64:96] = float("nan")
    # and a key group of token 58, which queries 1 and 2 see
    pg, off = int(table[0, 58 // P]), 58 % P
    ref.scales[pg, 0, 0, off, 1] = float("nan")
    out, lse, cu = attend(ref, table, lens, q, n_q, Hq)
    bad = torch.isnan(out.float())
    want = torch.zeros_like(bad)
    want[1:3, :4] = True                         # the key head 0's queries from token 58 on
    want[2, 4:, 64:96] = True                    # the value head 1's dimensions of that group
    want[3, 2] = want[3, 5] = True
    assert torch.equal(bad, want)
    assert torch.equal(torch.isnan(lse), want.all(-1))


@pytest.mark.usefixtures("both_layouts")
def test_bad_pages_and_lengths_are_zeros_and_reported():
    Hq, Hkv, D, P = 4, 2, 64, 16
    lens, n_q = [70, 30], [2, 1]
    ref, table = filled(4, Hkv, D, P, lens, seed=14)
    table[0, 2] = ref.codes.shape[0]
    table[0, 3] = -1
    q = queries(3, Hq, D, seed=14)
    out, lse, cu = attend(ref, table, lens, q, n_q, Hq)
    assert binding.device_status() == binding.RN_STATUS_BAD_INDEX
    check(out, lse, q, ref, table, lens, cu, D ** -0.5)
    # a length above the table is cut to it
    short = table[1:, :1].contiguous()
    got, gl = binding.kv_attention_fwd(q[2:].cuda(), to_gpu(ref), short.cuda(),
                                       torch.tensor([1000], dtype=torch.int32).cuda(), Hq)
    assert binding.device_status() == binding.RN_STATUS_BAD_INDEX
    check(got.cpu(), gl.cpu(), q[2:], ref, short, [16], [0, 1], D ** -0.5)
    # queries beyond max_q_len stay unwritten
    keep = torch.full((2, Hq, D), 5.0, dtype=torch.bfloat16, device="cuda")
    binding.kv_attention_fwd(q[:2].cuda(), to_gpu(ref), table[1:].cuda(),
                             torch.tensor([30], dtype=torch.int32).cuda(), Hq,
                             cu_q=torch.tensor([0, 2]).cuda(), max_q_len=1, out=keep)
    assert binding.device_status() == binding.RN_STATUS_BAD_INDEX
    assert (keep[1] == 5.0).all() and not (keep[0] == 5.0).all()


@pytest.mark.parametrize("bits,Hq,Hkv,D,n", [(4, 4, 1, 128, 20000), (8, 8, 1, 64, 9000),
                                             (4, 2, 1, 256, 6001)])
def test_long_contexts(bits, Hq, Hkv, D, n):
    """Many CTAs share a sequence; small sequences sit beside it."""
    lens = [3, n, 0, 40]
    ref, table = filled(bits, Hkv, D, 64, lens, seed=n)
    q = queries(4, Hq, D, seed=n)
    out, lse = binding.kv_attention_fwd(q.cuda(), to_gpu(ref), table.cuda(),
                                        torch.tensor(lens, dtype=torch.int32).cuda(), Hq)
    check(out.cpu(), lse.cpu(), q, ref, table, lens, [0, 1, 2, 3, 4], D ** -0.5)


# ---- more than 64 columns: 128 at a time, one or two such tiles side by side -------------

CHUNKS = [(4, 1, 64, 16), (8, 2, 128, 16), (6, 2, 128, 64), (3, 1, 256, 32), (70, 1, 128, 128),
          (5, 1, 64, 64), (8, 1, 256, 16)]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("Hq,Hkv,D,P", CHUNKS)
@pytest.mark.usefixtures("both_layouts")
def test_chunks_of_ragged_length(bits, Hq, Hkv, D, P):
    """Tiles of 128 columns that are full, partly full and empty, tiles of tokens that
    end anywhere, beside sequences of one query and of none."""
    lens, n_q = [140, 33, 257, 1, 96, 400], [33, 20, 70, 1, 0, 2]
    ref, table = filled(bits, Hkv, D, P, lens, seed=D + P + 2)
    q = queries(sum(n_q), Hq, D, seed=Hq)
    out, lse, cu = attend(ref, table, lens, q, n_q, Hq)
    check(out, lse, q, ref, table, lens, cu, D ** -0.5)
    again, lse2, _ = attend(ref, table, lens, q, n_q, Hq)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    assert binding.device_status() == 0


@pytest.mark.parametrize("window,sinks", [(1, 0), (40, 3), (129, 130), (300, 1)])
@pytest.mark.parametrize("Hq,Hkv,D,P,bits", [(8, 2, 128, 16, 4), (4, 1, 64, 32, 8), (4, 2, 256, 64, 4)])
@pytest.mark.usefixtures("both_layouts")
def test_chunks_with_window_and_sinks(window, sinks, Hq, Hkv, D, P, bits):
    lens, n_q = [500, 70], [60, 70]
    ref, table = filled(bits, Hkv, D, P, lens, seed=window)
    first = lens[0] - n_q[0] - window + 1                   # nothing between the sinks and here
    for j in range(sinks, max(first, 0)):
        ref.scales[int(table[0, j // P]), :, :, j % P] = float("nan")
    gone = table.clone()
    for pg in range(-(-sinks // P), max(first, 0) // P):
        gone[0, pg] = -3
    q = queries(sum(n_q), Hq, D, seed=9)
    out, lse, cu = attend(ref, gone, lens, q, n_q, Hq, window=window, sinks=sinks)
    check(out, lse, q, ref, table, lens, cu, D ** -0.5, window, sinks)
    assert binding.device_status() == 0


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.usefixtures("both_layouts")
def test_chunk_rows_that_see_nothing_and_rows_outside(D):
    Hq, Hkv, P = 4, 1, 16
    lens, n_q = [0, 25, 40], [40, 60, 40]
    ref, table = filled(8, Hkv, D, P, lens, seed=3)
    T = sum(n_q) + 5
    q = queries(T, Hq, D, seed=5)
    keep = torch.full((T, Hq, D), 2.5, dtype=torch.bfloat16, device="cuda")
    out, lse, cu = attend(ref, table, lens, q, n_q, Hq, out=keep)
    check(out, lse, q, ref, table, lens, cu, D ** -0.5)
    assert (out[:40] == 0).all() and (out[40:75] == 0).all() and torch.isneginf(lse[:75]).all()
    assert (out[140:] == 2.5).all()
    assert binding.device_status() == 0


@pytest.mark.parametrize("D,bits", [(64, 4), (128, 8), (256, 4), (256, 8)])
@pytest.mark.usefixtures("both_layouts")
def test_chunk_nan_and_infinite_queries_stay_in_their_place(D, bits):
    Hq, Hkv, P, n, L = 4, 2, 16, 50, 120
    ref, table = filled(bits, Hkv, D, P, [L], seed=17)
    q = queries(n, Hq, D, seed=17)
    q[7, 1, 3] = float("inf")
    g = D // 32 - 1
    spots = [(1, 0, 100, g), (1, 1, 60, 0), (0, 1, 110, 1)]  # value, value, key
    for which, h, t, grp in spots:
        pg, off = int(table[0, t // P]), t % P
        ref.scales[pg, which, h, off, grp] = float("nan")
        ref.vals[pg, which, h, off, 32 * grp:32 * grp + 32] = float("nan")
    out, lse, cu = attend(ref, table, [L], q, [n], Hq)
    want = torch.zeros(n, Hq, D, dtype=torch.bool)
    want[7, 1] = True
    want[100 - (L - n):, :2, 32 * g:32 * g + 32] = True     # queries from token 100 on
    want[:, 2:, :32] = True                                  # token 60 is before them all
    want[110 - (L - n):, 2:] = True
    assert torch.equal(torch.isnan(out.float()), want)
    assert torch.equal(torch.isnan(lse), want.all(-1))


@pytest.mark.parametrize("D,bits", [(64, 8), (128, 4), (256, 8)])
@pytest.mark.usefixtures("both_layouts")
def test_chunk_scales_above_255(D, bits):
    """Values (and, with small queries, keys) far above the rest: restored at 2^-8."""
    Hq, Hkv, P = 4, 1, 32
    lens, n_q = [300, 150], [40, 35]
    ref, table = filled(bits, Hkv, D, P, lens, seed=23)
    g = torch.Generator().manual_seed(1)
    for b, n in enumerate(lens):
        pos = torch.arange(n)
        x = torch.randn(n, 2, Hkv, D, generator=g)
        x[40:50, 1] *= 4000.0
        x[120, 0] *= 20000.0
        ref.write(x.to(torch.bfloat16), table[b, pos // P].long() * P + pos % P)
    q = queries(sum(n_q), Hq, D, seed=2, size=1e-4)
    out, lse, cu = attend(ref, table, lens, q, n_q, Hq)
    check(out, lse, q, ref, table, lens, cu, D ** -0.5)


@pytest.mark.usefixtures("both_layouts")
def test_chunk_bad_pages_are_zeros_and_reported():
    Hq, Hkv, D, P = 8, 2, 128, 16
    lens, n_q = [200], [30]
    ref, table = filled(4, Hkv, D, P, lens, seed=14)
    table[0, 2], table[0, 7] = ref.codes.shape[0], -1
    q = queries(30, Hq, D, seed=14)
    out, lse, cu = attend(ref, table, lens, q, n_q, Hq)
    assert binding.device_status() == binding.RN_STATUS_BAD_INDEX
    check(out, lse, q, ref, table, lens, cu, D ** -0.5)


def test_chunk_sizes_of_queries():
    Hq, Hkv, D, P = 4, 1, 128, 32
    lens, n_q = [200], [40]
    ref, table = filled(8, Hkv, D, P, lens, seed=33)
    for size, scale in ((40.0, None), (1e-20, None), (1e18, 1e-18), (1.5, 0.0), (1.5, -0.2)):
        q = queries(40, Hq, D, seed=33, size=size)
        out, lse, cu = attend(ref, table, lens, q, n_q, Hq, scale=scale)
        check(out, lse, q, ref, table, lens, cu, D ** -0.5 if scale is None else scale)


def test_chunk_captured_beside_another_on_a_second_stream():
    """A captured chunk call replays on new lengths; two calls run at the same time with
    a workspace each."""
    Hq, Hkv, D, P = 8, 2, 128, 16
    ref, table = filled(4, Hkv, D, P, [300, 180], seed=44)
    cache, dt = to_gpu(ref), table.cuda()
    T = 70
    q = queries(T, Hq, D, seed=44).cuda()
    lens = torch.tensor([300, 180], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 40, 70], device="cuda")
    ws = [binding.kv_attention_workspace(cache, 2, Hq, max_q_len=60) for _ in range(2)]
    outs = [torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    lses = [torch.empty(T, Hq, device="cuda") for _ in range(2)]

    def call(i):
        binding.kv_attention_fwd(q, cache, dt, lens, Hq, cu_q=cu, max_q_len=60, out=outs[i],
                                 lse=lses[i], workspace=ws[i])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(0)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(0)
    for a, b, c in ((300, 180, 40), (41, 177, 12), (259, 64, 58)):
        lens.copy_(torch.tensor([a, b], dtype=torch.int32))
        cu.copy_(torch.tensor([0, c, 70]))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            call(1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1]) and torch.equal(lses[0], lses[1])
        check(outs[0].cpu(), lses[0].cpu(), q.cpu(), ref, table, [a, b], [0, c, 70], D ** -0.5)


@pytest.mark.parametrize("Hq,Hkv,D,bits,n_q", [(4, 1, 128, 4, 64), (4, 1, 64, 8, 64), (2, 1, 256, 4, 40)])
def test_chunk_over_a_long_context(Hq, Hkv, D, bits, n_q):
    """Many CTAs share a chunk's tiles of tokens; the pieces are joined."""
    lens = [6000]
    ref, table = filled(bits, Hkv, D, 64, lens, seed=71)
    q = queries(n_q, Hq, D, seed=71)
    out, lse, cu = attend(ref, table, lens, q, [n_q], Hq)
    check(out, lse, q, ref, table, lens, cu, D ** -0.5)


@pytest.mark.parametrize("width", [0, 1, 70])
def test_short_and_long_tables_agree_with_the_formula(width):
    """The table's width decides between a CTA for each head and the line of units; rows
    that see nothing, a bad length and bad pages are the same on both."""
    Hq, Hkv, D, P = 8, 2, 128, 32
    lens, n_q = [0, 5, 90, 200, 31], [1, 3, 0, 2, 1]
    ref, table = filled(4, Hkv, D, P, lens, seed=61)
    table = torch.cat((table, torch.full((5, 100 * width), -1, dtype=torch.int32)), dim=1)
    q = queries(sum(n_q) + 1, Hq, D, seed=61)
    keep = torch.full((sum(n_q) + 1, Hq, D), 1.5, dtype=torch.bfloat16, device="cuda")
    out, lse, cu = attend(ref, table, lens, q, n_q, Hq, out=keep)
    check(out, lse, q, ref, table, lens, cu, D ** -0.5)
    assert (out[0] == 0).all() and (out[-1] == 1.5).all()
    assert binding.device_status() == 0
    table[3, 1] = -1
    out, lse, cu = attend(ref, table, lens, q, n_q, Hq)
    assert binding.device_status() == binding.RN_STATUS_BAD_INDEX
    check(out, lse, q, ref, table, lens, cu, D ** -0.5)
    if width == 0:
        binding.kv_attention_fwd(q[:5].cuda(), to_gpu(ref), table.cuda(),
                                 torch.tensor([0, 5, 90, 40000, 31], dtype=torch.int32).cuda(), Hq)
        assert binding.device_status() == binding.RN_STATUS_BAD_INDEX


def test_more_heads_than_ctas_of_every_length():
    """Notes by CTA instead of by head, pieces of every kind."""
    Hq, Hkv, D, P = 40, 20, 64, 16
    lens = [(37 * i) % 400 for i in range(40)]
    ref, table = filled(8, Hkv, D, P, lens, seed=5)
    table = torch.cat((table, torch.full((40, 200), -1, dtype=torch.int32)), dim=1)
    q = queries(len(lens), Hq, D, seed=5)
    ws = binding.kv_attention_workspace(to_gpu(ref), len(lens), Hq)
    ws.fill_(0xFF)
    out, lse = binding.kv_attention_fwd(q.cuda(), to_gpu(ref), table.cuda(),
                                        torch.tensor(lens, dtype=torch.int32).cuda(), Hq,
                                        workspace=ws)
    check(out.cpu(), lse.cpu(), q, ref, table, lens, list(range(len(lens) + 1)), D ** -0.5)


def test_many_sequences_and_a_long_chunk():
    Hq, Hkv, D, P = 4, 2, 64, 16
    lens = [(7 * i) % 50 for i in range(700)] + [500]
    n_q = [1 if n else 0 for n in lens[:-1]] + [150]
    ref, table = filled(4, Hkv, D, P, lens, seed=1)
    q = queries(sum(n_q), Hq, D, seed=1)
    out, lse, cu = attend(ref, table, lens, q, n_q, Hq)
    check(out, lse, q, ref, table, lens, cu, D ** -0.5)


@pytest.mark.parametrize("long,Hq,Hkv,D,P,bits", [(30, 24, 24, 64, 16, 8), (14, 48, 24, 64, 32, 4),
                                                  (90, 12, 12, 128, 16, 4), (40, 20, 10, 256, 32, 8),
                                                  (14, 40, 2, 64, 32, 8)])
@pytest.mark.usefixtures("both_layouts")
def test_one_chunk_among_single_tokens(long, Hq, Hkv, D, P, bits):
    """With heads enough (ten or more here) sequences of few queries are a launch of their
    own; each row has the arithmetic of its launch, and rows of neither keep their content."""
    G = Hq // Hkv
    split = Hkv >= (10 if long * G > 64 else 24)
    lens = [1, 0, 300, 64, 20, long + 33, 5, 2, 129, 31, 0, 90, 150, 17]
    n_q = [1, 0, 1, 2, 0, long, 1, 3, 1, 1, 1, 9, 8 // G + 1, max(8 // G, 1)]
    assert 2 * sum(n_q) <= len(n_q) * long
    ref, table = filled(bits, Hkv, D, P, lens, seed=long + D)
    q = queries(sum(n_q) + 3, Hq, D, seed=long)
    T = sum(n_q)
    out = torch.full((T + 3, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T + 3, Hq), 7.0, device="cuda")
    ws = binding.kv_attention_workspace(to_gpu(ref), len(lens), Hq, max_q_len=long)
    ws.fill_(0xFF)
    got, got_lse, cu = attend(ref, table, lens, q, n_q, Hq, out=out, lse=lse, workspace=ws)
    for b, n in enumerate(lens):
        few = split and n_q[b] <= max(8 // G, 1)
        check(got, got_lse, q, ref, table[b:b + 1], [n], cu[b:b + 2], D ** -0.5,
              wide=long * G > 64 and not few)
    assert (got[T:] == 7).all() and (got_lse[T:] == 7).all()
    assert binding.device_status() == 0


def test_a_mixed_step_captured_and_replayed():
    """Both launches of a mixed call read lengths and offsets at replay."""
    Hq, Hkv, D, P, B = 40, 20, 64, 32, 6
    lens = [200, 130, 90, 300, 64, 33]
    ref, table = filled(4, Hkv, D, P, lens, seed=12)
    q = queries(70, Hq, D, seed=12)
    cache, t, qd = to_gpu(ref), table.cuda(), q.cuda()
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    cu = torch.zeros(B + 1, dtype=torch.int64).cuda()
    ws = binding.kv_attention_workspace(cache, B, Hq, max_q_len=60)
    out = torch.empty(70, Hq, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(70, Hq, device="cuda")

    def step():
        binding.kv_attention_fwd(qd, cache, t, n, Hq, cu_q=cu, max_q_len=60, out=out, lse=lse,
                                 workspace=ws)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n_q in ([60, 1, 1, 1, 1, 1], [1, 2, 1, 40, 0, 20], [1] * 6, [2, 3, 2, 3, 2, 3]):
        offsets = [0]
        for x in n_q:
            offsets.append(offsets[-1] + x)
        cu.copy_(torch.tensor(offsets))
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        for b in range(B):
            check(out.cpu(), lse.cpu(), q, ref, table[b:b + 1], [lens[b]], offsets[b:b + 2], D ** -0.5,
                  wide=n_q[b] > 4)
        assert (out[offsets[-1]:] == 7).all()


def test_runs_repeat_bit_for_bit_and_share_a_workspace():
    Hq, Hkv, D = 8, 2, 128
    lens = [5000, 17, 900]
    ref, table = filled(4, Hkv, D, 32, lens, seed=40)
    cache = to_gpu(ref)
    q = queries(3, Hq, D, seed=40).cuda()
    args = (cache, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), Hq)
    ws = binding.kv_attention_workspace(cache, 3, Hq)
    ws.fill_(0x7F)                                          # it needs no clearing
    first = binding.kv_attention_fwd(q, *args, workspace=ws)
    other = binding.kv_attention_fwd(q.flip(0).contiguous(), *args, workspace=ws)
    again = binding.kv_attention_fwd(q, *args, workspace=ws)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    assert not torch.equal(first[0], other[0])


def test_captured_steps_replay_on_new_data():
    """The whole serving step in a graph: norm + RoPE, cache write, attention;
    lengths, slots and positions change between replays."""
    T, Hq, Hkv, D, P, pages = 3, 8, 2, 128, 16, 40
    cache = binding.new_kv_cache(pages, Hkv, D, page_size=P)
    ref = kv_ref.Cache(pages, Hkv, D, P, 4)
    ref.codes.copy_(cache.codes), ref.scales.copy_(cache.scales), ref.vals.zero_()
    table = torch.randperm(pages)[:T * 10].view(T, 10).int()
    static = {"qkv": torch.zeros(T, (Hq + 2 * Hkv) * D, dtype=torch.bfloat16, device="cuda"),
              "pos": torch.zeros(T, dtype=torch.int64, device="cuda"),
              "slots": torch.zeros(T, dtype=torch.int64, device="cuda"),
              "lens": torch.ones(T, dtype=torch.int32, device="cuda")}
    _, wq, wk, _ = qkv_inputs(1, Hq, Hkv, D, seed=2, device="cuda")
    trig = binding.rope_cos_sin_table(1e6, 160, D)
    dt = table.cuda()
    ws = binding.kv_attention_workspace(cache, T, Hq)
    out = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(T, Hq, device="cuda")

    def step():
        binding.qk_norm_rope_fwd(static["qkv"], wq, wk, trig, static["pos"], Hq, Hkv, D, D, 1e-6)
        binding.kv_cache_write(static["qkv"], static["slots"], cache, Hq, Hkv, D)
        binding.kv_attention_fwd(static["qkv"], cache, dt, static["lens"], Hq, out=out, lse=lse,
                                 workspace=ws)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        static["slots"].fill_(-1)
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(40):
        qkv, _, _, _ = qkv_inputs(T, Hq, Hkv, D, seed=100 + i)
        at = torch.tensor([i, i + 50, i + 119])             # sequences of different length
        if i == 0:                                          # their first tokens
            for b in range(T):
                n = int(at[b])
                pos = torch.arange(n)
                x, _, _, _ = qkv_inputs(max(n, 1), 0, Hkv, D, seed=500 + b)
                sl = table[b, pos // P].long() * P + pos % P
                x = x[:n]
                binding.kv_cache_write(x.cuda(), sl.cuda(), cache, 0, Hkv, D)
                ref.write(x.view(n, 2, Hkv, D), sl)
        slots = table[torch.arange(T), at // P].long() * P + at % P
        static["qkv"].copy_(qkv), static["pos"].copy_(at), static["slots"].copy_(slots)
        static["lens"].copy_((at + 1).int())
        graph.replay()
        torch.cuda.synchronize()
        normed = static["qkv"].cpu().view(T, Hq + 2 * Hkv, D)
        ref.write(normed[:, Hq:].unflatten(1, (2, Hkv)), slots)
        if i % 13 == 0 or i == 39:
            check(out.cpu(), lse.cpu(), normed[:, :Hq], ref, table, (at + 1).tolist(),
                  list(range(T + 1)), D ** -0.5)
    assert torch.equal(cache.codes.cpu(), ref.codes)
    assert binding.device_status() == 0


def test_another_stream_without_a_workspace():
    Hq, Hkv, D = 8, 2, 128
    lens = [3000, 90]
    ref, table = filled(8, Hkv, D, 64, lens, seed=50)
    q = queries(2, Hq, D, seed=50)
    args = [q.cuda(), to_gpu(ref), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), Hq]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    out, lse = binding.kv_attention_fwd(*args, stream=st)
    st.synchronize()
    check(out.cpu(), lse.cpu(), q, ref, table, lens, [0, 1, 2], D ** -0.5)


def test_results_dropped_at_once_are_not_reused_while_their_stream_writes():
    Hq, D, lens = 8, 128, [700] * 3
    ref, table = filled(4, 2, D, 64, lens, seed=1)
    q, cache, t = queries(3, Hq, D, seed=1).cuda(), to_gpu(ref), table.cuda()
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    ws = binding.kv_attention_workspace(cache, 3, Hq)
    cu = torch.tensor([0, 700, 1400, 2100]).cuda()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)          # the calls below start later than what follows
    binding.kv_attention_fwd(q, cache, t, n, Hq, workspace=ws, stream=side)
    binding.kv_cache_read(cache, t, cu, 2100, stream=side.cuda_stream)
    mine = [torch.full(shape, 7.0, dtype=dtype, device="cuda")
            for shape, dtype in (((3, Hq, D), torch.bfloat16), ((3, Hq), torch.float32),
                                 ((2100, 2, D), torch.bfloat16), ((2100, 2, D), torch.bfloat16))]
    torch.cuda.synchronize()
    assert all((x == 7).all() for x in mine)


@pytest.mark.parametrize("n_q,len_", [(5, 3), (40, 25), (200, 130)])
@pytest.mark.usefixtures("both_layouts")
def test_nan_queries_that_see_nothing_are_zeros(n_q, len_):
    Hq, Hkv, D = 8, 2, 128
    ref, table = filled(8, Hkv, D, 32, [len_], seed=n_q)
    q = queries(n_q, Hq, D, seed=n_q)
    blind = n_q - len_
    q[:blind] = float("nan")
    q[blind - 1] = float("inf")
    out, lse, cu = attend(ref, table, [len_], q, [n_q], Hq)
    assert (out[:blind] == 0).all() and (lse[:blind] == -math.inf).all()
    plain = q.clone()
    plain[:blind] = 0
    want, want_lse, _ = attend(ref, table, [len_], plain, [n_q], Hq)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_wild_row_offsets_are_no_queries():
    """Offsets whose difference leaves 64 bits; they are looked at one by one."""
    Hq, D = 4, 64
    ref, table = filled(4, 1, D, 16, [20, 20], seed=2)
    q, t = queries(4, Hq, D, seed=2).cuda(), table.cuda()
    n = torch.tensor([20, 20], dtype=torch.int32).cuda()
    for cu, bad in (([2 ** 62, -2 ** 63 + 1, -2 ** 63], False), ([2 ** 63 - 1, -2 ** 63, -2 ** 63 + 2], True),
                    ([-2 ** 63, 2 ** 62, 2 ** 62 + 1], True), ([3, 5, 4], True), ([-1, 1, 1], True)):
        for max_q_len in (2, 40):
            out = torch.full((4, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
            lse = torch.full((4, Hq), 7.0, device="cuda")
            binding.kv_attention_fwd(q, to_gpu(ref), t, n, Hq, cu_q=torch.tensor(cu).cuda(),
                                     max_q_len=max_q_len, out=out, lse=lse)
            assert (out == 7).all() and (lse == 7).all()
            assert binding.device_status() == (binding.RN_STATUS_BAD_INDEX if bad else 0)


def heads_of(ref, n):
    """The cache's first n heads, for the plain form."""
    few = copy.copy(ref)
    few.vals, few.scales = ref.vals[:, :, :n], ref.scales[:, :, :n]
    return few


def test_more_query_tiles_and_heads_than_a_grid_holds():
    """A million sequences that might have 8192 queries each, of which two have some."""
    Hq = Hkv = D = 64
    B, n_q = 2 ** 20, [130, 2]
    ref, table = filled(4, Hkv, D, 256, [200, 40], seed=3)
    q = queries(sum(n_q), Hq, D, seed=3)
    t = torch.full((B, table.shape[1]), -1, dtype=torch.int32)
    lens, cu = torch.zeros(B, dtype=torch.int32), torch.full((B + 1,), 130)
    t[0], t[-1], lens[0], lens[-1], cu[0], cu[-1] = table[0], table[1], 200, 40, 0, 132
    out, lse = binding.kv_attention_fwd(q.cuda(), to_gpu(ref), t.cuda(), lens.cuda(), Hq,
                                        cu_q=cu.cuda(), max_q_len=8192)
    check(out[:, :4].cpu(), lse[:, :4].cpu(), q[:, :4], heads_of(ref, 4), table, [200, 40],
          [0, 130, 132], D ** -0.5)
    assert binding.device_status() == 0


def test_refusals_of_the_binding():
    cache = binding.new_kv_cache(2, 2, 64, page_size=16)
    table = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    lens = torch.ones(1, dtype=torch.int32, device="cuda")
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TypeError):
        binding.kv_attention_fwd(q.half(), cache, table, lens, 4)
    with pytest.raises(TypeError):
        binding.kv_attention_fwd(q, cache, table.long(), lens, 4)
    with pytest.raises(ValueError):
        binding.kv_attention_fwd(q.expand(2, 4, 64), cache, table, lens, 4)     # T != B
    with pytest.raises(ValueError):
        binding.kv_attention_fwd(q.transpose(1, 2), cache, table, lens, 64)
    with pytest.raises(ValueError):
        binding.kv_attention_fwd(q.cpu(), cache, table, lens, 4)
    with pytest.raises(binding.RowNormError) as e:
        binding.kv_attention_fwd(q.view(1, 256)[:, :192].contiguous(), cache, table, lens, 3)
    assert e.value.code == binding.RN_ERR_SHAPE                                  # 3 % 2 heads
    with pytest.raises(binding.RowNormError) as e:
        binding.kv_attention_fwd(q, cache, table, lens, 4,
                                 workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        binding.kv_cache_write(torch.zeros(1, 4 * 64, dtype=torch.bfloat16, device="cuda"),
                               torch.zeros(1, dtype=torch.int64, device="cuda"), cache, 4, 2, 64)
    with pytest.raises(ValueError):
        binding.kv_cache_write(torch.zeros(1, 8 * 64, dtype=torch.bfloat16, device="cuda"),
                               torch.zeros(1, dtype=torch.int64, device="cuda"), cache, 6, 1, 64)
    with pytest.raises(TypeError):
        binding.kv_cache_read(cache, table, torch.zeros(2, dtype=torch.int32, device="cuda"), 1)
