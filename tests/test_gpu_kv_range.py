"""Attention over the quantised cache where sizes differ widely (GPU): a token that
dominates the softmax, values of any size, tokens whose scales are far above the
others'.  Against the 64-bit definition.

Tolerance of an output element (derived, nothing fitted), w the softmax weights, W the
largest of the row's, |v| the values' sizes, u = 2^-11 half a step of fp16:
  * the result is rounded once to bf16: eps/2 * |out|;
  * up to 64 columns: a weight and its product with a value's scale are rounded to fp16;
    more: the weight and the value.  Relative: 2 u * sum w |v|.  Absolute, where fp16 is
    subnormal (half a step is 2^-25), up to 64 columns: a token's weight counts 2^e, its
    scales 2^-e, 2^e at most twice its largest scale S, or 2^-14; the largest w 2^e = M
    counts 2^10 at least.  The weight and the product are off by 2^-35 M a unit of code
    each, the scale by 2^-25 2^e w.  More columns: the largest weight W counts 2^10 at
    least, so a weight is off by 2^-35 W;
  * more than 64 columns: a token with a scale above 65504 / Q (Q the largest code) counts
    at 2^-3 of its size in 4 bits, 2^-7 in 8, and its weight that much more.  Its scales
    are off by 2^-25 of that, half a step of subnormal fp16, a unit of code, and the
    largest weight W is that of w * 2^3 (2^7) for it;
  * the fp32 sums: an instruction adds 17 numbers, each cut to the largest one's 24 bits.
    Up to 304 instructions follow one another here (4000 tokens, 16 an instruction, shared
    by the warps of several CTAs): 300 * 17 * 2^-24 * sum w |v| is far above them all;
  * a logit: up to 64 columns a group's two instructions over q * stored code (0 .. 2z),
    z * sum q taken off, then D / 32 fused multiply-adds and two roundings; more columns
    D / 8 instructions over exact products.  A query's largest element counts 2^13 at
    least, so a subnormal one is off by 2^-38 of that, in 4 bits up to 64 columns, where
    every other one counts a 16th, by 2^-34.  A logit's error e_t moves the result by
    sum w e (|v| + |out|), lse by sum w e;
  * exp2 and the running sums: 2^-20.
"""
from __future__ import annotations

import math

import pytest
import torch

from row_normalization_gb300 import binding
from tests import kv_ref
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu

EPS = torch.finfo(torch.bfloat16).eps / 2
U = torch.finfo(torch.float16).eps / 2
DOWN = {4: 3, 8: 7}
TOP = {4: 9352.0, 8: 515.5}  # the largest scales of which Q is inside fp16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    binding.device_status()


def cache_of(kv, bits, P, extra=0):
    """kv [n, 2, Hkv, D] bf16 as one sequence's cache on shuffled pages."""
    n, _, Hkv, D = kv.shape
    need = -(-n // P)
    order = torch.randperm(need + 2, generator=torch.Generator().manual_seed(n))
    table = torch.full((1, need + extra // P), -1, dtype=torch.int32)
    table[0, :need] = order[:need].int()
    ref = kv_ref.Cache(need + 2, Hkv, D, P, bits)
    pos = torch.arange(n)
    ref.write(kv, table[0, pos // P].long() * P + pos % P)
    return ref, table


def run(ref, table, L, q):
    n, Hq, _ = q.shape
    out, lse = binding.kv_attention_fwd(
        q.cuda(), binding.KVCache(ref.codes.cuda(), ref.scales.cuda()), table.cuda(),
        torch.tensor([L], dtype=torch.int32).cuda(), Hq, cu_q=torch.tensor([0, n]).cuda(),
        max_q_len=n)
    assert binding.device_status() == 0
    return out.cpu(), lse.cpu()


def check(out, lse, q, ref, table, L, scale=None):
    n, Hq, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    pos = torch.arange(L)
    pg, off = table[0, pos // ref.P].long(), pos % ref.P
    K, V = (ref.vals[pg, w, :, off] for w in (0, 1))                   # [L, Hkv, D]
    SK, SV = (ref.scales[pg, w, :, off].double() for w in (0, 1))      # [L, Hkv, D / 32]
    G = Hq // K.shape[1]
    wide = n * G > 64
    z, Q = (8, 7) if ref.bits == 4 else (128, 127)
    down = 2.0 ** DOWN[ref.bits]
    worst = 0.0
    for h in range(Hq):
        k, v, sk, sv = (x[:, h // G] for x in (K, V, SK, SV))
        big_k, big_v = (x.amax(1) > TOP[ref.bits] for x in (sk, sv))
        for i in sorted({*range(0, n, max(1, n // 8)), n - 1}):
            see = L - n + i + 1
            x = q[i, h].double()
            s = k[:see] @ x * scale
            l = torch.logsumexp(s, 0)
            w = torch.exp(s - l)
            o = w @ v[:see]
            # the logits' errors
            qk = k[:see].abs() @ x.abs()
            if wide:
                e = (17 * D / 8 + 10) * 2.0 ** -24 * qk
                e += big_k[:see] * 2.0 ** -25 * down * Q * x.abs().sum()
            else:
                grp = x.view(-1, 32)
                per = torch.maximum(2 * z * grp.abs().amax(1), z * grp.sum(1).abs())
                e = (34 * (sk[:see] @ per) + 10 * qk) * 2.0 ** -24
            e += 2.0 ** (-34 if ref.bits == 4 and not wide else -38) * x.abs().max() * k[:see].abs().sum(1)
            e *= abs(scale)
            moved = float(w @ e)
            a = w @ v[:see].abs()
            tol = 2.0 ** -40 + EPS * o.abs() + 1.01 * (2 * U + 2.0 ** -20 + 300 * 17 * 2.0 ** -24) * a
            tol += 1.01 * ((w * e) @ v[:see].abs() + moved * o.abs())
            if wide:
                top = (w * (1 + (down - 1) * big_v[:see])).max()
                tol += 2.0 ** -35 * top * v[:see].abs().sum(0)
                tol += (w * big_v[:see]).sum() * 2.0 ** -25 * down * Q
            else:
                part = w * torch.clamp(2 * sv[:see].amax(1), min=2.0 ** -14)
                tol += Q * (2.0 ** -34 * see * part.max() + 2.0 ** -25 * part.sum())
            r = float(((out[i, h].double() - o).abs() / tol).max())
            worst = max(worst, r)
            assert r <= 1.0, (h, i, r)
            assert abs(float(lse[i, h]) - float(l)) <= 1.01 * moved + 2.0 ** -20 + 2.0 ** -22 * abs(float(l))
    return worst


SHAPES = [(4, 1, 64), (4, 1, 128), (8, 2, 128), (2, 1, 256)]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("Hq,Hkv,D", SHAPES)
@pytest.mark.parametrize("n_q", [1, 9, 70])
@pytest.mark.parametrize("L,ahead,size", [(900, 9.0, 1.0), (900, 18.0, 0.1), (3500, 14.0, 0.01),
                                          (3500, 18.0, 0.001), (3500, 16.0, 30.0)])
def test_a_token_that_dominates(bits, Hq, Hkv, D, n_q, L, ahead, size):
    """One token has nearly all the weight and a value of zero (a sink); what is left of
    the others is the result."""
    g = torch.Generator().manual_seed(L + D)
    base = torch.randn(Hkv, D, generator=g)
    q = (base.repeat_interleave(Hq // Hkv, 0) * (1 + 0.05 * torch.randn(n_q, Hq, 1, generator=g)))
    kv = torch.randn(L, 2, Hkv, D, generator=g)
    kv[:, 0] *= 0.3
    kv[:, 1] = size * (0.75 + 0.25 * kv[:, 1].clamp(-2, 2))
    for sink in (0, (L - n_q) // 2):     # before and behind others of its share
        x = kv.clone()
        x[sink, 0] = base * ahead / (D ** -0.5 * (base * base).sum(-1, keepdim=True))
        x[sink, 1] = 0.0
        ref, table = cache_of(x.to(torch.bfloat16), bits, 32)
        qb = q.to(torch.bfloat16)
        out, lse = run(ref, table, L, qb)
        check(out, lse, qb, ref, table, L)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("Hq,Hkv,D", SHAPES)
@pytest.mark.parametrize("n_q", [2, 50])
@pytest.mark.parametrize("size", [1e-6, 1e-4, 1.0, 1e3])
def test_values_of_any_size(bits, Hq, Hkv, D, n_q, size):
    """Groups of different size beside one another, in a cache of any size."""
    L = 500
    g = torch.Generator().manual_seed(D)
    kv = torch.randn(L, 2, Hkv, D, generator=g)
    kv[:, 1] *= size * 10.0 ** -(torch.arange(D) // 32 % 4).float()
    kv[L // 2:, 1] *= 0.01                   # the newer half far below the older one
    ref, table = cache_of(kv.to(torch.bfloat16), bits, 16)
    q = torch.randn(n_q, Hq, D, generator=g).to(torch.bfloat16)
    out, lse = run(ref, table, L, q)
    check(out, lse, q, ref, table, L)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("Hq,Hkv,D", SHAPES)
@pytest.mark.parametrize("n_q,extra", [(3, 0), (9, 4096), (50, 0), (50, 4096)])
def test_a_huge_token_changes_no_other(bits, Hq, Hkv, D, n_q, extra):
    """A value and a key of 2e5 beside ones of a thousandth: queries that do not see
    them have the same bits as without them, the others are as exact as ever."""
    L = 300
    g = torch.Generator().manual_seed(D + n_q)
    q = torch.randn(n_q, Hq, D, generator=g)
    q[:, :, :32] = 0.0                       # where the huge key lies
    q[:, :, 33] = 4.0
    kv = torch.randn(L, 2, Hkv, D, generator=g)
    kv[:, 1] *= 1e-3
    plain, at_v, at_k = kv.clone(), L - n_q // 2 - 1, L - n_q // 3 - 1
    kv[at_v, 1, :, 32:64] = 2e5              # a value of next to no weight
    kv[at_v, 0, :, 33] = -40.0 * D ** 0.5 / 4
    kv[at_k, 0, :, :32] = -2e5               # a key whose size no query meets
    q = q.to(torch.bfloat16)
    ref, table = cache_of(kv.to(torch.bfloat16), bits, 32, extra)
    ref0, table0 = cache_of(plain.to(torch.bfloat16), bits, 32, extra)
    out, lse = run(ref, table, L, q)
    out0, lse0 = run(ref0, table0, L, q)
    check(out, lse, q, ref, table, L)
    before = min(at_v, at_k) - (L - n_q)     # queries in front of both
    assert before > 0 and torch.equal(out[:before], out0[:before])
    assert torch.equal(lse[:before], lse0[:before])


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("Hq,Hkv,D", SHAPES)
@pytest.mark.parametrize("n_q", [1, 50])
def test_huge_values_with_weight(bits, Hq, Hkv, D, n_q):
    """Several huge tokens of which each may dominate, NaN beside them in another group."""
    L = 400
    g = torch.Generator().manual_seed(7 * D + n_q)
    kv = torch.randn(L, 2, Hkv, D, generator=g)
    kv[5:60:11, 1] *= 1e5
    kv[100:350:50, 1, :, :32] *= 3e4
    q = 2.0 * torch.randn(n_q, Hq, D, generator=g).to(torch.bfloat16)
    ref, table = cache_of(kv.to(torch.bfloat16), bits, 64)
    out, lse = run(ref, table, L, q)
    check(out, lse, q, ref, table, L)
    # a NaN in the last group of one of them stays there
    pg, off = int(table[0, 16 // 64]), 16
    ref.scales[pg, 1, :, off, D // 32 - 1] = float("nan")
    got, lse2 = run(ref, table, L, q)
    want = torch.zeros(D, dtype=torch.bool)
    want[D - 32:] = True
    assert torch.equal(torch.isnan(got.float()), want.expand_as(got))
    assert torch.equal(got[..., :D - 32], out[..., :D - 32]) and torch.equal(lse2, lse)


def test_rescaling_inside_a_tile_keeps_weights():
    """Logits that climb by 2^20 and more between the quarters of one tile: what was stored
    before is brought down without being lost."""
    Hq, Hkv, D, L, n_q = 4, 1, 128, 128, 20
    g = torch.Generator().manual_seed(3)
    base = torch.randn(Hkv, D, generator=g)
    q = base.expand(n_q, Hq, D).to(torch.bfloat16)
    for step in (12.0, 17.0, 21.0):          # nats between the second quarter and the third
        kv = torch.zeros(L, 2, Hkv, D)
        ahead = torch.zeros(L)
        ahead[64] = step
        kv[:, 0] = base * (ahead / (D ** -0.5 * (base * base).sum())).view(-1, 1, 1)
        kv[:, 1] = 1.0 + torch.rand(L, Hkv, D, generator=g)
        kv[64, 1] = 0.0
        kv = kv.to(torch.bfloat16)
        ref, table = cache_of(kv, 8, 32)
        out, lse = run(ref, table, L, q)
        check(out, lse, q, ref, table, L)
