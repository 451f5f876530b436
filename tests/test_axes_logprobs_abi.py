"""The several-axes Q/K step and the log probabilities refuse bad arguments on the host,
before anything is launched, and their plain definitions hold together (CPU only)."""
from __future__ import annotations

import ctypes

import pytest
import torch

from row_normalization_gb300 import binding
from row_normalization_gb300.binding import (RN_ERR_ALIGN, RN_ERR_ARG, RN_ERR_NULL, RN_ERR_SHAPE, RN_OK,
                                             RopeAxes, rope_axes)
from row_normalization_gb300.build import build
from tests import axes_ref

P = 0x10000  # well-formed pointers that nothing dereferences


@pytest.fixture(scope="module")
def lib():
    build()
    return binding.load()


def pairs(values):
    return (ctypes.c_uint8 * len(values))(*values)


def fwd(lib, dtype=0, qkv=P, xs=1024, wq=P, wk=P, table=P, bf16=0, max_pos=100, pos=P, ps=64, axes=(0,) * 64, n=3,
        T=4, Hq=4, Hkv=2, D=128, r=128, style=0, out=P, os=1024):
    return lib.qk_norm_rope_axes_fwd(dtype, qkv, xs, wq, wk, table, bf16, max_pos, pos, ps,
                                     None if axes is None else pairs(axes), n, T, Hq, Hkv, D, r, 1e-6, style, out,
                                     os, None)


def bwd(lib, dtype=0, qkv=P, xs=1024, wq=P, wk=P, table=P, bf16=0, max_pos=100, pos=P, ps=64, axes=(0,) * 64, n=3,
        T=4, Hq=4, Hkv=2, D=128, r=128, style=0, out=P, os=1024, dout=P, gs=1024, dwq=P, dwk=P + 512, acc=0, ws=P,
        ws_bytes=1 << 40):
    return lib.qk_norm_rope_axes_bwd(dtype, dout, gs, qkv, xs, wq, wk, table, bf16, max_pos, pos, ps,
                                     None if axes is None else pairs(axes), n, T, Hq, Hkv, D, r, 1e-6, style, out,
                                     os, dwq, dwk, acc, ws, ws_bytes, None)


@pytest.mark.parametrize("call", [fwd, bwd])
@pytest.mark.parametrize("kw,expect", [
    ({"dtype": 2}, RN_ERR_ARG), ({"dtype": -1}, RN_ERR_ARG), ({"style": 2}, RN_ERR_ARG),
    ({"bf16": 2}, RN_ERR_ARG),
    ({"T": -1}, RN_ERR_SHAPE), ({"Hq": -1}, RN_ERR_SHAPE), ({"Hkv": -1}, RN_ERR_SHAPE),
    ({"D": 96}, RN_ERR_SHAPE), ({"r": 96}, RN_ERR_SHAPE), ({"D": 512, "r": 512}, RN_ERR_SHAPE),
    ({"n": 0}, RN_ERR_SHAPE), ({"n": 5}, RN_ERR_SHAPE), ({"max_pos": 0}, RN_ERR_SHAPE), ({"max_pos": 1 << 31}, RN_ERR_SHAPE),
    ({"T": 1 << 29, "xs": 1024}, RN_ERR_SHAPE), ({"Hq": (1 << 31) - 1, "Hkv": 1}, RN_ERR_SHAPE),
    ({"xs": 760}, RN_ERR_SHAPE), ({"xs": 1028}, RN_ERR_SHAPE), ({"os": 0}, RN_ERR_SHAPE),
    ({"os": 1025}, RN_ERR_SHAPE), ({"ps": 3}, RN_ERR_SHAPE), ({"ps": -64}, RN_ERR_SHAPE),
    ({"axes": (0,) * 63 + (3,)}, RN_ERR_ARG), ({"axes": (255,) + (0,) * 63}, RN_ERR_ARG),
    ({"axes": None}, RN_ERR_NULL), ({"qkv": None}, RN_ERR_NULL), ({"out": None}, RN_ERR_NULL),
    ({"wq": None}, RN_ERR_NULL), ({"wk": None}, RN_ERR_NULL), ({"table": None}, RN_ERR_NULL),
    ({"pos": None}, RN_ERR_NULL),
    ({"qkv": P + 8}, RN_ERR_ALIGN), ({"out": P + 2}, RN_ERR_ALIGN), ({"wk": P + 8}, RN_ERR_ALIGN),
    ({"table": P + 4}, RN_ERR_ALIGN), ({"pos": P + 4}, RN_ERR_ALIGN),
    ({"os": 1032}, RN_ERR_ARG),  # in place with other strides
])
def test_axes_arguments(lib, call, kw, expect):
    assert call(lib, **kw) == expect


def test_axes_calls_without_work(lib):
    assert fwd(lib, T=0) == RN_OK
    assert fwd(lib, Hq=0, Hkv=0) == RN_OK
    assert bwd(lib, T=0, dwq=None, dwk=None) == RN_OK


@pytest.mark.parametrize("kw,expect", [
    ({"gs": 760}, RN_ERR_SHAPE), ({"dout": None}, RN_ERR_NULL), ({"ws": None}, RN_ERR_NULL),
    ({"dout": P + 8}, RN_ERR_ALIGN), ({"ws": P + 8}, RN_ERR_ALIGN), ({"dwq": P + 2}, RN_ERR_ALIGN),
    ({"dwk": P}, RN_ERR_ARG), ({"acc": 2}, RN_ERR_ARG), ({"gs": 1032}, RN_ERR_ARG),
])
def test_axes_gradient_arguments(lib, kw, expect):
    assert bwd(lib, **kw) == expect


def test_workspace_bytes_refuses_head_sizes(lib):
    assert lib.qk_norm_rope_axes_workspace_bytes(96) == RN_ERR_SHAPE


def rows(lib, dtype=0, x=P, stride=1000, targets=P, T=4, V=1000, scale=1.0, k=2, lp=P, lse=P, H=P, top=P, ids=P):
    return lib.token_logprobs_fwd(dtype, x, stride, targets, T, V, scale, k, lp, lse, H, top, ids, None)


def rows_grad(lib, dtype=0, x=P, stride=1000, targets=P, T=4, V=1000, scale=1.0, lp=P, lse=P, H=P, dp=P, dps=1, dh=P,
              dhs=1, dl=P, dls=1, out=P, os=1000):
    return lib.token_logprobs_bwd(dtype, x, stride, targets, lp, lse, H, dp, dps, dh, dhs, dl, dls, T, V, scale, out,
                                  os, None)


@pytest.mark.parametrize("call", [rows, rows_grad])
@pytest.mark.parametrize("kw,expect", [
    ({"dtype": 3}, RN_ERR_ARG), ({"dtype": -1}, RN_ERR_ARG), ({"scale": 0.0}, RN_ERR_ARG),
    ({"scale": -1.0}, RN_ERR_ARG), ({"scale": float("nan")}, RN_ERR_ARG), ({"scale": float("inf")}, RN_ERR_ARG),
    ({"T": -1}, RN_ERR_SHAPE), ({"T": 1 << 28}, RN_ERR_SHAPE), ({"V": 0}, RN_ERR_SHAPE),
    ({"V": (1 << 31) - 1}, RN_ERR_SHAPE), ({"stride": 999}, RN_ERR_SHAPE),
    ({"T": 0}, RN_OK), ({"x": None}, RN_ERR_NULL), ({"targets": None}, RN_ERR_NULL),
    ({"x": P + 1}, RN_ERR_ALIGN), ({"x": P + 2, "dtype": 2}, RN_ERR_ALIGN), ({"targets": P + 4}, RN_ERR_ALIGN),
    ({"lp": P + 2}, RN_ERR_ALIGN), ({"lse": P + 2}, RN_ERR_ALIGN), ({"H": P + 1}, RN_ERR_ALIGN),
])
def test_logprobs_arguments(lib, call, kw, expect):
    assert call(lib, **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    ({"k": -1}, RN_ERR_SHAPE), ({"k": 33}, RN_ERR_SHAPE), ({"V": 1, "k": 2}, RN_ERR_SHAPE),
    ({"top": None}, RN_ERR_NULL), ({"ids": None}, RN_ERR_NULL), ({"top": P + 2}, RN_ERR_ALIGN),
    ({"ids": P + 4}, RN_ERR_ALIGN),
])
def test_logprobs_top_arguments(lib, kw, expect):
    assert rows(lib, **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    ({"os": 999}, RN_ERR_SHAPE), ({"out": None}, RN_ERR_NULL), ({"lse": None}, RN_ERR_NULL),
    ({"lp": None}, RN_ERR_NULL), ({"H": None}, RN_ERR_NULL), ({"out": P + 1}, RN_ERR_ALIGN),
    ({"dp": P + 2}, RN_ERR_ALIGN), ({"dh": P + 2}, RN_ERR_ALIGN), ({"dl": P + 2}, RN_ERR_ALIGN),
    ({"dps": -1}, RN_ERR_SHAPE), ({"dhs": -1}, RN_ERR_SHAPE), ({"dls": -1}, RN_ERR_SHAPE),
    ({"T": 1 << 20, "V": 1 << 27, "stride": 1 << 27, "os": 1 << 27}, RN_ERR_SHAPE),
    ({"os": 1008}, RN_ERR_ARG),  # in place with another stride
])
def test_logprobs_gradient_arguments(lib, kw, expect):
    assert rows_grad(lib, **kw) == expect


def test_rope_axes():
    assert rope_axes((2, 1, 3)).axes == (0, 0, 1, 2, 2, 2)
    assert rope_axes((4, 2, 2), interleaved=True).axes == (0, 1, 2, 0, 1, 2, 0, 0)
    assert rope_axes((5,)).axes == (0,) * 5 and rope_axes((0, 2)).num_axes == 2
    assert len(RopeAxes([0, 3])) == 2 and RopeAxes([0, 3]).num_axes == 4
    for bad in ([], [4], [-1, 0]):
        with pytest.raises(ValueError):
            RopeAxes(bad)
    for bad in ((), (1, 2, 3, 4, 5), (0, 0), (-1, 5)):
        with pytest.raises(ValueError):
            rope_axes(bad)
    with pytest.raises(ValueError, match="do not fit"):
        rope_axes((2, 3, 3), interleaved=True)


def test_binding_refuses_tensors_that_are_on_no_gpu():
    x = torch.zeros(2, 768, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        binding.qk_norm_rope_axes_fwd(x, x, x, x, x, [0] * 32, 4, 2, 64, 64, 1e-6)
    with pytest.raises(ValueError, match="CUDA"):
        binding.token_logprobs_fwd(x, torch.zeros(2, dtype=torch.int64))


# ---- the definitions ------------------------------------------------------------------

@pytest.mark.parametrize("gptj", [False, True])
@pytest.mark.parametrize("r", [64, 32, 16])
def test_the_gradient_of_the_definition_is_its_differences(gptj, r):
    g = torch.Generator().manual_seed(1)
    T, Hq, Hkv, D, eps = 3, 2, 1, 64, 1e-5
    qkv = torch.randn(T, 4 * D, generator=g, dtype=torch.float64)
    wq, wk = 1 + 0.3 * torch.randn(2, D, generator=g, dtype=torch.float64)
    ang = torch.rand(20, r // 2, generator=g, dtype=torch.float64) * 6
    table = torch.cat((ang.cos(), ang.sin()), 1)
    pos = torch.randint(0, 20, (3, T), generator=g)
    axes = [i % 3 for i in range(r // 2)]
    do = torch.randn(T, 4 * D, generator=g, dtype=torch.float64)

    def loss(x, q, k):
        o, _ = axes_ref.qk_axes(x, q, k, table, pos, axes, Hq, Hkv, D, r, eps, gptj)
        return float((o.flatten(1) * do[:, :3 * D]).sum())

    (dx, dq, dk), _ = axes_ref.qk_axes_grad(do, qkv, wq, wk, table, pos, axes, Hq, Hkv, D, r, eps, gptj)
    h = 1e-5
    for which, grad in ((0, dx.flatten(1)), (1, dq), (2, dk)):
        args = [qkv, wq, wk]
        for _ in range(12):
            at = tuple(int(torch.randint(0, n, (1,), generator=g)) for n in grad.shape)
            lo, hi = args[which].clone(), args[which].clone()
            lo[at] -= h
            hi[at] += h
            d = (loss(*[hi if i == which else a for i, a in enumerate(args)]) -
                 loss(*[lo if i == which else a for i, a in enumerate(args)])) / (2 * h)
            # third derivatives are of order one here, 64-bit sums of about 100 off by 1e-13
            assert abs(d - float(grad[at])) < 1e-6


def test_the_gradient_of_log_probabilities_is_their_differences():
    g = torch.Generator().manual_seed(2)
    T, V, scale = 4, 11, 1.3
    x = torch.randn(T, V, generator=g, dtype=torch.float64) * 2
    x[1, 3] = x[1, 4] = float("-inf")
    targets = torch.tensor([2, 0, -1, 10])
    dp, dh, dl = torch.randn(3, T, generator=g, dtype=torch.float64)

    def results(v):
        return axes_ref.logprobs(v, targets, scale, 1)[0]

    lp, lse, H = results(x)[:3]
    grad, _ = axes_ref.logprobs_grad(x, targets, lp, lse, H, dp, dh, dl, scale)
    assert (grad[1, 3:5] == 0).all()
    h = 1e-5
    for t in range(T):
        for v in range(V):
            if x[t, v].isinf():
                continue
            lo, hi = x.clone(), x.clone()
            lo[t, v] -= h
            hi[t, v] += h
            d = 0.0
            for sign, y in ((1, hi), (-1, lo)):
                a, b, c = results(y)[:3]
                d += sign * float((a * dp + b * dl + c * dh).sum()) / (2 * h)
            assert abs(d - float(grad[t, v])) < 1e-7
