"""The query of a layout for rows of logits refuses bad arguments on the host (CPU only)."""
from __future__ import annotations

import ctypes

import pytest
import torch

from row_normalization_gb300 import binding
from row_normalization_gb300.binding import RN_ERR_ARG, RN_ERR_DEVICE, RN_ERR_NULL, RN_ERR_SHAPE
from row_normalization_gb300.build import build


@pytest.fixture(scope="module")
def lib():
    build()
    return binding.load()


@pytest.mark.parametrize("kw,expect", [
    ({"dtype": 3}, RN_ERR_ARG), ({"dtype": -1}, RN_ERR_ARG), ({"T": 0}, RN_ERR_SHAPE), ({"T": -1}, RN_ERR_SHAPE),
    ({"T": 1 << 28}, RN_ERR_SHAPE), ({"V": 0}, RN_ERR_SHAPE), ({"V": (1 << 31) - 64}, RN_ERR_SHAPE),
    ({"threads": False}, RN_ERR_NULL), ({"blocks": False}, RN_ERR_NULL),
])
def test_layout_query_arguments(lib, kw, expect):
    a = dict(dtype=0, T=4, V=1000, threads=True, blocks=True) | kw
    places = [ctypes.byref(ctypes.c_int()) if a[name] else None for name in ("threads", "blocks")]
    assert lib.token_logprobs_select_layout(a["dtype"], a["T"], a["V"], *places) == expect


def test_layout_query_needs_a_device(lib):
    if torch.cuda.is_available():
        pytest.skip("there is one")
    places = [ctypes.byref(ctypes.c_int()) for _ in range(2)]
    assert lib.token_logprobs_select_layout(0, 4, 1000, *places) == RN_ERR_DEVICE
    with pytest.raises(TypeError):
        binding.token_logprobs_select_layout(torch.int32, 4, 1000)
