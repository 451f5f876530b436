"""Refusals of the key/value cache binding that come before any device is looked at (CPU)."""
from __future__ import annotations

import pytest
import torch

from row_normalization_gb300 import binding


def test_row_offsets_without_their_longest_sequence_are_refused():
    """Sequences of several queries would have all but their first left unwritten."""
    cache = binding.new_kv_cache(2, 2, 64, page_size=16, device="cpu")
    args = (torch.zeros(3, 4 * 64, dtype=torch.bfloat16), cache, torch.zeros(1, 2, dtype=torch.int32),
            torch.ones(1, dtype=torch.int32), 4)
    with pytest.raises(ValueError, match="max_q_len"):
        binding.kv_attention_fwd(*args, cu_q=torch.tensor([0, 3]))
    # without offsets, or with both, the next check answers: the cache is on no GPU
    for kw in ({}, {"max_q_len": 2}, {"cu_q": torch.tensor([0, 3]), "max_q_len": 3}):
        with pytest.raises(ValueError, match="CUDA device"):
            binding.kv_attention_fwd(*args, **kw)
