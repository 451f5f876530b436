"""A tensor on another device is named with the tensors that it does not go with (GPU)."""
from __future__ import annotations

import pytest
import torch

from row_normalization_gb300 import binding
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


def test_message_speaks_of_the_other_tensors():
    require_gpu()
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda:0")
    with pytest.raises(ValueError, match="wq must be on the same CUDA device as the other tensors"):
        binding._on(1, w, "wq", torch.bfloat16, 128)
