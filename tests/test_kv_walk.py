"""The CTAs' walk over the attention's work, run on the host (CPU only): the joining
kernel's notes are complete whatever becomes of the waits."""
from __future__ import annotations

import os
import subprocess

from row_normalization_gb300 import build as b


def test_every_cut_is_noted_also_by_ctas_that_give_up(tmp_path):
    here = os.path.dirname(os.path.abspath(__file__))
    exe = str(tmp_path / "kv_walk")
    res = subprocess.run([b._nvcc(), *b.ARCH_FLAGS, *b.NVCC_FLAGS, os.path.join(here, "kv_walk.cu"),
                          "-o", exe], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    res = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and "3000 layouts" in res.stdout, res.stdout + res.stderr
    assert int(res.stdout.split(",")[1].split()[0]) > 1000
