"""Plain 64-bit definitions of the quantised key/value cache and the attention
over it, written from the formulas of include/row_norm.h (numpy / torch on the
CPU; shares no code with the library)."""
from __future__ import annotations

import math

import numpy as np
import torch

QMAX = {4: 7, 8: 127}


def stored_order(D: int, value: bool) -> np.ndarray:
    """dims[e]: the dimension that stored element e of a row holds."""
    if value:
        return np.array([16 * b + 2 * r + h for r in range(8) for b in range(D // 16)
                         for h in range(2)])
    return np.array([32 * g + 8 * j + n for j in range(4) for g in range(D // 32)
                     for n in range(8)])


def quantise(x: torch.Tensor, bits: int):
    """x [..., D] bf16 -> (codes int64 [..., D] without offset, scales fp16 [..., D / 32])."""
    Q = QMAX[bits]
    g = x.double().unflatten(-1, (-1, 32))
    top = g.abs().amax(-1)
    ok = torch.isfinite(g).all(-1)
    # fp32 division, then fp16: the quotient is never near a tie of the second rounding but on it
    s = (top.float() / Q).clamp(max=65504.0).to(torch.float16)
    s = torch.where(ok, s, torch.full_like(s, float("nan")))
    d = torch.where(ok & (s > 0), s.double(), torch.ones_like(top)).unsqueeze(-1)
    c = torch.round(g / d).clamp(-Q, Q)
    c = torch.where((ok & (s > 0)).unsqueeze(-1), c, torch.zeros_like(c))
    return c.to(torch.int64).flatten(-2), s


def pack(codes: torch.Tensor, bits: int, value: bool) -> torch.Tensor:
    """Codes [..., D] -> stored bytes [..., D * bits / 8] uint8."""
    D = codes.shape[-1]
    c = (codes + (8 if bits == 4 else 128))[..., torch.from_numpy(stored_order(D, value))]
    if bits == 4:
        c = c[..., 0::2] + 16 * c[..., 1::2]
    return c.to(torch.uint8)


def values(codes: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    """Codes [..., D], scales [..., D / 32] -> fp64 values."""
    return codes.double() * scales.double().repeat_interleave(32, dim=-1)


def scale_bits(scales: torch.Tensor) -> np.ndarray:
    """fp16 bit patterns with every NaN as the cache's one (0xFFFF)."""
    b = scales.contiguous().view(torch.int16).numpy().view(np.uint16).copy()
    b[np.isnan(scales.numpy())] = 0xFFFF
    return b


class Cache:
    """A paged cache on the CPU, filled by slots, and its tensors on the GPU."""

    def __init__(self, pages: int, Hkv: int, D: int, P: int, bits: int, fill: int = 0x5A):
        self.bits, self.P, self.D = bits, P, D
        self.codes = torch.full((pages, 2, Hkv, P, D * bits // 8), fill, dtype=torch.uint8)
        # what was never written reads as NaN
        self.scales = torch.from_numpy(np.full((pages, 2, Hkv, P, D // 32), 0xFFFF, np.uint16)
                                       .view(np.float16))
        self.vals = torch.full((pages, 2, Hkv, P, D), float("nan"), dtype=torch.float64)

    def write(self, kv: torch.Tensor, slots: torch.Tensor):
        """kv [T, 2, Hkv, D] bf16."""
        live = (slots >= 0) & (slots < self.codes.shape[0] * self.P)
        kv, slots = kv[live], slots[live]
        c, s = quantise(kv, self.bits)
        pg, off = slots // self.P, slots % self.P
        for which in (0, 1):
            self.codes[pg, which, :, off] = pack(c[:, which], self.bits, which == 1)
            self.scales[pg, which, :, off] = torch.from_numpy(
                scale_bits(s[:, which]).view(np.float16))
            self.vals[pg, which, :, off] = values(c[:, which], s[:, which])

    def token_scales(self, table_row, which: int, lo: int, hi: int) -> torch.Tensor:
        """fp64 [hi - lo, Hkv, D]: the scale of every element, NaN as zero."""
        out = []
        for p in range(lo, hi):
            pg = int(table_row[p // self.P])
            if 0 <= pg < self.codes.shape[0]:
                sc = torch.nan_to_num(self.scales[pg, which, :, p % self.P].double(), nan=0.0)
                out.append(sc.repeat_interleave(32, dim=-1))
            else:
                out.append(torch.zeros_like(self.vals[0, which, :, 0]))
        return torch.stack(out) if out else self.vals.new_zeros(0, *self.vals.shape[2:3], self.D)

    def tokens(self, table_row, which: int, lo: int, hi: int) -> torch.Tensor:
        """fp64 [hi - lo, Hkv, D]; pages outside the cache read as zeros."""
        out = []
        for p in range(lo, hi):
            pg = int(table_row[p // self.P])
            if 0 <= pg < self.codes.shape[0]:
                out.append(self.vals[pg, which, :, p % self.P])
            else:
                out.append(torch.zeros_like(self.vals[0, which, :, 0]))
        return torch.stack(out) if out else self.vals.new_zeros(0, *self.vals.shape[2:3], self.D)


def attention(q, K, V, L: int, scale: float, window: int = 0, sinks: int = 0):
    """q [n, Hq, D], K and V [L, Hkv, D]: the newest n of L tokens.
    Returns (out, lse, weights) in fp64; weights[i][h] is (token numbers, their weights)."""
    n, Hq, D = q.shape
    G = Hq // K.shape[1] if K.shape[1] else 1
    q = q.double()
    out = torch.zeros(n, Hq, D, dtype=torch.float64)
    lse = torch.full((n, Hq), -math.inf, dtype=torch.float64)
    weights = [[None] * Hq for _ in range(n)]
    for i in range(n):
        p = L - n + i
        js = [j for j in range(0, p + 1) if window == 0 or j > p - window or j < sinks]
        if not js:
            continue
        for h in range(Hq):
            s = (K[js, h // G] @ q[i, h]) * scale
            lse[i, h] = torch.logsumexp(s, 0)
            w = torch.exp(s - lse[i, h])
            out[i, h] = w @ V[js, h // G]
            weights[i][h] = (js, w)
    return out, lse, weights
