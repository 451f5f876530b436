"""Plain 64-bit definitions of the several-axes Q/K step, of token log probabilities
and of both gradients, with bounds on how far fp32 arithmetic may be from them.

A result rounded once to a format t is off by at most eps(t) / 2 of itself, on top of
what fp32 arithmetic (unit U = 2^-24) is off before; every bound counts those.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -126}


def half(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def assert_near(got: torch.Tensor, want: torch.Tensor, slack: torch.Tensor | float, what: str,
                rounds: bool = True):
    """|got - want| within `slack` (of fp32 arithmetic) and one rounding to got's type."""
    g, w = got.double(), want.double()
    bound = (1 + 2.0 ** -7) * slack + half(got.dtype) * w.abs() + TINY[got.dtype]
    same = (g == w) | (g.isnan() & w.isnan())
    off = ((g - w).abs() <= bound) | same
    if not bool(off.all()):
        ratio = ((g - w).abs() / bound).masked_fill(same, 0).nan_to_num(float("inf"))
        at = int(ratio.argmax())
        raise AssertionError(f"{what}: {int((~off).sum())} of {off.numel()} values off; worst at {at}: "
                             f"{g.flatten()[at].item()} for {w.flatten()[at].item()}, {float(ratio.max()):.3g} bounds")


# ---- the Q/K step -------------------------------------------------------------------

def turn(x, c, s, r, gptj):
    """The first r dimensions of x [T, H, D] turned; c, s [T, r / 2]."""
    c, s = c[:, None], s[:, None]
    if gptj:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        o = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        o = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((o, x[..., r:]), -1)


def angles(table, positions, axes, r):
    pos = positions[torch.tensor(axes, device=table.device)].T
    pair = torch.arange(r // 2, device=table.device)
    return table[pos, pair].double(), table[pos, pair + r // 2].double()


def heads_of(qkv, Hq, Hkv, D):
    return qkv[:, :(Hq + Hkv) * D].double().reshape(-1, Hq + Hkv, D)


def weights_of(wq, wk, Hq, Hkv):
    return torch.cat((wq.double().expand(Hq, -1), wk.double().expand(Hkv, -1)))


def qk_axes(qkv, wq, wk, table, positions, axes, Hq, Hkv, D, r, eps, gptj):
    """(results [T, H, D], slack of fp32 arithmetic).

    A sum of squares of D values is off by 20 U at most (16 of a lane one after another
    and up to 4 joins), rstd by half of that and 3 roundings, and weight, cosine, product
    and sum add 5: 18 U of the two products' sizes; 24 are allowed."""
    x, w = heads_of(qkv, Hq, Hkv, D), weights_of(wq, wk, Hq, Hkv)
    c, s = angles(table, positions, axes, r)
    n = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w
    size = turn(n.abs(), c.abs(), s.abs(), r, gptj).abs() + turn(n.abs(), c.abs(), -s.abs(), r, gptj).abs()
    return turn(n, c, s, r, gptj), 24 * U * size


def qk_axes_grad(dout, qkv, wq, wk, table, positions, axes, Hq, Hkv, D, r, eps, gptj):
    """((dx, dwq, dwk), their slacks).

    g is off by 3 U of its products, u = g w by 4, n^ by 14, the mean of u n^ by
    4 + 14 + 20 + 1 of the mean of its sizes; the difference and rstd add 12 + 2: 64 U.
    A lane's sum of g n^ has 60 terms at most in these tests, a block's 64 lanes' sums, and
    the blocks' come as 10 and 5: with 18 U a term 200 U of the sum of sizes."""
    x, w = heads_of(qkv, Hq, Hkv, D), weights_of(wq, wk, Hq, Hkv)
    do = heads_of(dout, Hq, Hkv, D)
    c, s = angles(table, positions, axes, r)
    rstd = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    n = x * rstd
    g = turn(do, c, -s, r, gptj)
    size = turn(do.abs(), c.abs(), s.abs(), r, gptj).abs() + turn(do.abs(), c.abs(), -s.abs(), r, gptj).abs()
    u, us = g * w, size * w.abs()
    dx = rstd * (u - n * (u * n).mean(-1, keepdim=True))
    dxs = 64 * U * rstd * (us + n.abs() * (us * n.abs()).mean(-1, keepdim=True))
    dw, dws = (g * n).sum(0), 200 * U * (size * n.abs()).sum(0)
    return ((dx, dw[:Hq].sum(0), dw[Hq:].sum(0)), (dxs, dws[:Hq].sum(0), dws[Hq:].sum(0)))


# ---- log probabilities ----------------------------------------------------------------

def logprobs(x, targets, scale, k):
    """(logprobs, lse, entropy, top_logprobs, top_ids) and the first four's slacks, for rows
    whose largest logit is finite.

    A term 2^t, t = (x - m) scale log2 e, is off by 3 U of |t| ln 2 and 4 U; weighted by the
    terms that is 3 U times (entropy - ln Z), at most 3 U H.  A thread adds n terms one after
    another, rescales at most once for every 8 of them (6 U each), and 60 joins follow: Z, and
    what it has beside its largest term, are off by K U, K = 4 H + 2 n + 100."""
    s = x.double() * scale
    V = x.shape[1]
    m, at = s.max(1, keepdim=True)
    d = s - m
    e = d.exp()
    # what there is beside one largest term, by itself: 64 bits lose 1e-16 beside 1, too
    rest = e.scatter(1, at, 0.0).sum(1)
    ln_z = torch.log1p(rest)
    lp = d - ln_z[:, None]
    m = m.squeeze(1)
    lse = m + ln_z
    H = ln_z - (e * d.masked_fill(e == 0, 0.0)).sum(1) / (1 + rest)
    top = torch.sort(x.double(), dim=1, descending=True, stable=True).indices[:, :k]
    K = 4 * H + 2 * (V / 512 + 8) + 100
    ln_z = K * U * rest / (1 + rest)
    t = targets.clamp(min=0)[:, None]
    ignored = targets < 0

    def row(ids):
        far = (s.gather(1, ids) - m[:, None]).abs()
        far = far.masked_fill(far.isinf(), 0.0)
        return lp.gather(1, ids), 4 * U * far + ln_z[:, None]

    given, given_slack = row(t)
    tops, top_slack = row(top)
    given = given.squeeze(1).masked_fill(ignored, 0.0)
    want = (given, lse, H, tops, top)
    slack = (given_slack.squeeze(1), 2 * U * m.abs() + ln_z, ln_z + 2 * K * U * H, top_slack)
    return want, slack


def logprobs_grad(x, targets, given, lse, entropy, dp, dh, dl, scale):
    """(gradient, slack) by the formula, with the forward results as they are given.

    s - lse = l is off by U |l|, p = e^l by (3 |l| + 4) U, c0 - c1 l by 6 U of its parts.  A
    given token's l is its log probability as it is given, where that gets a gradient."""
    T, V = x.shape
    targets = targets if dp is not None else torch.full_like(targets, -1)
    zero = torch.zeros(T, dtype=torch.float64, device=x.device)
    given, lse, entropy, dp, dh, dl = (zero if v is None else v.double()
                                       for v in (given, lse, entropy, dp, dh, dl))
    dp = dp.masked_fill(targets < 0, 0.0)
    l = x.double() * scale - lse[:, None]
    p = l.exp()
    l = l.masked_fill(p == 0, 0.0)
    want = p * (dl - dp - dh * entropy)[:, None] - p * l * dh[:, None]
    size = p * (dl.abs() + dp.abs() + (dh * entropy).abs())[:, None] + p * l.abs() * dh.abs()[:, None]
    slack = size * (3 * l.abs() + 16) * U
    rows = torch.nonzero(targets >= 0).squeeze(1)
    t = targets[rows]
    gl = given[rows]
    gp = gl.exp()
    gl = gl.masked_fill(gp == 0, 0.0)
    one = -torch.expm1(given[rows]) * dp[rows]
    want[rows, t] = one + gp * (dl[rows] - dh[rows] * (gl + entropy[rows]))
    slack[rows, t] = 16 * U * (one.abs() + gp * (dl[rows].abs() + dh[rows].abs() *
                                                 (gl.abs() + entropy[rows].abs())))
    return want * scale, (slack + 1e-37) * scale
