"""Workloads of the training and scoring operators: what is computed, in plain
torch operations and through the library, at the sizes a model of text, images
and video meets.

Four operators, two with their gradients:

* ``rope``           per-head RMSNorm of queries and keys, then rotary positions with several
  axes (time, height, width): every pair of dimensions turns by the position of its own axis;
* ``rope_grad``      its gradient, with those of the two weights;
* ``logprobs``       log probabilities of given tokens, log-sum-exp, entropy and the largest
  alternatives of rows of logits;
* ``logprobs_grad``  the gradient of log probability, entropy and log-sum-exp by the logits.

Head layouts are those of the fused Q/K norm + RoPE workloads of this repository (32 query
and 8 key/value heads of 128; heads of 64 and 256).
"""
import math
import random

import torch

own = False

EPS = 1e-6
TABLE = 32768     # positions of the cos/sin table
DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _rope(op, T, Hq, Hkv, D, r, sections, interleaved=False, style="neox", dtype="bf16",
          table="fp32", pad=0, text=0.3, name=None):
    c = {"op": op, "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "r": r, "sections": sections,
         "interleaved": interleaved, "style": style, "dtype": dtype, "table": table, "pad": pad,
         "text": text}
    if name:
        c["name"] = name
    return c


def _rows(op, T, V, dtype="bf16", k=0, scale=1.0, banned=0.0, pad=0, name=None):
    c = {"op": op, "T": T, "V": V, "dtype": dtype, "k": k, "scale": scale, "banned": banned,
         "pad": pad}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # a decode step: one text token for each of 48 running sequences
        _rope("rope", 48, 32, 8, 128, 128, "16,24,24", text=1.0, name="rope_decode"),
        # a prompt with images, sections one after another
        _rope("rope", 4096, 32, 8, 128, 128, "16,24,24", name="rope_prompt"),
        # a long video with wide heads that turn half of their dimensions, axes interleaved
        _rope("rope", 16384, 16, 4, 256, 128, "24,20,20", interleaved=True, text=0.05,
              name="rope_video"),
        # fine-tuning on short samples: fp16, neighbouring pairs, two axes, an odd token count
        _rope("rope_grad", 777, 32, 8, 64, 64, "16,16", style="gptj", dtype="fp16",
              name="rope_grad_short"),
        # a training batch
        _rope("rope_grad", 16384, 32, 8, 128, 128, "16,24,24", name="rope_grad_batch"),
        # one sampled token of one request, fp32 logits of an odd vocabulary
        _rows("logprobs", 1, 50021, "fp32", k=5, name="logprobs_one"),
        # a sampling step with temperature; most tokens banned by a grammar
        _rows("logprobs", 32, 131072, "bf16", k=20, scale=1.25, banned=0.9, name="logprobs_step"),
        # scoring a batch of prompts with alternatives
        _rows("logprobs", 2048, 131072, "bf16", k=8, name="logprobs_prompts"),
        # the log probabilities of a training batch, fp16 rows of an odd vocabulary, padded
        _rows("logprobs", 1500, 50021, "fp16", pad=3, name="logprobs_batch_odd"),
        # the gradient of a policy step's log probabilities and entropy bonus
        _rows("logprobs_grad", 4096, 131072, "bf16", name="policy_grad"),
        # the same with fp32 logits of an odd vocabulary, at a temperature
        _rows("logprobs_grad", 333, 50021, "fp32", scale=0.8, name="policy_grad_fp32_odd"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope_grad", "logprobs", "logprobs", "logprobs_grad"])
    if op.startswith("rope"):
        D = rng.choice([64, 128, 128, 256])
        r = D // rng.choice([1, 1, 2, 4])
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 8])
        T = _log_int(rng, 1, min(65536, 2 ** 26 // ((Hq + Hkv) * D)))
        A = rng.randrange(1, 5)
        cuts = sorted(rng.sample(range(1, r // 2), A - 1)) if r // 2 > A else list(range(1, A))
        sections = [b - a for a, b in zip([0] + cuts, cuts + [r // 2])]
        interleaved = A > 1 and rng.random() < 0.4
        if interleaved:
            # axes 1.. take every A-th pair, axis 0 the rest
            n = r // 2 // A
            sections = [r // 2 - (A - 1) * n] + [n] * (A - 1)
        return _rope(op, T, Hq, Hkv, D, r, ",".join(map(str, sections)), interleaved,
                     rng.choice(["neox", "neox", "gptj"]), rng.choice(["bf16", "bf16", "fp16"]),
                     rng.choice(["fp32", "bf16"]), rng.choice([0, 0, 8, 64]),
                     rng.choice([0.0, 0.3, 1.0]))
    T = _log_int(rng, 1, 4096)
    V = _log_int(rng, 1000, 131072)
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if dtype == "fp32" or op == "logprobs":
        T = max(1, min(T, 2 ** 28 // V))
    return _rows(op, T, V, dtype, rng.choice([0, 1, 5, 20]) if op == "logprobs" else 0,
                 rng.choice([1.0, 1.0, 0.7, 1.6]), rng.choice([0.0, 0.0, 0.5, 0.99]),
                 rng.choice([0, 0, 3, 8]))


# ---- sizes ------------------------------------------------------------------

def work(case):
    e = 4 if case["dtype"] == "fp32" else 2
    T = case["T"]
    if case["op"].startswith("rope"):
        n = T * (case["Hq"] + case["Hkv"]) * case["D"]
        # a token's positions; of the table no more than its rows, of its columns once each token
        axes = T * 8 * len(case["sections"].split(","))
        table = min(T, TABLE) * case["r"] * (4 if case["table"] == "fp32" else 2)
        if case["op"] == "rope":
            return {"bytes": 2 * n * e + axes + table + 2 * case["D"] * e, "flops": 9 * n}
        return {"bytes": 3 * n * e + axes + table + 2 * case["D"] * (e + 4), "flops": 18 * n}
    n = T * case["V"]
    if case["op"] == "logprobs":
        return {"bytes": n * e + T * (8 + 12 + 12 * case["k"]), "flops": 7 * n}
    return {"bytes": 2 * n * e + T * 32, "flops": 7 * n}


# ---- inputs -----------------------------------------------------------------

def _axes(case):
    """The axis that turns each pair."""
    sections = [int(s) for s in case["sections"].split(",")]
    A = len(sections)
    if not case["interleaved"]:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    axes = [0] * (case["r"] // 2)
    for a in range(1, A):
        axes[a:a + A * sections[a]:A] = [a] * sections[a]
    return axes


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    T, dtype = case["T"], DTYPE[case["dtype"]]
    st = {"case": case}
    if case["op"].startswith("rope"):
        return _prepare_rope(st, case, T, dtype, gen, seed)
    V = case["V"]
    # most rows spread over many tokens, some are nearly sure of one
    room = torch.empty(T, V + case["pad"], dtype=dtype, device=dev)
    x = torch.randn(T, V, generator=gen, device=dev).mul_(2.0)
    targets = torch.randint(0, V, (T,), generator=gen, device=dev)
    if case["banned"]:
        # the same tokens in every row, as a grammar bans them; the given ones stay
        ban = torch.rand(V, generator=gen, device=dev) < case["banned"]
        kept = x.gather(1, targets[:, None])
        x[:, ban] = float("-inf")
        x.scatter_(1, targets[:, None], kept)
    sure = torch.rand(T, 1, generator=gen, device=dev) * 14.0
    x.scatter_add_(1, targets[:, None], sure)
    room[:, :V] = x
    del x
    st["logits"], st["targets"] = room[:, :V], targets
    if case["op"] == "logprobs_grad":
        # as the forward pass left them, and what the loss hands back
        s = st["logits"].double() * case["scale"]
        lse = torch.logsumexp(s, 1)
        p = torch.exp(s - lse[:, None])
        st["logprobs"] = (s.gather(1, targets[:, None]).squeeze(1) - lse).float()
        st["lse"] = lse.float()
        st["entropy"] = (lse - torch.where(p > 0, p * s, 0.0).sum(1)).float()
        st["dlogprobs"] = torch.randn(T, generator=gen, device=dev)
        st["dentropy"] = torch.randn(T, generator=gen, device=dev) * 0.1
        st["dlse"] = torch.randn(T, generator=gen, device=dev) * 0.01
        del s, p
        st["dlogits"] = torch.empty(T, V, dtype=dtype, device=dev)
    return st


def _prepare_rope(st, case, T, dtype, gen, seed):
    dev = "cuda"
    D, Hq, Hkv, r = case["D"], case["Hq"], case["Hkv"], case["r"]
    W, axes = (Hq + 2 * Hkv) * D, _axes(case)
    A = len(case["sections"].split(","))
    qkv = torch.randn(T, W + case["pad"], generator=gen, device=dev).mul_(1.3).to(dtype)
    st["qkv"] = qkv[:, :W]
    st["wq"], st["wk"] = (1.0 + 0.2 * torch.randn(2, D, generator=gen, device=dev)).to(dtype)
    # text first: one position on every axis; then frames of a video, each a grid of patches
    rng = random.Random(seed)
    n_text = int(T * case["text"])
    rows, cols = rng.randrange(8, 33), rng.randrange(8, 49)
    base = rng.randrange(0, TABLE // 2)
    i = torch.arange(T, device=dev)
    j = (i - n_text).clamp(min=0)
    grid = torch.stack([j // (rows * cols), j // cols % rows, j % cols, j // 7])[:A] + n_text
    st["positions"] = (base + torch.where(i < n_text, i, grid)) % TABLE
    st["axes"] = torch.tensor(axes, device=dev)
    h = r // 2
    angle = torch.arange(TABLE, dtype=torch.float64, device=dev)[:, None] * \
        10000.0 ** (-torch.arange(h, dtype=torch.float64, device=dev) / h)
    st["table"] = torch.cat((angle.cos(), angle.sin()), 1).to(DTYPE[case["table"]])
    n = (Hq + Hkv) * D
    if case["op"] == "rope":
        st["out"] = torch.empty(T, n, dtype=dtype, device=dev)
    else:
        st["dout"] = torch.randn(T, W, generator=gen, device=dev).to(dtype)
        st["dx"] = torch.empty(T, n, dtype=dtype, device=dev)
    if own:
        import row_normalization_gb300 as rn
        st["rope_axes"] = rn.RopeAxes(axes)
        if case["op"] == "rope_grad":
            st["workspace"] = rn.qk_norm_rope_axes_workspace(D)
    return st


# ---- one pass ---------------------------------------------------------------

def run(st):
    case = st["case"]
    return _run_own(st, case) if own else _run_plain(st, case)


def _run_own(st, case):
    import row_normalization_gb300 as rn
    if case["op"].startswith("rope"):
        style = rn.RN_ROPE_GPTJ if case["style"] == "gptj" else rn.RN_ROPE_NEOX
        sizes = (case["Hq"], case["Hkv"], case["D"], case["r"], EPS)
        if case["op"] == "rope":
            return rn.qk_norm_rope_axes_fwd(
                st["qkv"], st["wq"], st["wk"], st["table"], st["positions"], st["rope_axes"],
                *sizes, rope_style=style, out=st["out"])
        return rn.qk_norm_rope_axes_bwd(
            st["dout"], st["qkv"], st["wq"], st["wk"], st["table"], st["positions"],
            st["rope_axes"], *sizes, rope_style=style, dx=st["dx"], workspace=st["workspace"])
    if case["op"] == "logprobs":
        got = rn.token_logprobs_fwd(st["logits"], st["targets"], scale=case["scale"],
                                    top_k=case["k"])
        return tuple(got) if case["k"] else tuple(got)[:3]
    forward = rn.TokenLogprobs(st["logprobs"], st["lse"], st["entropy"])
    return rn.token_logprobs_bwd(st["logits"], st["targets"], forward, st["dlogprobs"],
                                 st["dentropy"], st["dlse"], scale=case["scale"],
                                 dlogits=st["dlogits"])


def _turn(x, c, s, style):
    """Every pair of x [T, H, r] turned by the angle of cosine c and sine s [T, 1, r / 2]."""
    if style == "gptj":
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat((a * c - b * s, b * c + a * s), -1)


def _run_plain(st, case):
    if case["op"].startswith("rope"):
        return _rope_plain(st, case)
    s = st["logits"].float() * case["scale"]
    rows = torch.arange(case["T"], device=s.device)
    if case["op"] == "logprobs_grad":
        lp = s - st["lse"][:, None]
        p = torch.exp(lp)
        g = -p * (st["dlogprobs"] - st["dlse"])[:, None]
        g -= torch.where(p > 0, p * (lp + st["entropy"][:, None]), 0.0) * st["dentropy"][:, None]
        # where a given token is nearly sure, 1 - p is all there is
        lt = st["logprobs"].double()
        pt = torch.exp(lt)
        gt = pt * st["dlse"] - torch.expm1(lt) * st["dlogprobs"] - \
            pt * (lt + st["entropy"]) * st["dentropy"]
        g[rows, st["targets"]] = gt.float()
        return (g * case["scale"]).to(DTYPE[case["dtype"]])
    m = s.amax(1, keepdim=True)
    d = s - m
    e = torch.exp(d)
    z = e.sum(1, dtype=torch.float64)
    lz = torch.log(z)
    entropy = lz - torch.where(e > 0, e * d, 0.0).sum(1, dtype=torch.float64) / z
    out = ((d[rows, st["targets"]] - lz).float(), (m.squeeze(1) + lz).float(), entropy.float())
    if case["k"] == 0:
        return out
    # the k largest, the lowest index first among equals: by one whole number for each
    u = (st["logits"].float() + 0.0).view(torch.int32).long()
    u = torch.where(u < 0, -(u & 0x7FFFFFFF), u)
    key = u * 2 ** 31 + (2 ** 31 - 1 - torch.arange(case["V"], device=s.device))
    ids = 2 ** 31 - 1 - torch.topk(key, case["k"], 1).values % 2 ** 31
    return out + ((d.gather(1, ids) - lz[:, None]).float(), ids)


def _rope_plain(st, case):
    T, Hq, Hkv, D, r = (case[k] for k in ("T", "Hq", "Hkv", "D", "r"))
    H, dtype = Hq + Hkv, DTYPE[case["dtype"]]
    x = st["qkv"][:, :H * D].float().view(T, H, D)
    w = torch.cat((st["wq"].expand(Hq, D), st["wk"].expand(Hkv, D))).float()
    pair = torch.arange(r // 2, device=x.device)
    pos = st["positions"][st["axes"]].T                           # [T, r / 2]
    c = st["table"][pos, pair].float()[:, None]
    s = st["table"][pos, pair + r // 2].float()[:, None]
    rstd = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    n = x * rstd
    if case["op"] == "rope":
        y = n * w
        return torch.cat((_turn(y[..., :r], c, s, case["style"]), y[..., r:]), -1) \
            .to(dtype).view(T, H * D)
    g = st["dout"][:, :H * D].float().view(T, H, D)
    g = torch.cat((_turn(g[..., :r], c, -s, case["style"]), g[..., r:]), -1)
    dw = (g * n).sum(0, dtype=torch.float64)
    u = g * w
    dx = rstd * (u - n * (u * n).mean(-1, keepdim=True))
    return dx.to(dtype).view(T, H * D), dw[:Hq].sum(0).float(), dw[Hq:].sum(0).float()


# ---- the definitions in 64 bits ---------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return _exact_rope(st, case) if case["op"].startswith("rope") else _exact_rows(st, case)


def _exact_rope(st, case):
    T, Hq, Hkv, D, r = (case[k] for k in ("T", "Hq", "Hkv", "D", "r"))
    grad = case["op"] == "rope_grad"
    at = st["positions"].index_select(0, st["axes"])               # [r / 2, T]
    wide = st["table"].double()
    turn = torch.complex(wide[:, :r // 2], wide[:, r // 2:]).T.gather(1, at).T   # [T, r / 2]
    res, dws = [], []
    for first, heads, w in ((0, Hq, st["wq"]), (Hq, Hkv, st["wk"])):
        x = st["qkv"][:, first * D:(first + heads) * D].double().reshape(T, heads, D)
        w = w.double()
        if grad:
            x.requires_grad_()
            w.requires_grad_()
        y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + EPS) * w
        if case["style"] == "gptj":
            z = torch.complex(y[..., 0:r:2], y[..., 1:r:2]) * turn[:, None]
            o = torch.cat((torch.view_as_real(z).reshape(T, heads, r), y[..., r:]), -1)
        else:
            z = torch.complex(y[..., :r // 2], y[..., r // 2:r]) * turn[:, None]
            o = torch.cat((z.real, z.imag, y[..., r:]), -1)
        if grad:
            do = st["dout"][:, first * D:(first + heads) * D].double().reshape(T, heads, D)
            o, dw = torch.autograd.grad(o, (x, w), do)
            dws.append(dw)
        res.append(o.detach().reshape(T, heads * D))
    res = torch.cat(res, 1)
    return (res, *dws) if grad else res


def _exact_rows(st, case):
    parts = []
    step = max(1, 2 ** 27 // case["V"])
    for a in range(0, case["T"], step):
        x = st["logits"][a:a + step].double()
        t = st["targets"][a:a + step, None]
        if case["op"] == "logprobs_grad":
            x.requires_grad_()
        lp = torch.log_softmax(x * case["scale"], 1)
        lse = torch.logsumexp(x * case["scale"], 1)
        p = lp.exp()
        entropy = -(p * lp.masked_fill(p == 0, 0.0)).sum(1)
        if case["op"] == "logprobs_grad":
            loss = (lp.gather(1, t).squeeze(1) * st["dlogprobs"][a:a + step] +
                    entropy * st["dentropy"][a:a + step] + lse * st["dlse"][a:a + step]).sum()
            parts.append((torch.autograd.grad(loss, x)[0],))
        else:
            out = (lp.gather(1, t).squeeze(1), lse, entropy)
            if case["k"]:
                ids = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :case["k"]]
                out += (lp.gather(1, ids), ids)
            parts.append(out)
    out = tuple(torch.cat(p) for p in zip(*parts))
    return out[0] if case["op"] == "logprobs_grad" else out
