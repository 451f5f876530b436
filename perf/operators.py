"""Workloads of the key/value cache operators: what is computed, in plain
torch operations and through the library, at the sizes serving meets.

Three operators work on one paged cache that holds keys and values in 8 or 4
bits with one fp16 scale per group of 32 elements:

* ``write``   quantise the key and value heads of a packed QKV tensor into
  their cache slots (and read the written tokens back, so that the stored
  values can be looked at);
* ``read``    gather ragged token ranges of the cache back as bf16;
* ``attend``  causal attention of ragged queries over the cache, optionally
  with a sliding window and a few first tokens that stay visible.

Head layouts are those of the fused Q/K norm + RoPE workloads of this
repository (32 query and 8 key/value heads of 128; 64 and 256 as the other
head sizes it takes), contexts reach its 131072 positions.
"""
import math
import random

import torch

own = False

BITS = {"int4": 4, "int8": 8}
QMAX = {"int4": 7, "int8": 127}


def _case(op, fmt, D, Hq, Hkv, page, B, kv, q=(1, 1), window=0, sinks=0, lens=1, name=None):
    c = {"op": op, "fmt": fmt, "D": D, "Hq": Hq, "Hkv": Hkv, "page": page, "B": B,
         "kv_lo": kv[0], "kv_hi": kv[1], "q_lo": q[0], "q_hi": q[1], "window": window,
         "sinks": sinks, "lens": lens}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one new token for each of 64 running sequences: a decode step's cache update
        _case("write", "int4", 128, 32, 8, 64, 64, (1, 9000), (1, 1), name="write_decode_int4"),
        # prompts of a prefill batch, odd lengths, 8-bit cache of 256-wide heads
        _case("write", "int8", 256, 16, 4, 32, 5, (700, 2100), (700, 2100), name="write_prefill_int8"),
        # one long prompt's chunk going into the 4-bit cache
        _case("write", "int4", 128, 32, 8, 64, 2, (16384, 16384), (8192, 8192),
              name="write_prefill_int4"),
        # a short cached prefix fetched for a prefill of the rest
        _case("read", "int8", 64, 32, 8, 16, 3, (90, 400), (90, 400), name="read_prefix_int8"),
        # cached conversations fetched for a prefill batch
        _case("read", "int4", 128, 32, 8, 64, 12, (1000, 16000), (1000, 16000),
              name="read_batch_int4"),
        # a few short conversations, one token each: latency
        _case("attend", "int4", 128, 32, 8, 64, 4, (1, 700), name="attend_short_int4"),
        # an ordinary decode batch of ragged lengths
        _case("attend", "int4", 128, 32, 8, 64, 64, (200, 16000), name="attend_decode_int4"),
        # the same service with an 8-bit cache of 64-wide heads and small pages
        _case("attend", "int8", 64, 32, 8, 16, 96, (500, 9000), name="attend_decode_int8"),
        # four full contexts
        _case("attend", "int4", 128, 32, 8, 128, 4, (131072, 131072), name="attend_long_int4"),
        # sliding-window layers with four sinks, long contexts
        _case("attend", "int4", 128, 32, 8, 64, 48, (3000, 60000), window=4096, sinks=4,
              name="attend_window_int4"),
        # a draft of a few tokens checked at once, 256-wide heads
        _case("attend", "int8", 256, 16, 2, 32, 17, (1000, 8000), (3, 5), name="attend_draft_int8"),
        # chunks of a prompt against what the cache already holds
        _case("attend", "int4", 128, 32, 8, 64, 3, (3001, 9001), (500, 1300),
              name="attend_chunk_int4"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "attend"])
    fmt = rng.choice(["int4", "int8"])
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 8])
    page = rng.choice([16, 32, 64, 128, 256])
    lens = rng.randrange(1 << 30)
    # the tokens of a case, so that its bytes stay below the largest listed ones
    room = 2 ** 28 // (Hkv * D)
    if op in ("write", "read"):
        total = _log_int(rng, 2, max(4, room // 16))
        B = _log_int(rng, 1, min(256, total))
        hi = max(1, total // B)
        lo = max(1, hi // rng.choice([1, 2, 7]))
        return _case(op, fmt, D, Hq, Hkv, page, B, (lo, hi), (lo, hi), lens=lens)
    window, sinks = (0, 0) if rng.random() < 0.6 else (_log_int(rng, 16, 4096), rng.randrange(0, 9))
    kind = rng.choice(["token", "token", "draft", "chunk"])
    if kind == "chunk":
        hi = _log_int(rng, 40, 8000)
        B = rng.randrange(1, 4)
        most = int(1.5e11 // (4 * D * Hq * hi * B))
        qhi = _log_int(rng, min(20, hi), max(1, min(1200, hi, most)))
        return _case(op, fmt, D, Hq, Hkv, page, B, (max(1, hi // 2), hi), (max(1, qhi // 3), qhi),
                     window, sinks, lens)
    total = _log_int(rng, 4, max(8, room))
    B = _log_int(rng, 1, min(128, total))
    hi = max(1, min(131072, total // B))
    q = (1, 1) if kind == "token" else (1, rng.randrange(2, 9))
    return _case(op, fmt, D, Hq, Hkv, page, B, (max(1, hi // rng.choice([1, 3, 20])), hi), q,
                 window, sinks, lens)


# ---- sizes ------------------------------------------------------------------

def _lengths(case):
    """Context length and new (or fetched) tokens of every sequence."""
    rng = random.Random(case["lens"])
    kv, q = [], []
    for _ in range(case["B"]):
        n = rng.randint(case["kv_lo"], case["kv_hi"])
        kv.append(n)
        q.append(min(n, rng.randint(case["q_lo"], case["q_hi"])))
    return kv, q


def _visible(case, L, n):
    """(cached tokens some query sees, query-token pairs) of one sequence."""
    w, s = case["window"], case["sinks"]
    pairs = 0
    for p in range(L - n, L):
        pairs += p + 1 if w == 0 or w > p else min(p + 1, w + min(s, p + 1 - w))
    first = 0 if w == 0 else max(0, L - n - w + 1)
    return L - first + min(s, first), pairs


def work(case):
    D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
    row = 2 * Hkv * (D * BITS[case["fmt"]] // 8 + D // 16)   # a token's keys, values and scales
    kv, q = _lengths(case)
    T = sum(q)
    if case["op"] == "write":
        return {"bytes": T * (2 * Hkv * D * 2 * 2 + 2 * row + 8), "flops": T * 2 * Hkv * D * 4}
    if case["op"] == "read":
        return {"bytes": T * (2 * Hkv * D * 2 + row), "flops": T * 2 * Hkv * D}
    seen, pairs = map(sum, zip(*(_visible(case, L, n) for L, n in zip(kv, q))))
    return {"bytes": seen * row + T * Hq * (2 * D * 2 + 4), "flops": 4 * D * Hq * pairs}


# ---- inputs -----------------------------------------------------------------

def _stored_order(D, value):
    """dims[e]: the head dimension that stored element e holds."""
    if value:
        return [16 * b + 2 * r + h for r in range(8) for b in range(D // 16) for h in range(2)]
    return [32 * g + 8 * j + n for j in range(4) for g in range(D // 32) for n in range(8)]


def prepare(case, seed):
    dev = "cuda"
    D, Hq, Hkv, P, B, fmt = (case[k] for k in ("D", "Hq", "Hkv", "page", "B", "fmt"))
    bits, qmax = BITS[fmt], QMAX[fmt]
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    kv, q = _lengths(case)
    T = sum(q)
    need = [-(-n // P) for n in kv]
    width = max(need)
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    table = torch.zeros(B, width, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    st = {"case": case, "kv": kv, "q": q, "T": T, "table": table,
          "kv_lens": torch.tensor(kv, dtype=torch.int32, device=dev),
          "cu_q": torch.tensor([sum(q[:i]) for i in range(B + 1)], dtype=torch.int64, device=dev),
          "starts": torch.tensor([n - m for n, m in zip(kv, q)], dtype=torch.int32, device=dev)}
    codes = torch.zeros(pages, 2, Hkv, P, D * bits // 8, dtype=torch.uint8, device=dev)
    scales = torch.zeros(pages, 2, Hkv, P, D // 32, dtype=torch.float16, device=dev)
    k_dims = torch.tensor(_stored_order(D, False), device=dev)
    v_dims = torch.tensor(_stored_order(D, True), device=dev)
    if case["op"] != "write":
        # a cache that earlier steps filled with unit-variance heads
        step = max(1, 2 ** 26 // (Hkv * P * D))
        for which, dims in ((0, k_dims), (1, v_dims)):
            for a in range(0, pages, step):
                x = torch.randn(min(step, pages - a), Hkv, P, D, generator=gen, device=dev)
                codes[a:a + step, which], scales[a:a + step, which] = _quantise(x, fmt, dims)
    if case["op"] != "read":
        # the packed tensor as the fused norm + RoPE leaves it: unit-variance heads
        qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=gen, device=dev)
        qkv[:, :Hq * D] *= 1.5
        st["qkv"] = qkv.to(torch.bfloat16)
    if case["op"] == "write":
        slots = torch.cat([_slots(table[b], torch.arange(n - m, n, device=dev), P)
                           for b, (n, m) in enumerate(zip(kv, q))])
        st["slots"] = slots
    st["codes"], st["scales"] = codes, scales
    if own:
        import row_normalization_gb300 as rn
        st["cache"] = rn.KVCache(codes, scales)
        if case["op"] == "attend":
            st["workspace"] = rn.kv_attention_workspace(st["cache"], B, Hq, max_q_len=max(q))
    else:
        st["k_dims"], st["v_dims"] = k_dims, v_dims
    return st


def _quantise(x, fmt, dims):
    """Stored bytes and fp16 scales of fp32 rows [..., D]; stored element e is dimension dims[e]."""
    qmax = QMAX[fmt]
    g = x.unflatten(-1, (-1, 32))
    s = (g.abs().amax(-1) / qmax).clamp(max=65504.0).to(torch.float16)
    d = torch.where(s > 0, s.float(), torch.ones_like(s, dtype=torch.float32)).unsqueeze(-1)
    c = torch.round(g / d).clamp(-qmax, qmax) * (s > 0).unsqueeze(-1) + (qmax + 1)
    c = c.flatten(-2)[..., dims].to(torch.uint8)
    return (c[..., 0::2] | (c[..., 1::2] << 4) if fmt == "int4" else c), s


def _slots(pages, positions, P):
    return pages[positions // P].long() * P + positions % P


# ---- one pass ---------------------------------------------------------------

def run(st):
    case = st["case"]
    return _run_own(st, case) if own else _run_plain(st, case)


def _run_own(st, case):
    import row_normalization_gb300 as rn
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "attend":
        return rn.kv_attention_fwd(
            st["qkv"], st["cache"], st["table"], st["kv_lens"], Hq, cu_q=st["cu_q"],
            max_q_len=max(st["q"]), window=case["window"], sinks=case["sinks"],
            workspace=st["workspace"])
    if case["op"] == "write":
        rn.kv_cache_write(st["qkv"], st["slots"], st["cache"], Hq, Hkv, D)
    return rn.kv_cache_read(st["cache"], st["table"], st["cu_q"], st["T"], starts=st["starts"])


def _values(st, which, slots):
    """The fp32 values [n, Hkv, D] that the cache holds at these slots."""
    case = st["case"]
    P = case["page"]
    pg, off = slots // P, slots % P
    c = st["codes"][pg, which, :, off]                    # [n, Hkv, bytes]
    s = st["scales"][pg, which, :, off].float()           # [n, Hkv, D / 32]
    if case["fmt"] == "int4":
        c = torch.stack((c & 15, c >> 4), dim=-1).flatten(-2).float() - 8.0
    else:
        c = c.float() - 128.0
    vals = torch.empty_like(c)
    vals[..., st["v_dims"] if which else st["k_dims"]] = c
    return (vals.unflatten(-1, (-1, 32)) * s.unsqueeze(-1)).flatten(-2)


def _run_plain(st, case):
    Hq, Hkv, D, P = case["Hq"], case["Hkv"], case["D"], case["page"]
    if case["op"] == "write":
        kvh = st["qkv"][:, Hq * D:].float().view(-1, 2, Hkv, D)
        pg, off = st["slots"] // P, st["slots"] % P
        for which, dims in ((0, st["k_dims"]), (1, st["v_dims"])):
            c, s = _quantise(kvh[:, which], case["fmt"], dims)
            st["codes"][pg, which, :, off] = c
            st["scales"][pg, which, :, off] = s
    if case["op"] in ("write", "read"):
        slots = torch.cat([_slots(st["table"][b], torch.arange(n - m, n, device="cuda"), P)
                           for b, (n, m) in enumerate(zip(st["kv"], st["q"]))])
        return tuple(_values(st, which, slots).to(torch.bfloat16) for which in (0, 1))
    T = st["T"]
    out = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(T, Hq, dtype=torch.float32, device="cuda")
    w, sinks, at = case["window"], case["sinks"], 0
    for b, (L, n) in enumerate(zip(st["kv"], st["q"])):
        first = max(0, L - n - w + 1) if w else 0         # nothing between sinks and here is seen
        j = torch.arange(first, L, device="cuda")
        if first > 0 and sinks > 0:
            j = torch.cat((torch.arange(0, min(sinks, first), device="cuda"), j))
        slots = _slots(st["table"][b], j, P)
        k, v = _values(st, 0, slots), _values(st, 1, slots)        # [L, Hkv, D]
        q = st["qkv"][at:at + n, :Hq * D].float().view(n, Hkv, Hq // Hkv, D)
        p = torch.arange(L - n, L, device="cuda")[:, None]
        see = j[None] <= p
        if w:
            see &= (j[None] > p - w) | (j[None] < sinks)
        s = torch.einsum("nhgd,lhd->hgnl", q, k) * D ** -0.5
        s = s.masked_fill(~see, float("-inf"))
        m = s.amax(-1, keepdim=True)
        e = torch.exp(s - m)
        z = e.sum(-1, keepdim=True)
        o = torch.einsum("hgnl,lhd->nhgd", e / z, v)
        out[at:at + n] = o.reshape(n, Hq, D).to(torch.bfloat16)
        lse[at:at + n] = (m + torch.log(z)).squeeze(-1).permute(2, 0, 1).reshape(n, Hq)
        at += n
    return out, lse


# ---- the definitions in 64 bits ---------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    D, Hq, Hkv, P = case["D"], case["Hq"], case["Hkv"], case["page"]
    four = case["fmt"] == "int4"
    qmax = QMAX[case["fmt"]]
    if case["op"] == "write":
        res = []
        for base in (Hq * D, (Hq + Hkv) * D):
            x = st["qkv"][:, base:base + Hkv * D].double().reshape(st["T"], Hkv, D // 32, 32)
            top = x.abs().max(dim=3, keepdim=True).values
            step = (top / qmax).clamp(max=65504.0).half().double()
            safe = step + (step == 0)
            res.append((torch.round(x / safe).clamp(-qmax, qmax) * step).reshape(st["T"], Hkv, D))
        return tuple(res)

    # where in a token's stored row each head dimension lies
    place = [[0] * D, [0] * D]
    for which in (0, 1):
        for e, d in enumerate(_stored_order(D, which == 1)):
            place[which][d] = e
    place = torch.tensor(place, device="cuda")

    def decode(which, b, lo, hi):
        pos = torch.arange(lo, hi, device="cuda")
        pg = st["table"][b].long()[torch.div(pos, P, rounding_mode="floor")]
        rows = st["codes"][pg, which, :, pos % P].int()
        e = place[which]
        c = rows[..., e // 2] >> (4 * (e % 2)) & 15 if four else rows[..., e]
        step = st["scales"][pg, which, :, pos % P].double().repeat_interleave(32, dim=-1)
        return (c.double() - (qmax + 1)) * step

    kv, q = st["kv"], st["q"]
    if case["op"] == "read":
        return tuple(torch.cat([decode(which, b, n - m, n) for b, (n, m) in enumerate(zip(kv, q))])
                     for which in (0, 1))
    # this card's 64-bit rate is low: about a second for each 5e11 operations
    if work(case)["flops"] + 4.0 * D * Hq * sum(kv) > 4e12:
        return None
    out = torch.zeros(st["T"], Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(st["T"], Hq, dtype=torch.float64, device="cuda")
    G, at = Hq // Hkv, 0
    for b, (L, n) in enumerate(zip(kv, q)):
        K, V = decode(0, b, 0, L), decode(1, b, 0, L)
        query = st["qkv"][at:at + n, :Hq * D].double().view(n, Hq, D)
        here = torch.arange(L, device="cuda")
        for i0 in range(0, n, 128):
            i1 = min(n, i0 + 128)
            pos = torch.arange(L - n + i0, L - n + i1, device="cuda").view(-1, 1)
            hidden = here > pos
            if case["window"]:
                hidden = hidden | ((here <= pos - case["window"]) & (here >= case["sinks"]))
            for h in range(Hq):
                logit = query[i0:i1, h] @ K[:, h // G].T / math.sqrt(D)
                logit[hidden] = -math.inf
                l = torch.logsumexp(logit, dim=1)
                out[at + i0:at + i1, h] = torch.exp(logit - l[:, None]) @ V[:, h // G]
                lse[at + i0:at + i1, h] = l
        at += n
    return out, lse
