"""The several-axes Q/K step, the cache, attention and log probabilities together, as a
program that answers and one that learns use them (GPU)."""
from __future__ import annotations

import pytest
import torch

from row_normalization_gb300 import binding
from tests import axes_ref, kv_ref
from tests.axes_ref import assert_near, half
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
HQ, HKV, D, R, EPS, VOCAB = 8, 2, 64, 64, 1e-6, 5003
AXES = (16, 8, 8)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    binding.device_status()


def image_positions(T, n_text, rows, cols):
    """Text, one position on all axes; then frames of rows x cols patches."""
    i = torch.arange(T, device="cuda")
    j = (i - n_text).clamp(min=0)
    grid = torch.stack((j // (rows * cols), j // cols % rows, j % cols)) + n_text
    return torch.where(i < n_text, i, grid)


def weights(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    wq, wk = (1 + 0.2 * torch.randn(2, D, generator=g, device="cuda")).to(BF)
    head = (torch.randn(HQ * D, VOCAB, generator=g, device="cuda") * 0.15).to(BF)
    return wq, wk, head, g


def test_a_prompt_with_an_image_is_scored_and_a_token_sampled():
    """Prompt chunk and then a single token: each step against the 64-bit definition of what
    the step before it left."""
    wq, wk, head, g = weights(1)
    axes, table = binding.rope_axes(AXES), binding.rope_cos_sin_table(1e4, 256, R)
    T, P = 70, 16
    cache = binding.new_kv_cache(16, HKV, D, page_size=P, format=binding.RN_KV_INT8)
    pages = torch.randperm(16, generator=g, device="cuda")[:6].to(torch.int32)
    at = torch.arange(T + 1, device="cuda")
    slots = pages[at // P].long() * P + at % P
    positions = image_positions(T + 1, 20, 5, 6)
    qkv = torch.randn(T + 1, (HQ + 2 * HKV) * D, generator=g, device="cuda").to(BF)
    tokens = torch.randint(0, VOCAB, (T + 1,), generator=g, device="cuda")
    tokens[3] = -1                                           # not scored
    kept = []
    for a, b in ((0, T), (T, T + 1)):
        x = qkv[a:b].clone()
        want, slack = axes_ref.qk_axes(x, wq, wk, table, positions[:, a:b], axes.axes, HQ, HKV, D, R, EPS, False)
        binding.qk_norm_rope_axes_fwd(x, wq, wk, table, positions[:, a:b], axes, HQ, HKV, D, R, EPS)
        assert_near(x[:, :(HQ + HKV) * D].reshape(want.shape), want, slack, "queries and keys")
        assert torch.equal(x[:, (HQ + HKV) * D:], qkv[a:b, (HQ + HKV) * D:])
        kept.append(x)
        binding.kv_cache_write(x, slots[a:b].contiguous(), cache, HQ, HKV, D)
        out, lse = binding.kv_attention_fwd(
            x, cache, pages[None], torch.tensor([b], dtype=torch.int32, device="cuda"), HQ,
            cu_q=torch.tensor([0, b - a], device="cuda"), max_q_len=b - a)
        heads = torch.cat(kept).cpu().view(b, HQ + 2 * HKV, D)
        codes, scales = kv_ref.quantise(heads[:, HQ:].unflatten(1, (2, HKV)), 8)
        vals = kv_ref.values(codes, scales)
        o, l, _ = kv_ref.attention(heads[a:, :HQ], vals[:, 0], vals[:, 1], b, D ** -0.5)
        # values up to about 4: half a step of bf16 there, and weights rounded by 2^-11
        assert (out.cpu().double() - o).abs().max() <= 2.0 ** -6
        assert (lse.cpu().double() - l).abs().max() <= 2.0 ** -13
        logits = out.view(b - a, HQ * D) @ head
        logits[:, 100:200] = float("-inf")                   # a grammar's ban
        scored = binding.token_logprobs_fwd(logits, tokens[a:b].contiguous(), scale=0.9, top_k=5)
        want, slack = axes_ref.logprobs(logits, tokens[a:b], 0.9, 5)
        for got, w, s in zip(scored, want, slack):
            assert_near(got, w, s, "log probabilities")
        assert torch.equal(scored.top_ids, want[4])
    assert binding.device_status() == 0


def attention(q, k, v, dtype):
    """Causal attention [T, HQ, D] in `dtype`."""
    T = q.shape[0]
    k, v = (x.repeat_interleave(HQ // HKV, 1) for x in (k, v))
    s = torch.einsum("thd,shd->hts", q, k) * D ** -0.5
    s = s.masked_fill(torch.ones(T, T, dtype=torch.bool, device=q.device).triu(1), float("-inf"))
    return torch.einsum("hts,shd->thd", torch.softmax(s, -1), v)


def test_a_policy_step_and_its_gradients():
    """Loss = -mean(advantage log p) - 0.01 mean(entropy), from qkv to the loss and back.

    Against 64-bit autograd.  On the way results are rounded to bf16 (by 2^-8 of each value
    at most): queries, keys, attention, logits, dlogits, the gradients of attention's inputs
    and dx; a logit of up to 8 that is off by 8 * 2^-8 moves its weight by 2^-5 of itself.
    All of them the same way would be 7 * 2^-8 + 2^-5 = 0.06 of a gradient's norm."""
    wq, wk, head, g = weights(2)
    axes, table = binding.rope_axes(AXES, interleaved=True), binding.rope_cos_sin_table(1e4, 256, R)
    T, n = 96, (HQ + HKV) * D
    positions = image_positions(T, 10, 4, 6)
    qkv = torch.randn(T, (HQ + 2 * HKV) * D, generator=g, device="cuda").to(BF)
    tokens = torch.randint(0, VOCAB, (T,), generator=g, device="cuda")
    advantage = torch.randn(T, generator=g, device="cuda")

    # the step
    qk = binding.qk_norm_rope_axes_fwd(qkv, wq, wk, table, positions, axes, HQ, HKV, D, R, EPS,
                                       out=torch.empty(T, n, dtype=BF, device="cuda"))
    leaves = torch.cat((qk, qkv[:, n:]), 1).float().requires_grad_()
    h = leaves.view(T, HQ + 2 * HKV, D)
    mixed = attention(h[:, :HQ], h[:, HQ:HQ + HKV], h[:, HQ + HKV:], torch.float32).reshape(T, HQ * D)
    logits = mixed.detach().to(BF) @ head
    forward = binding.token_logprobs_fwd(logits, tokens)
    dlogits = binding.token_logprobs_bwd(logits, tokens, forward, -advantage / T,
                                         torch.tensor(-0.01 / T, device="cuda").expand(T))
    dmixed = dlogits @ head.T
    dhead = mixed.detach().to(BF).T @ dlogits
    (dleaves,) = torch.autograd.grad(mixed, leaves, dmixed.float())
    dqkv, dwq, dwk = binding.qk_norm_rope_axes_bwd(dleaves.to(BF), qkv, wq, wk, table, positions, axes, HQ, HKV, D,
                                                   R, EPS)

    # its definition
    x, a, b, w = (v.double().requires_grad_() for v in (qkv, wq, wk, head))
    o, _ = axes_ref.qk_axes(x, a, b, table, positions, axes.axes, HQ, HKV, D, R, EPS, False)
    v = x[:, n:].reshape(T, HKV, D)
    z = attention(o[:, :HQ], o[:, HQ:], v, torch.float64).reshape(T, HQ * D) @ w
    lp = torch.log_softmax(z, 1)
    loss = -(lp.gather(1, tokens[:, None]).squeeze(1) * advantage).mean() + \
        0.01 * (lp.exp() * lp).sum(1).mean()
    wants = torch.autograd.grad(loss, (x, a, b, w))
    got_loss = -(forward.logprobs.double() * advantage).mean() - 0.01 * forward.entropy.double().mean()
    assert abs(float(got_loss - loss.detach())) <= 2.0 ** -5 * float(advantage.abs().mean())
    for name, got, want in zip(("dqkv", "dwq", "dwk", "dhead"), (dqkv, dwq, dwk, dhead), wants):
        off = (got.double() - want).norm() / want.norm()
        assert off <= 0.06, f"{name}: {float(off):.3g} of its norm off"
    assert binding.device_status() == 0
