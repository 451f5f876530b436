"""The several-axes Q/K step and its gradient against their 64-bit definitions (GPU)."""
from __future__ import annotations

import pytest
import torch

from row_normalization_gb300 import binding
from row_normalization_gb300.binding import (RN_ROPE_GPTJ, RN_ROPE_NEOX, RN_STATUS_BAD_POSITION, RowNormError, RopeAxes,
                                             rope_axes)
from tests import axes_ref
from tests.axes_ref import U, assert_near, half
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu

BF, HALF = torch.bfloat16, torch.float16
LAYOUTS = [(D, r) for D in (64, 128, 256) for r in (D, D // 2, D // 4)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    binding.device_status()


def axes_for(kind, r):
    h = r // 2
    if kind == "sections":            # multiples of four or not, as they come
        a = h // 4 + 1
        return rope_axes((a, (h - a) // 2, h - a - (h - a) // 2))
    if kind == "eights":
        return RopeAxes([min(2, i // max(4, h // 4)) for i in range(h)])
    if kind == "interleaved":
        return rope_axes((h - 2 * (h // 3), h // 3, h // 3), interleaved=True)
    if kind == "four":
        return RopeAxes([(i * 7 + i // 5) % 4 for i in range(h)])
    return RopeAxes([0] * h)


def inputs(T, Hq, Hkv, D, r, kind="sections", dtype=BF, table=torch.float32, pad=0, max_pos=500, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    W = (Hq + 2 * Hkv) * D
    axes = axes_for(kind, r)
    st = dict(
        qkv=(torch.randn(T, W + pad, generator=g, device="cuda") * 1.4).to(dtype)[:, :W],
        dout=torch.randn(T, W + 2 * pad, generator=g, device="cuda").to(dtype)[:, :W],
        wq=(1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(dtype),
        wk=(1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(dtype),
        table=binding.rope_cos_sin_table(1e4, max_pos, r, dtype=table),
        positions=torch.randint(0, max_pos, (axes.num_axes, T), generator=g, device="cuda"),
        axes=axes)
    return st


def forward(st, sizes, **kw):
    return binding.qk_norm_rope_axes_fwd(st["qkv"], st["wq"], st["wk"], st["table"], st["positions"], st["axes"],
                                         *sizes, **kw)


def backward(st, sizes, **kw):
    return binding.qk_norm_rope_axes_bwd(st["dout"], st["qkv"], st["wq"], st["wk"], st["table"], st["positions"],
                                         st["axes"], *sizes, **kw)


def want_forward(st, sizes, style):
    return axes_ref.qk_axes(st["qkv"], st["wq"], st["wk"], st["table"], st["positions"], st["axes"].axes, *sizes,
                            style == RN_ROPE_GPTJ)


def want_backward(st, sizes, style):
    return axes_ref.qk_axes_grad(st["dout"], st["qkv"], st["wq"], st["wk"], st["table"], st["positions"],
                                 st["axes"].axes, *sizes, style == RN_ROPE_GPTJ)


def check_both(st, sizes, style, what):
    Hq, Hkv, D = sizes[:3]
    T = st["qkv"].shape[0]
    want, slack = want_forward(st, sizes, style)
    grads, slacks = want_backward(st, sizes, style)
    n = (Hq + Hkv) * D
    out = torch.empty(T, n, dtype=st["qkv"].dtype, device="cuda")
    before = st["qkv"].clone()
    assert forward(st, sizes, rope_style=style, out=out) is out
    assert torch.equal(before, st["qkv"])
    assert_near(out.view(T, -1, D), want, slack, what)
    dx = torch.empty_like(out)
    got = backward(st, sizes, rope_style=style, dx=dx)
    assert got[0] is dx and torch.equal(before, st["qkv"])
    for name, a, b, s in zip(("dx", "dwq", "dwk"), got, grads, slacks):
        assert_near(a.view(b.shape), b, s, f"{what} {name}")
    # in place: the same bits, and the value heads as they were
    dout, values = st["dout"].clone(), st["dout"][:, n:].clone()
    st2 = dict(st, dout=dout)
    again = backward(st2, sizes, rope_style=style)
    assert again[0] is dout and torch.equal(dout[:, :n], dx) and torch.equal(dout[:, n:], values)
    assert torch.equal(again[1], got[1]) and torch.equal(again[2], got[2])
    assert forward(st, sizes, rope_style=style) is st["qkv"]
    assert torch.equal(st["qkv"][:, :n], out) and torch.equal(st["qkv"][:, n:], before[:, n:])
    assert binding.device_status() == 0


@pytest.mark.parametrize("D,r", LAYOUTS)
@pytest.mark.parametrize("style", [RN_ROPE_NEOX, RN_ROPE_GPTJ])
@pytest.mark.parametrize("dtype", [BF, HALF])
@pytest.mark.parametrize("kind,table", [("sections", torch.float32), ("eights", BF), ("interleaved", torch.float32),
                                        ("four", BF), ("one", torch.float32)])
def test_every_layout(D, r, style, dtype, kind, table):
    sizes = (3, 1, D, r, 1e-6)
    check_both(inputs(13, 3, 1, D, r, kind, dtype, table), sizes, style, f"D {D} r {r} {kind}")


@pytest.mark.parametrize("T,Hq,Hkv,D,pad", [
    (1, 1, 1, 64, 0), (1, 32, 8, 128, 0), (2, 5, 5, 256, 8), (3, 17, 1, 128, 24), (31, 9, 3, 64, 8),
    (300, 32, 8, 128, 64), (1000, 12, 4, 64, 0), (513, 20, 4, 256, 0), (2500, 33, 1, 64, 0)])
@pytest.mark.parametrize("style", [RN_ROPE_NEOX, RN_ROPE_GPTJ])
def test_token_and_head_counts(T, Hq, Hkv, D, pad, style):
    """From one head of one token to heads in uneven parts, with strided rows."""
    check_both(inputs(T, Hq, Hkv, D, D // 2, pad=pad), (Hq, Hkv, D, D // 2, 1e-6), style, f"T {T} {Hq}+{Hkv}")


@pytest.mark.parametrize("Hq,Hkv", [(4, 0), (0, 4)])
def test_query_or_key_heads_alone(Hq, Hkv):
    st = inputs(40, Hq, Hkv, 64, 64)
    sizes = (Hq, Hkv, 64, 64, 1e-6)
    want, slack = want_forward(st, sizes, RN_ROPE_NEOX)
    grads, slacks = want_backward(st, sizes, RN_ROPE_NEOX)
    out = torch.empty(40, 4 * 64, dtype=BF, device="cuda")
    assert_near(forward(st, sizes, out=out).view(want.shape), want, slack, "results")
    for a, b, s in zip(backward(st, sizes, dx=out), grads, slacks):
        assert_near(a.view(b.shape), b, s, "gradient")
    dw = backward(st, sizes, dx=out)[1 if Hq == 0 else 2]
    assert (dw == 0).all()


def test_one_axis_is_the_one_axis_step():
    """The same rows through qk_norm_rope_fwd: apart by what two roundings can be."""
    st = inputs(700, 8, 2, 128, 64, "one")
    sizes = (8, 2, 128, 64, 1e-6)
    want, slack = want_forward(st, sizes, RN_ROPE_NEOX)
    packed = st["qkv"].clone()
    binding.qk_norm_rope_fwd(packed, st["wq"], st["wk"], st["table"], st["positions"][0].contiguous(), *sizes)
    forward(st, sizes)
    got = st["qkv"][:, :1280].double().view(want.shape)
    other = packed[:, :1280].double().view(want.shape)
    assert ((got - other).abs() <= 2 * (half(BF) * want.abs() + 1.01 * slack) + 1e-30).all()
    assert torch.equal(packed[:, 1280:], st["qkv"][:, 1280:])


def test_rows_behind_and_columns_beside_stay_as_they_were():
    T, D, sizes = 21, 64, (3, 1, 64, 64, 1e-6)
    st = inputs(T, 3, 1, D, 64)
    for call, name in ((forward, "out"), (backward, "dx")):
        room = torch.full((T + 2, 4 * D + 40), 7.0, dtype=BF, device="cuda")
        call(st, sizes, **{name: room[1:T + 1, 16:16 + 4 * D]})
        torch.cuda.synchronize()
        mask = torch.ones_like(room, dtype=torch.bool)
        mask[1:T + 1, 16:16 + 4 * D] = False
        assert (room[mask] == 7.0).all()
        assert not (room[~mask] == 7.0).all()


@pytest.mark.parametrize("axis,value", [(0, -1), (2, 500), (1, 1 << 40), (0, -(1 << 62))])
def test_a_position_outside_the_table_leaves_its_token(axis, value):
    sizes = (3, 1, 128, 128, 1e-6)
    st = inputs(19, 3, 1, 128, 128)
    st["positions"][axis, 5] = value
    good = [t for t in range(19) if t != 5]
    st2 = {k: (v[good] if k in ("qkv", "dout") else v[:, good] if k == "positions" else v) for k, v in st.items()}
    want, slack = want_forward(st2, sizes, RN_ROPE_NEOX)
    grads, slacks = want_backward(st2, sizes, RN_ROPE_NEOX)
    before, dbefore = st["qkv"].clone(), st["dout"].clone()
    _, dwq, dwk = backward(st, sizes)
    assert binding.device_status() == RN_STATUS_BAD_POSITION
    assert torch.equal(st["dout"][5], dbefore[5])
    assert_near(st["dout"][good, :512].reshape(want.shape), grads[0], slacks[0], "dx")
    assert_near(dwq, grads[1], slacks[1], "dwq")
    assert_near(dwk, grads[2], slacks[2], "dwk")
    forward(st, sizes)
    assert binding.device_status() == RN_STATUS_BAD_POSITION
    assert torch.equal(st["qkv"][5], before[5])
    assert_near(st["qkv"][good, :512].reshape(want.shape), want, slack, "results")
    assert binding.device_status() == 0


def test_positions_of_axes_that_turn_nothing_are_not_looked_at():
    st = inputs(9, 3, 1, 64, 64, "one")
    st["positions"] = torch.cat((st["positions"], torch.full((1, 9), -5, device="cuda"), st["positions"]))
    st["axes"] = RopeAxes([0, 2] * 16)
    check_both(st, (3, 1, 64, 64, 1e-6), RN_ROPE_NEOX, "unused axis")


def test_one_row_of_positions_for_all_axes():
    st = inputs(50, 4, 2, 64, 64)
    st["positions"] = st["positions"][:1].expand(3, 50)
    check_both(st, (4, 2, 64, 64, 1e-6), RN_ROPE_NEOX, "expanded")


def test_rows_beyond_31_and_32_bits():
    """Row offsets past 2^32 bytes and 2^32 elements."""
    if torch.cuda.get_device_properties(0).total_memory < 60e9:
        pytest.skip("needs 60 GB")
    D, sizes, T = 64, (3, 1, 64, 64, 1e-6), 3
    small = inputs(T, 3, 1, D, 64)
    stride = (1 << 32) - (1 << 30) + 8
    for name in ("qkv", "dout"):
        far = torch.empty(2 * stride + 512, dtype=BF, device="cuda").as_strided((T, 320), (stride, 1))
        small[name] = far.copy_(small[name])
    check_both(small, sizes, RN_ROPE_NEOX, "far rows")


def test_weight_gradients_are_added_or_overwritten():
    sizes = (8, 2, 128, 128, 1e-6)
    st = inputs(200, 8, 2, 128, 128)
    dx = torch.empty(200, 1280, dtype=BF, device="cuda")
    _, q, k = backward(st, sizes, dx=dx)
    dwq, dwk = torch.full((128,), 3.0, device="cuda"), torch.full((128,), float("nan"), device="cuda")
    backward(st, sizes, dx=dx, dwq=dwq, dwk=dwk)
    assert torch.equal(dwq, q) and torch.equal(dwk, k)
    dwq.fill_(3.0)
    backward(st, sizes, dx=dx, dwq=dwq, dwk=dwk, accumulate=True)
    assert torch.equal(dwq, 3.0 + q) and torch.equal(dwk, k + k)
    with pytest.raises(ValueError, match="accumulate"):
        backward(st, sizes, dx=dx, dwq=dwq, accumulate=True)


@pytest.mark.parametrize("T,Hq,Hkv", [(0, 4, 2), (5, 0, 0)])
def test_no_token_gives_no_gradient(T, Hq, Hkv):
    st = inputs(T, Hq, Hkv, 64, 64)
    dwq = torch.full((64,), 9.0, device="cuda")
    dwk = torch.full((64,), 9.0, device="cuda")
    backward(st, (Hq, Hkv, 64, 64, 1e-6), dwq=dwq, dwk=dwk, accumulate=True)
    assert (dwq == 9).all() and (dwk == 9).all()
    backward(st, (Hq, Hkv, 64, 64, 1e-6), dwq=dwq, dwk=dwk)
    assert (dwq == 0).all() and (dwk == 0).all()
    forward(st, (Hq, Hkv, 64, 64, 1e-6))


def test_heads_of_zeros_and_heads_whose_squares_leave_fp32():
    """A head of zeros stays zero; one with a zero scale gives zeros, and no gradient."""
    sizes = (3, 1, 64, 64, 1e-6)
    st = inputs(6, 3, 1, 64, 64)
    st["qkv"][1, :64] = 0
    st["qkv"][2, 64:128] = 3e38
    dout = st["dout"].clone()
    out = torch.empty(6, 256, dtype=BF, device="cuda")
    forward(st, sizes, out=out)
    assert (out[1, :64] == 0).all() and (out[2, 64:128] == 0).all()
    dx, dwq, dwk = backward(st, sizes, dx=torch.empty_like(out))
    assert (dx[2, 64:128] == 0).all() and dwq.isfinite().all() and dwk.isfinite().all()
    # no norm to speak of: dx is the turned gradient times weight and eps ** -0.5
    (want, _, _), (slack, _, _) = want_backward(dict(st, qkv=st["qkv"].clone().fill_(0)), sizes, RN_ROPE_NEOX)
    assert_near(dx[1, :64], want[1, 0], slack[1, 0], "zeros")
    assert torch.equal(dout, st["dout"])


def test_a_nan_reaches_its_head_and_the_sums_alone():
    sizes = (3, 1, 128, 64, 1e-6)
    st = inputs(6, 3, 1, 128, 64)
    st["qkv"][4, 128 + 100] = float("nan")
    out = torch.empty(6, 512, dtype=BF, device="cuda")
    forward(st, sizes, out=out)
    bad = out.isnan().view(6, 4, 128)
    assert bad[4, 1].all() and int(bad.sum()) == 128
    dx, dwq, dwk = backward(st, sizes, dx=out)
    bad = dx.isnan().view(6, 4, 128)
    assert bad[4, 1].all() and int(bad.sum()) == 128 and dwq.isnan().all() and dwk.isfinite().all()


def test_the_gradient_in_place_of_qkv():
    st = inputs(333, 8, 2, 128, 128, pad=8)
    sizes = (8, 2, 128, 128, 1e-6)
    want, dwq, dwk = backward(st, sizes, dx=torch.empty(333, 1280, dtype=BF, device="cuda"))
    values = st["qkv"][:, 1280:].clone()
    got = backward(st, sizes, dx=st["qkv"])
    assert got[0] is st["qkv"] and torch.equal(st["qkv"][:, :1280], want) and torch.equal(st["qkv"][:, 1280:], values)
    assert torch.equal(got[1], dwq) and torch.equal(got[2], dwk)


@pytest.mark.parametrize("kind", ["eights", "interleaved"])
@pytest.mark.parametrize("T,Hq,Hkv,D", [(9000, 16, 2, 128), (20000, 8, 1, 64), (5000, 10, 5, 256)])
def test_units_that_follow_one_another(T, Hq, Hkv, D, kind):
    """More units than warps: a warp's stream of heads goes from one into the next."""
    st = inputs(T, Hq, Hkv, D, D // 2, kind)
    st["positions"][1, T // 2] = -1
    sizes = (Hq, Hkv, D, D // 2, 1e-6)
    good = torch.arange(T, device="cuda") != T // 2
    st2 = {k: (v[good] if k in ("qkv", "dout") else v[:, good] if k == "positions" else v) for k, v in st.items()}
    n = (Hq + Hkv) * D
    want, slack = want_forward(st2, sizes, RN_ROPE_NEOX)
    out = torch.full((T, n), 5.0, dtype=BF, device="cuda")
    forward(st, sizes, out=out)
    assert (out[T // 2] == 5).all()
    assert_near(out[good].view(want.shape), want, slack, "results")
    del want, slack
    grads, slacks = want_backward(st2, sizes, RN_ROPE_NEOX)
    out.fill_(5.0)
    _, dwq, dwk = backward(st, sizes, dx=out)
    assert (out[T // 2] == 5).all()
    assert_near(out[good].view(grads[0].shape), grads[0], slacks[0], "dx")
    assert_near(dwq, grads[1], slacks[1], "dwq")
    assert_near(dwk, grads[2], slacks[2], "dwk")
    assert binding.device_status() == RN_STATUS_BAD_POSITION


def test_two_calls_at_once():
    """Calls on two streams, each with its own workspace."""
    sizes = (8, 2, 128, 128, 1e-6)
    sts = [inputs(3000, 8, 2, 128, 128, seed=s) for s in (1, 2)]
    outs = [torch.empty(3000, 1280, dtype=BF, device="cuda") for _ in sts]
    want = [[x.clone() for x in backward(st, sizes, dx=o)] for st, o in zip(sts, outs)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    spaces = [binding.qk_norm_rope_axes_workspace(128) for _ in sts]
    torch.cuda.synchronize()
    for _ in range(4):
        got = [backward(st, sizes, dx=o, workspace=w, stream=s)
               for st, o, w, s in zip(sts, outs, spaces, streams)]
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            for p, q in zip(w, g):
                assert torch.equal(p, q)


@pytest.mark.parametrize("which", ["forward", "backward"])
def test_captured_and_replayed(which):
    """Graphs of a call and its plain run give the same bits, on new inputs as well."""
    sizes = (8, 2, 128, 128, 1e-6)
    st = inputs(300, 8, 2, 128, 128)
    n = 1280
    out = torch.empty(300, n, dtype=BF, device="cuda")
    ws = binding.qk_norm_rope_axes_workspace(128)
    dw = [torch.empty(128, device="cuda") for _ in range(2)]

    def call():
        if which == "forward":
            return [forward(st, sizes, out=out)]
        return list(backward(st, sizes, dx=out, dwq=dw[0], dwk=dw[1], workspace=ws))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    other = inputs(300, 8, 2, 128, 128, seed=5)
    for name in ("qkv", "dout", "positions"):
        st[name].copy_(other[name])
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    kept = [x.clone() for x in got]
    ws.fill_(255)
    for a, b in zip(kept, call()):
        assert torch.equal(a, b)


def test_on_another_stream_with_results_made_for_it():
    sizes = (8, 2, 128, 128, 1e-6)
    st = inputs(2000, 8, 2, 128, 128)
    want = [x.clone() for x in backward(st, sizes, dx=torch.empty(2000, 1280, dtype=BF, device="cuda"))]
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        dx = torch.empty(2000, 1280, dtype=BF, device="cuda")
        torch.cuda.synchronize()
        got = backward(st, sizes, dx=dx, stream=stream)
        side.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)


def test_refusals_of_the_binding():
    sizes = (3, 1, 64, 64, 1e-6)
    st = inputs(4, 3, 1, 64, 64)
    with pytest.raises(ValueError, match="each of the 32 pairs"):
        forward(dict(st, axes=[0] * 31), sizes)
    with pytest.raises(ValueError, match="positions"):
        forward(dict(st, positions=st["positions"][:2]), sizes)
    with pytest.raises(ValueError, match="positions"):
        forward(dict(st, positions=st["positions"].int()), sizes)
    with pytest.raises(TypeError, match="qkv"):
        forward(dict(st, qkv=st["qkv"].float()), sizes)
    with pytest.raises(TypeError, match="wq"):
        forward(dict(st, wq=st["wq"].half()), sizes)
    with pytest.raises(ValueError, match="cos_sin"):
        forward(st, (3, 1, 64, 32, 1e-6))
    with pytest.raises(ValueError, match="out"):
        forward(st, sizes, out=torch.empty(4, 255, dtype=BF, device="cuda"))
    with pytest.raises(ValueError, match="dout"):
        backward(dict(st, dout=st["dout"][:, :1].expand(4, 320)), sizes)
    with pytest.raises(RowNormError, match="sizes"):
        forward(dict(st, qkv=torch.zeros(4, 321, dtype=BF, device="cuda")[:, :320]), sizes)
    with pytest.raises(RowNormError, match="aligned"):
        forward(dict(st, qkv=torch.zeros(4, 328, dtype=BF, device="cuda")[:, 4:324]), sizes)
    with pytest.raises(RowNormError, match="argument"):
        backward(st, sizes, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(RowNormError, match="argument"):
        dw = torch.empty(64, device="cuda")
        backward(st, sizes, dwq=dw, dwk=dw)


def test_the_gradient_is_the_kernel_forward_s_differences():
    """fp16 results against a weight of one: differences of the forward kernel along a
    direction, by steps that its rounding leaves visible."""
    T, Hq, Hkv, D = 64, 4, 2, 64
    sizes = (Hq, Hkv, D, D, 1e-6)
    st = inputs(T, Hq, Hkv, D, D, dtype=HALF, seed=3)
    n = (Hq + Hkv) * D
    d = torch.randn(T, n, device="cuda")
    dx, _, _ = backward(st, sizes, dx=torch.empty(T, n, dtype=HALF, device="cuda"))
    x = st["qkv"][:, :n].float()
    h = 2.0 ** -4
    out = []
    moved = []
    for sign in (1, -1):
        y = (x + sign * h * d).half()
        moved.append(y.double())
        s2 = dict(st, qkv=torch.cat((y, st["qkv"][:, n:]), 1))
        out.append(forward(s2, sizes, out=torch.empty_like(y)).double())
    do = st["dout"][:, :n].double()
    found = ((out[0] - out[1]) * do).sum()
    want = (dx.double() * (moved[0] - moved[1])).sum()
    # roundings of the results (2^-11 of values up to about 4, independent) and of dx, and
    # third differences h^2 / 6 of sums over T n values: all well below 3% of their norm
    norm = (dx.double().square().sum() * (moved[0] - moved[1]).square().sum()).sqrt()
    assert abs(found - want) <= 0.03 * norm
