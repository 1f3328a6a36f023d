"""Decayed linear attention on the GPU (chunked forward, backward, single-token step) against the
float64 recurrence, element by element.

Tolerances (linattn_ref): with `big` the majorant of a value (its sum over absolute values),
  fp32 results and states   n 2^-23 big, n = T + dk + dv + 64: the tokens a state is carried
                            through, the channels and chunk tokens summed for one output, and the
                            decay factors; fp32 operands enter with terms down to 2^-24
  bf16 results              2^-8 (|value| + big) on top: the output's rounding, and that of the
                            scores and the state where they enter a product
"""
import pytest
import torch

import gated_delta_rule_82_b200 as ck
import linattn_ref as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from gated_delta_rule_82_b200 import build
    build.build()


def _offsets(lens):
    return torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32)


def _bound(want, big, n, rounded):
    b = n * ref.F32 * big + 1e-30
    return b + ref.BF16 * (want.abs() + big) if rounded else b


def _terms(d, T):
    return T + d["q"].shape[-1] + d["v"].shape[-1] + 64


def _check_forward(d, out, hT, cu=None, T=None, scale=None):
    (o, s), (ob, sb) = ref.forward(d["q"], d["k"], d["v"], d["g"], d["h0"], cu, scale)
    n = _terms(d, T or d["q"].shape[-3])
    assert ref.off(out, o, _bound(o, ob, n, out.dtype == torch.bfloat16)) <= 1
    assert ref.off(hT, s, _bound(s, sb, n, False)) <= 1


# head sizes, types, lengths around a chunk and across units, grouped heads, both kinds of decay
@pytest.mark.parametrize("B,T,H,Hk,dk,dv,dtype,per_token,h0", [
    (1, 1, 1, 1, 16, 16, "f32", True, True),
    (2, 1, 3, 3, 128, 128, "bf16", True, False),
    (1, 63, 2, 2, 128, 128, "bf16", True, True),
    (1, 64, 2, 1, 128, 128, "bf16", False, True),
    (2, 65, 4, 2, 64, 128, "bf16", True, False),
    (1, 127, 2, 2, 128, 128, "bf16", False, False),
    (1, 128, 2, 2, 128, 128, "bf16", True, True),
    (1, 129, 2, 2, 128, 128, "bf16", True, False),
    (1, 700, 4, 4, 128, 128, "bf16", True, True),
    (2, 513, 3, 1, 128, 64, "bf16", False, True),
    (1, 300, 2, 2, 32, 16, "bf16", True, True),
    (1, 300, 2, 2, 16, 32, "f32", False, True),
    (2, 257, 6, 3, 64, 64, "f32", True, True),
    (1, 450, 2, 2, 128, 128, "f32", True, True),
    (1, 190, 3, 3, 128, 32, "f32", True, False),
    (3, 100, 160, 160, 16, 64, "bf16", True, False),     # more heads than units side by side
])
def test_forward(B, T, H, Hk, dk, dv, dtype, per_token, h0):
    d = ref.make((B, T), H, Hk, dk, dv, DT[dtype], per_token=per_token, states=B if h0 else 0,
                 seed=T + H, device="cuda")
    out, hT = ck.linattn_fwd_chunked(d["q"], d["k"], d["v"], d["g"], d["h0"])
    _check_forward(d, out, hT)


@pytest.mark.parametrize("lens,H,Hk,dk,dv,dtype", [
    ([1, 0, 64, 65, 200], 2, 2, 128, 128, "bf16"),
    ([0, 0, 5], 3, 1, 16, 64, "f32"),
    ([700, 3, 0, 130, 1], 4, 2, 64, 128, "f32"),
    ([300, 41, 0, 600], 16, 16, 128, 128, "bf16"),
    ([2] * 70 + [0] * 3 + [33], 2, 1, 32, 32, "bf16"),   # more sequences than a warp counts at once
])
def test_packed(lens, H, Hk, dk, dv, dtype):
    cu = _offsets(lens)
    d = ref.make((sum(lens),), H, Hk, dk, dv, DT[dtype], states=len(lens), seed=len(lens),
                 device="cuda")
    out, hT = ck.linattn_fwd_chunked(d["q"], d["k"], d["v"], d["g"], d["h0"], cu_seqlens=cu.cuda(),
                                     cu_seqlens_cpu=cu)
    _check_forward(d, out, hT, cu, max(lens))
    for s, n in enumerate(lens):
        if n == 0:
            assert torch.equal(hT[s], d["h0"][s])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128])
def test_resets_and_strong_decays(dtype, dim):
    """g = -inf forgets the state exactly; decays that underflow, and none at all (g = 0)."""
    d = ref.make((1, 400), 4, 4, dim, dim, DT[dtype], states=1, seed=5, device="cuda")
    g = d["g"]
    g[0, [0, 5, 63, 64, 200, 201, 330], 0] = -float("inf")
    g[0, :, 1] = -120.0
    g[0, :, 2] = 0.0
    g[0, ::7, 3] = -90.0
    out, hT = ck.linattn_fwd_chunked(d["q"], d["k"], d["v"], g, d["h0"])
    _check_forward(d, out, hT)
    # what lies before a reset has no influence at all
    v2 = d["v"].clone()
    v2[0, :64, 0] += 3.0
    out2, hT2 = ck.linattn_fwd_chunked(d["q"], d["k"], v2, g, d["h0"])
    assert torch.equal(out2[0, 64:, 0], out[0, 64:, 0]) and torch.equal(hT2[0, 0], hT[0, 0])


def test_causality_and_splitting():
    """Later tokens do not touch earlier outputs; a call continued from hT gives the whole call."""
    d = ref.make((1, 900), 2, 2, 128, 128, torch.float32, seed=9, device="cuda")
    out, hT = ck.linattn_fwd_chunked(d["q"], d["k"], d["v"], d["g"])
    part = lambda a, b: [x[:, a:b].contiguous() for x in (d["q"], d["k"], d["v"], d["g"])]
    o1, h1 = ck.linattn_fwd_chunked(*part(0, 333))
    o2, h2 = ck.linattn_fwd_chunked(*part(333, 900), h1)
    _check_forward(d, torch.cat([o1, o2], 1), h2)
    _check_forward(d, out, hT)
    changed = {n: d[n].clone() for n in "qkvg"}
    for n in "qkv":
        changed[n][:, 640:] *= 2
    o3, _ = ck.linattn_fwd_chunked(*(changed[n] for n in "qkvg"))
    assert torch.equal(o3[:, :640], out[:, :640])


def test_scale_state_in_place_and_no_state():
    d = ref.make((2, 150), 2, 2, 32, 64, torch.float32, states=2, seed=3, device="cuda")
    want = ck.linattn_fwd_chunked(d["q"], d["k"], d["v"], d["g"], d["h0"], scale=0.7)
    _check_forward(d, *want, scale=0.7)
    out, none = ck.linattn_fwd_chunked(d["q"], d["k"], d["v"], d["g"], d["h0"], scale=0.7,
                                       want_state=False)
    assert none is None and torch.equal(out, want[0])
    h = d["h0"].clone()
    out, hT = ck.linattn_fwd_chunked(d["q"], d["k"], d["v"], d["g"], h, scale=0.7, hT=h)
    assert hT is h and torch.equal(h, want[1]) and torch.equal(out, want[0])


# ------------------------------------------------------------------------------------- backward

@pytest.mark.parametrize("B,T,H,Hk,dk,dv,dtype,per_token,h0", [
    (1, 1, 2, 1, 16, 16, "f32", True, True),
    (1, 64, 2, 2, 128, 128, "bf16", True, True),
    (2, 65, 4, 2, 64, 128, "bf16", True, False),
    (1, 129, 2, 2, 128, 128, "bf16", False, True),
    (1, 600, 4, 4, 128, 128, "bf16", True, True),
    (1, 600, 2, 2, 128, 128, "bf16", True, False),
    (2, 333, 6, 3, 64, 64, "f32", False, True),
    (1, 450, 2, 2, 128, 128, "f32", True, True),
    (2, 200, 3, 1, 16, 64, "f32", True, False),
    (1, 300, 40, 40, 32, 16, "bf16", False, True),
    (3, 100, 160, 80, 16, 32, "bf16", True, False),
])
def test_backward(B, T, H, Hk, dk, dv, dtype, per_token, h0):
    d = ref.make((B, T), H, Hk, dk, dv, DT[dtype], per_token=per_token, states=B if h0 else 0,
                 seed=T + H, grads=True, device="cuda")
    got = ck.linattn_bwd_chunked(d["q"], d["k"], d["v"], d["g"], d["h0"], d["do"], d["dhT"])
    _check_backward(d, got, T)


def _check_backward(d, got, T, cu=None):
    want, big = ref.backward(d["q"], d["k"], d["v"], d["g"], d["h0"], d["do"], d["dhT"], cu)
    n = _terms(d, T)
    for name, x in got.items():
        if x is None:
            continue
        # (a fixed decay's gradient sums over all tokens, in fp64)
        assert ref.off(x, want[name], _bound(want[name], big[name], n, x.dtype == torch.bfloat16)) \
            <= 1, name


@pytest.mark.parametrize("per_token", [True, False])
@pytest.mark.parametrize("lens,H,Hk,dk,dv,dtype", [
    ([1, 0, 64, 65, 200], 2, 2, 128, 128, "bf16"),
    ([700, 3, 0, 130, 1], 4, 2, 64, 128, "f32"),
    ([2] * 40 + [0, 33], 34, 17, 32, 16, "f32"),
])
def test_backward_packed(lens, H, Hk, dk, dv, dtype, per_token):
    cu = _offsets(lens)
    d = ref.make((sum(lens),), H, Hk, dk, dv, DT[dtype], states=len(lens), seed=len(lens),
                 per_token=per_token, grads=True, device="cuda")
    got = ck.linattn_bwd_chunked(d["q"], d["k"], d["v"], d["g"], d["h0"], d["do"], d["dhT"],
                                 cu_seqlens=cu.cuda(), cu_seqlens_cpu=cu)
    _check_backward(d, got, max(lens), cu)
    for s, m in enumerate(lens):
        if m == 0:
            assert torch.equal(got["dh0"][s], d["dhT"][s])


def test_backward_resets_and_unwanted_gradients():
    d = ref.make((1, 300), 2, 2, 64, 64, torch.float32, states=1, seed=4, grads=True, device="cuda")
    d["g"][0, [0, 70, 71, 255], 0] = -float("inf")
    got = ck.linattn_bwd_chunked(d["q"], d["k"], d["v"], d["g"], d["h0"], d["do"], d["dhT"])
    _check_backward(d, got, 300)
    assert bool((got["dlog_decay"][0, [0, 70, 71, 255], 0] == 0).all())
    assert bool((got["dh0"][0, 0] == 0).all())
    less = ck.linattn_bwd_chunked(d["q"], d["k"], d["v"], d["g"], d["h0"], d["do"], d["dhT"],
                                  want_dlog_decay=False, want_dh0=False)
    assert less["dlog_decay"] is None and less["dh0"] is None
    for n in ("dq", "dk", "dv"):
        assert torch.equal(less[n], got[n])


def test_backward_is_the_slope():
    """<gradient, direction> against a central difference of the float64 loss."""
    d = ref.make((1, 130), 2, 1, 32, 16, torch.float32, states=1, seed=6, grads=True, device="cuda")
    got = ck.linattn_bwd_chunked(d["q"], d["k"], d["v"], d["g"], d["h0"], d["do"], d["dhT"])
    gen = torch.Generator().manual_seed(1)
    step = 1e-5

    def loss(p):
        (o, s), _ = ref.forward(p["q"], p["k"], p["v"], p["g"], p["h0"])
        return float((o * d["do"].double().cpu()).sum() + (s * d["dhT"].double().cpu()).sum())

    base = {n: d[n].double().cpu() for n in ("q", "k", "v", "g", "h0")}
    for n, name in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dlog_decay"), ("h0", "dh0")):
        r = torch.randn(base[n].shape, generator=gen, dtype=torch.float64)
        up, down = ({**base, n: base[n] + s * step * r} for s in (1, -1))
        slope = (loss(up) - loss(down)) / (2 * step)
        mine = float((got[name].double().cpu() * r).sum())
        # the difference's own error: step^2 times third derivatives (order 1 here), and the
        # rounding of the loss, 2^-53 |loss| / step; the gradient's: n 2^-23 of its terms
        scale = float((got[name].double().cpu().abs() * r.abs()).sum())
        assert abs(mine - slope) <= 1e-6 * (1 + abs(slope)) + 1e-4 * scale, name


# ------------------------------------------------------------------------------------- one token

@pytest.mark.parametrize("N,H,Hk,dk,dv,dtype,per_token", [
    (1, 1, 1, 16, 16, "f32", True),
    (1, 16, 16, 128, 128, "bf16", True),
    (5, 6, 3, 64, 128, "bf16", False),
    (3, 4, 1, 128, 16, "f32", True),
    (7, 3, 3, 16, 128, "bf16", True),
    (33, 5, 5, 32, 64, "f32", False),
])
def test_step(N, H, Hk, dk, dv, dtype, per_token):
    d = ref.make((N, 1), H, Hk, dk, dv, DT[dtype], per_token=per_token, states=N, seed=N + H,
                 device="cuda")
    state = d["h0"].clone()
    one = lambda x: x[:, 0].contiguous()
    out = ck.linattn_decode_step(one(d["q"]), one(d["k"]), one(d["v"]),
                                 one(d["g"]) if per_token else d["g"], state)
    _check_forward(d, out[:, None], state)


def test_steps_continue_a_prompt():
    """Prompt, then single tokens: the same tokens in one call."""
    d = ref.make((2, 140), 4, 2, 128, 64, torch.bfloat16, states=2, seed=8, device="cuda")
    cut = lambda a, b: [x[:, a:b].contiguous() for x in (d["q"], d["k"], d["v"], d["g"])]
    o, h = ck.linattn_fwd_chunked(*cut(0, 130), d["h0"])
    outs = [o]
    for t in range(130, 140):
        outs.append(ck.linattn_decode_step(*(x[:, 0] for x in cut(t, t + 1)), h)[:, None])
    _check_forward(d, torch.cat(outs, 1), h)


def test_step_reset():
    d = ref.make((2, 1), 2, 2, 32, 32, torch.float32, states=2, seed=8, device="cuda")
    d["g"][0, 0, 1] = -float("inf")
    state = d["h0"].clone()
    ck.linattn_decode_step(*(d[n][:, 0].contiguous() for n in "qkvg"), state)
    assert torch.equal(state[0, 1], d["k"][0, 0, 1, :, None] * d["v"][0, 0, 1, None, :])


# ----------------------------------------------------------------------------------- how it runs

def test_graph_replay_and_side_stream():
    d = ref.make((1, 520), 4, 4, 128, 128, torch.bfloat16, states=1, seed=2, grads=True,
                 device="cuda")
    args = (d["q"], d["k"], d["v"], d["g"], d["h0"])
    want = ck.linattn_fwd_chunked(*args)
    grads = ck.linattn_bwd_chunked(*args, d["do"], d["dhT"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = ck.linattn_fwd_chunked(*args)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ck.linattn_fwd_chunked(*args)
        back = ck.linattn_bwd_chunked(*args, d["do"], d["dhT"])
    for _ in range(2):
        for x in (*got, *back.values()):
            x.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        for n, x in back.items():
            assert torch.equal(x, grads[n]), n


def test_runs_are_identical_and_outputs_stay_inside():
    """No atomics: the same bits every time; nothing behind the outputs is written."""
    d = ref.make((1, 333), 3, 3, 64, 64, torch.bfloat16, seed=12, device="cuda")
    buf = torch.full((333 * 3 * 64 + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:333 * 3 * 64].view(1, 333, 3, 64)
    a = ck.linattn_fwd_chunked(d["q"], d["k"], d["v"], d["g"], out=out)
    assert bool((buf[333 * 3 * 64:] == 7).all())
    first = out.clone()
    ck.linattn_fwd_chunked(d["q"], d["k"], d["v"], d["g"], out=out)
    assert torch.equal(first, out) and a[0] is out
