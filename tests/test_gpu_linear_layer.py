"""The linear attention and the block norms together, as a layer uses them (GPU): a training step
against float64 differentiation, serving (packed prompts, then single tokens) against the whole
sequences, a captured layer, and calls on two streams at once.

Layer (fp32, rows of H dv channels):
    o = linear attention(q, k, v, g, h0);   a = norm_head(o) w sigmoid(z);   y = a Wo
    h = x + s r norm_row(y) w2;             n = norm_row(h) w3

Tolerance of the training step: every operator is within (D + T + 64) 2^-23 < 1e-4 of the sum of the
absolute values of a result's terms (see the operators' own tests), D = 128 and T = 200 here; five of
them follow each other, each at most doubling the share of its input's error (two factors of a product,
a norm and its mean), and sums over absolute values are a few times the values: 1e-3 in the 2-norm
bounds it with room, and an error in any formula is of order one.
"""
import pytest
import torch

import gated_delta_rule_82_b200 as ck
import linattn_ref as ref

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from gated_delta_rule_82_b200 import build
    build.build()


def _layer_inputs(B=2, T=200, H=4, Hk=2, d=32, seed=0):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s, std=1.0: (torch.randn(*s, generator=gen) * std).cuda()
    D = H * d
    p = ref.make((B, T), H, Hk, d, d, torch.float32, states=B, seed=seed + 1, device="cuda")
    p.update(z=rn(B, T, D), x=rn(B, T, D), w1=1 + rn(d, std=0.1), Wo=rn(D, D, std=D ** -0.5),
             w2=1 + rn(D, std=0.1), r=1 + rn(D, std=0.1), w3=1 + rn(D, std=0.1))
    return p, rn(B, T, D), rn(B, T, D), rn(B, H, d, d, std=0.1)


HEAD = dict(gate_act="sigmoid", eps=EPS)
BLOCK = dict(res_scale=0.5, pre_norm=True, eps=EPS)


def _forward(p):
    B, T, D = p["x"].shape
    o, hT = ck.linattn_fwd_chunked(p["q"], p["k"], p["v"], p["g"], p["h0"])
    a, _ = ck.block_norm(o.view(B, T, D), gate=p["z"], post_group=o.shape[-1], post_weight=p["w1"], **HEAD)
    y = a @ p["Wo"]
    h, n = ck.block_norm(y, residual=p["x"], post_group=D, post_weight=p["w2"], res_vector=p["r"],
                         pre_weight=p["w3"], **BLOCK)
    return o, a, y, h, n, hT


def _training_step(p, dh, dn, dhT):
    B, T, D = p["x"].shape
    o, a, y, h, n, hT = _forward(p)
    g2 = ck.block_norm_bwd(y, dh, dn, residual=p["x"], post_group=D, post_weight=p["w2"], res_vector=p["r"],
                           pre_weight=p["w3"], **BLOCK)
    da, dWo = g2["dy"] @ p["Wo"].T, a.reshape(-1, D).T @ g2["dy"].reshape(-1, D)
    g1 = ck.block_norm_bwd(o.view(B, T, D), da, gate=p["z"], post_group=o.shape[-1], post_weight=p["w1"],
                           **HEAD)
    g0 = ck.linattn_bwd_chunked(p["q"], p["k"], p["v"], p["g"], p["h0"], g1["dy"].view_as(o), dhT)
    grads = dict(q=g0["dq"], k=g0["dk"], v=g0["dv"], g=g0["dlog_decay"], h0=g0["dh0"], z=g1["dgate"],
                 w1=g1["dpost_weight"], Wo=dWo, w2=g2["dpost_weight"], r=g2["dres_vector"],
                 w3=g2["dpre_weight"], x=g2["dresidual"])
    return (h, n, hT), grads


def _float64(p, dh, dn, dhT):
    """The same from plain formulas, differentiated by torch."""
    P = {n: t.double().requires_grad_() for n, t in p.items()}
    B, T, D = p["x"].shape
    H, d = p["v"].shape[2:]
    rep = H // p["q"].shape[2]
    q, k = P["q"].repeat_interleave(rep, 2), P["k"].repeat_interleave(rep, 2)
    S, outs = P["h0"], []
    for t in range(T):
        S = torch.exp(P["g"][:, t])[..., None, None] * S + k[:, t, :, :, None] * P["v"][:, t, :, None, :]
        outs.append((q[:, t, :, :, None] * S).sum(2) * d ** -0.5)
    rms = lambda x: x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt()
    a = (rms(torch.stack(outs, 1)) * P["w1"]).reshape(B, T, D) * torch.sigmoid(P["z"])
    h = P["x"] + 0.5 * P["r"] * rms(a @ P["Wo"]) * P["w2"]
    n = rms(h) * P["w3"]
    loss = (h * dh.double()).sum() + (n * dn.double()).sum() + (S * dhT.double()).sum()
    return (h, n, S), dict(zip(P, torch.autograd.grad(loss, list(P.values()))))


def _rel(got, want):
    return float((got.double() - want).norm() / want.norm())


def test_training_step():
    p, dh, dn, dhT = _layer_inputs()
    tf32 = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    try:
        outs, grads = _training_step(p, dh, dn, dhT)
    finally:
        torch.backends.cuda.matmul.allow_tf32 = tf32
    wout, want = _float64(p, dh, dn, dhT)
    for got, w in zip(outs, wout):
        assert _rel(got, w.detach()) <= 1e-3
    for name in grads:
        assert _rel(grads[name], want[name]) <= 1e-3, name


def test_captured_training_step():
    """Captured and replayed on new values: the bits of the eager step."""
    p, dh, dn, dhT = _layer_inputs(seed=3)
    args = {n: t.clone() for n, t in p.items()}
    _training_step(args, dh, dn, dhT)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs, grads = _training_step(args, dh, dn, dhT)
    for seed in (3, 4):
        q = _layer_inputs(seed=seed)[0]
        for n, t in args.items():
            t.copy_(q[n])
        graph.replay()
        torch.cuda.synchronize()
        want, wgrads = _training_step(q, dh, dn, dhT)
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        assert all(torch.equal(grads[n], wgrads[n]) for n in grads)


def test_serving():
    """Packed prompts through prologue, attention and head norm, then single tokens on the states:
    the outputs of the whole sequences (bf16: two roundings of each, of the attention's output and of
    the norm's, as each operator's tests bound them; the norm divides by a root mean square that the
    attention's rounding moves by no more than 2^-8 of it)."""
    lens, steps, H, d = [70, 1, 200], 3, 4, 128
    n = len(lens)
    cu = torch.tensor([0, *torch.tensor(lens).cumsum(0)], dtype=torch.int32)
    full = ref.make((n, max(lens) + steps), H, H, d, d, torch.bfloat16, states=n, seed=2, device="cuda")
    z = torch.randn(n, max(lens) + steps, H * d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    w = torch.ones(d, device="cuda")
    q, k = ck.qk_prologue(full["q"], full["k"], rope_theta=1e4)
    norm = lambda o, gate: ck.block_norm(o.reshape(-1, H * d), gate=gate.reshape(-1, H * d), gate_act="silu",
                                         post_group=d, post_weight=w)[0]
    pack = lambda t: torch.cat([t[s, :lens[s]] for s in range(n)])
    o, state = ck.linattn_fwd_chunked(pack(q), pack(k), pack(full["v"]), pack(full["g"]), full["h0"],
                                      cu_seqlens=cu.cuda(), cu_seqlens_cpu=cu)
    prompt = norm(o, pack(z))
    later = []
    for t in range(steps):
        at = lambda x: torch.stack([x[s, lens[s] + t] for s in range(n)])
        later.append(norm(ck.linattn_decode_step(at(q), at(k), at(full["v"]), at(full["g"]), state), at(z)))
    for s in range(n):
        L = lens[s] + steps
        one = [x[s:s + 1, :L].contiguous() for x in (q, k, full["v"], full["g"])]
        (ref_o, _), (big, _) = ref.forward(*one, full["h0"][s:s + 1])
        ref_o, big = ref_o[0].cuda(), big[0].cuda()
        root = (ref_o.pow(2).mean(-1, keepdim=True) + 1e-5).sqrt()
        zz = z[s, :L].double().view(L, H, d)
        act = zz * torch.sigmoid(zz)
        want = ref_o / root * act
        # the attention's own bound, through the norm's root (its share and its root's), then rounding
        err = (2 ** -8 * (ref_o.abs() + big) + 1e-4 * big) / root
        bound = (err + want.abs() / act.abs().clamp_min(1e-30) * err.pow(2).mean(-1, keepdim=True).sqrt()) * act.abs()
        bound = bound + 2 ** -8 * want.abs() + 1e-6
        got = torch.cat([prompt[int(cu[s]):int(cu[s + 1])]] + [x[s:s + 1] for x in later]).double().view(L, H, d)
        assert float(((got - want).abs() / bound).max()) <= 1


def test_two_streams_at_once():
    """Calls that overlap on the device, each with a workspace of its own."""
    cases = []
    for seed, T in ((1, 3000), (2, 700)):
        p = ref.make((1, T), 8, 8, 128, 128, torch.bfloat16, states=1, seed=seed, grads=True, device="cuda")
        args = (p["q"], p["k"], p["v"], p["g"], p["h0"])
        cases.append((args, p, ck.linattn_fwd_chunked(*args), ck.linattn_bwd_chunked(*args, p["do"], p["dhT"])))
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for (args, p, _, _), s in zip(cases, streams):
            with torch.cuda.stream(s):
                got.append((ck.linattn_fwd_chunked(*args), ck.linattn_bwd_chunked(*args, p["do"], p["dhT"])))
        torch.cuda.synchronize()
        for (_, _, want, grads), (out, back) in zip(cases, got):
            assert all(torch.equal(a, b) for a, b in zip(out, want))
            assert all(torch.equal(back[n], grads[n]) for n in grads)
    assert ck.last_device_status() == 0


def test_state_in_place_across_units():
    """hT written over h0 where several units of a sequence read h0's share."""
    for T, H in ((520, 40), (3000, 4)):
        p = ref.make((2, T), H, H, 128, 128, torch.bfloat16, states=2, seed=T, device="cuda")
        want = ck.linattn_fwd_chunked(p["q"], p["k"], p["v"], p["g"], p["h0"])
        h = p["h0"].clone()
        out, hT = ck.linattn_fwd_chunked(p["q"], p["k"], p["v"], p["g"], h, hT=h)
        assert hT is h
        # (the states entering the units are added up in another order: fp32 rounding of the states,
        # which can move a bf16 operand or output by a step)
        assert _rel(h, want[1].double()) <= 1e-6
        assert _rel(out, want[0].double()) <= 2 ** -8


def test_prompt_after_other_shapes_and_last_rows():
    """A tail that ends inside a tile leaves the rows behind the last sequence as they were."""
    lens = [100, 29]
    cu = torch.tensor([0, 100, 129], dtype=torch.int32)
    p = ref.make((129,), 2, 2, 128, 128, torch.bfloat16, states=2, seed=4, device="cuda")
    buf = torch.full((200, 2, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:129]
    ck.linattn_fwd_chunked(p["q"], p["k"], p["v"], p["g"], p["h0"], cu_seqlens=cu.cuda(), cu_seqlens_cpu=cu, out=out)
    assert bool((buf[129:] == 5).all())
    (o, _), (big, _) = ref.forward(p["q"], p["k"], p["v"], p["g"], p["h0"], [0, 100, 129])
    assert ref.off(out, o, 2 ** -8 * (o.abs() + big) + 500 * ref.F32 * big) <= 1
    # NaN in a neighbouring sequence stays there
    v = p["v"].clone()
    v[100:] = float("nan")
    out2, _ = ck.linattn_fwd_chunked(p["q"], p["k"], v, p["g"], p["h0"], cu_seqlens=cu.cuda(), cu_seqlens_cpu=cu)
    assert torch.equal(out2[:100], out[:100])


@pytest.mark.parametrize("per_token", [True, False])
def test_all_sequences_empty(per_token):
    """A batch without tokens: empty outputs, states and their gradients passed through."""
    cu = torch.zeros(4, dtype=torch.int32)
    q, v = torch.empty(0, 2, 64, device="cuda"), torch.empty(0, 4, 32, device="cuda")
    g = torch.empty(0, 4, device="cuda") if per_token else torch.full((4,), -0.1, device="cuda")
    h0, dhT = torch.randn(3, 4, 64, 32, device="cuda"), torch.randn(3, 4, 64, 32, device="cuda")
    kw = dict(cu_seqlens=cu.cuda(), cu_seqlens_cpu=cu)
    out, hT = ck.linattn_fwd_chunked(q, q, v, g, h0, **kw)
    assert out.shape == v.shape and torch.equal(hT, h0)
    assert bool((ck.linattn_fwd_chunked(q, q, v, g, **kw)[1] == 0).all())
    grads = ck.linattn_bwd_chunked(q, q, v, g, h0, v, dhT, **kw)
    assert grads["dq"].shape == q.shape and torch.equal(grads["dh0"], dhT)
    assert grads["dlog_decay"].shape == g.shape and bool((grads["dlog_decay"] == 0).all())


def test_binding_refusals():
    """Arguments that only a device can hold wrong."""
    q, g = torch.zeros(1, 8, 2, 16, device="cuda"), torch.zeros(1, 8, 2, device="cuda")
    cu = torch.tensor([0, 8], dtype=torch.int32)
    for bad in (lambda: ck.linattn_fwd_chunked(q, q.transpose(1, 2).contiguous().transpose(1, 2), q, g),
                lambda: ck.linattn_fwd_chunked(q, q.bfloat16(), q, g),
                lambda: ck.linattn_fwd_chunked(q, q[:, :7].contiguous(), q, g),
                lambda: ck.linattn_fwd_chunked(q, q, q, g.double()),
                lambda: ck.linattn_fwd_chunked(q, q, q, g, cu_seqlens=cu.cuda(), cu_seqlens_cpu=cu.cuda()),
                lambda: ck.linattn_fwd_chunked(q, q, q, g, cu_seqlens=cu.cuda() - 1),
                lambda: ck.linattn_fwd_chunked(q, q, q, g, out=q),
                lambda: ck.linattn_bwd_chunked(q, q, q, g, None, q.cpu()),
                lambda: ck.linattn_decode_step(q[0], q[0], q[0], g[0], torch.zeros(8, 2, 16, 32, device="cuda")),
                lambda: ck.block_norm(q, gate=q, gate_act="relu"),
                lambda: ck.block_norm(q, gate=q),
                lambda: ck.block_norm(q, post_group=48),
                lambda: ck.block_norm(q, pre_weight=q[0, 0, 0])):
        with pytest.raises((ValueError, TypeError, ck.CkdaError)):
            bad()
    torch.cuda.synchronize()
