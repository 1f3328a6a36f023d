"""The block norms (norm after a block, gate, scale, residual, norm before the next) on the GPU,
forward and backward, against float64 formulas; gradients by differentiating those.

Tolerances.  Forward: an fp32 evaluation rounds every factor of a value, and a mean of squares of
K channels is off by at most K 2^-24 relative (half that enters through the root): with the
exponential, root and division at a few 2^-23 each, (D + 64) 2^-23 relative to the value's terms;
a bf16 result adds its rounding, 2^-8 |value|.  Backward: the same relative to the sum of absolute
values of a gradient's terms (the majorants below); a weight gradient also sums over the rows.
"""
import pytest
import torch

import gated_delta_rule_82_b200 as ck

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
F32, BF16 = 2.0 ** -23, 2.0 ** -8
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from gated_delta_rule_82_b200 import build
    build.build()


def make(rows, D, W, act, res, pre, dtype, seed, scale=0.5):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen)
    cast = lambda x: x.to(DT[dtype]).cuda()
    kw = dict(gate=None if act == "none" else cast(2 * rn(rows, D)), gate_act=act,
              residual=cast(rn(rows, D)) if res else None, post_group=W,
              post_weight=(1 + 0.2 * rn(W)).cuda() if W else None, res_scale=scale,
              res_vector=(1 + 0.2 * rn(D)).cuda() if res else None, pre_norm=pre,
              pre_weight=(1 + 0.2 * rn(D)).cuda() if pre else None, eps=EPS)
    return cast(2 * rn(rows, D)), kw, cast(rn(rows, D)), cast(rn(rows, D)) if pre else None


def formulas(y, gate=None, gate_act="none", residual=None, post_group=0, post_weight=None,
             res_scale=1.0, res_vector=None, pre_norm=False, pre_weight=None, eps=EPS):
    R, D = y.shape
    W, m = post_group, y
    if W:
        g = y.reshape(R, D // W, W)
        m = g / (g.pow(2).mean(-1, keepdim=True) + eps).sqrt()
        m = (m if post_weight is None else m * post_weight).reshape(R, D)
    if gate is not None:
        m = m * torch.sigmoid(gate) * (gate if gate_act == "silu" else 1.0)
    s = res_scale * (1.0 if res_vector is None else res_vector)
    h = s * m + (0.0 if residual is None else residual)
    n = None
    if pre_norm:
        n = h / (h.pow(2).mean(-1, keepdim=True) + eps).sqrt()
        n = n if pre_weight is None else n * pre_weight
    return h, n


def in64(kw):
    return {k: v.double() if torch.is_tensor(v) else v for k, v in kw.items()}


def assert_close(got, want, terms, big, name):
    assert got.shape == want.shape and bool(torch.isfinite(got).all()), name
    tol = terms * F32 * big + 1e-30
    if got.dtype == torch.bfloat16:
        tol = tol + BF16 * want.abs()
    worst = float(((got.double() - want).abs() / tol).max())
    assert worst <= 1, f"{name}: {worst:.3g} of the bound"


CASES = [
    # rows, D, W, act, res, pre
    (1, 1, 0, "none", False, True),
    (1, 1, 1, "sigmoid", True, True),
    (3, 7, 7, "silu", True, False),
    (5, 8, 8, "none", True, True),
    (2, 250, 250, "silu", True, True),
    (9, 255, 0, "silu", False, True),
    (130, 256, 64, "sigmoid", False, False),
    (33, 80, 16, "sigmoid", True, True),
    (17, 640, 128, "silu", True, True),
    (65, 1001, 1001, "sigmoid", True, True),
    (700, 2048, 2048, "silu", True, True),
    (1500, 512, 32, "sigmoid", False, False),
    (3, 4104, 4104, "none", True, True),
    (4, 8192, 128, "silu", True, True),
    (2, 8192, 8192, "silu", True, True),
    (2, 8191, 8191, "silu", True, True),
    (5000, 16, 16, "silu", True, True),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,D,W,act,res,pre", CASES)
def test_forward(rows, D, W, act, res, pre, dtype):
    y, kw, _, _ = make(rows, D, W, act, res, pre, dtype, rows + D)
    h, n = ck.block_norm(y, **kw)
    p = in64(kw)
    wh, wn = formulas(y.double(), **p)
    # terms of h: |residual| + |s m|; n's error is h's (in every channel, through the mean too)
    zero = {**p, "residual": None}
    big = formulas(y.double(), **zero)[0].abs() + (0 if p["residual"] is None else p["residual"].abs())
    assert_close(h, wh, D + 64, big, "h")
    if pre:
        ratio = (big.pow(2).mean(-1, keepdim=True) / (wh.pow(2).mean(-1, keepdim=True) + EPS)).sqrt()
        root = (wh.pow(2).mean(-1, keepdim=True) + EPS).sqrt()
        assert_close(n, wn, D + 64, (big / root + wn.abs() * ratio) * (p["pre_weight"].abs() + 1), "n")
    else:
        assert n is None


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,D,W,act,res,pre", CASES)
def test_backward(rows, D, W, act, res, pre, dtype):
    y, kw, dh, dn = make(rows, D, W, act, res, pre, dtype, rows + D)
    got = ck.block_norm_bwd(y, dh, dn, **kw)
    p, y64 = in64(kw), y.double()
    names = {"dy": y64, "dgate": p["gate"], "dresidual": p["residual"],
             "dpost_weight": p["post_weight"], "dres_vector": p["res_vector"],
             "dpre_weight": p["pre_weight"]}
    leaves = {n: t for n, t in names.items() if t is not None}
    for t in leaves.values():
        t.requires_grad_()
    h, n = formulas(y64, **p)
    loss = (h * dh.double()).sum() + ((n * dn.double()).sum() if pre else 0)
    want = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))

    # Majorants: every product and sum of the reverse mode over absolute values (row by row).
    with torch.no_grad():
        ab = lambda t: t.detach().abs()
        norm = lambda t, k: (t.reshape(rows, -1, k).pow(2).mean(-1, keepdim=True) + EPS).sqrt()
        r1 = 1 / norm(y64, W).expand(rows, D // W, W).reshape(rows, D) if W else 1.0
        yhat = ab(y64) * r1
        wp = ab(p["post_weight"]).repeat(D // W) if W else 1.0
        u = yhat * wp
        z = None if p["gate"] is None else p["gate"].detach()
        a = 1.0 if z is None else torch.sigmoid(z) * (z.abs() if act == "silu" else 1.0)
        s = abs(kw["res_scale"]) * (1.0 if p["res_vector"] is None else ab(p["res_vector"]))
        big_h = s * u * a + (0 if p["residual"] is None else ab(p["residual"]))
        G = ab(dh.double())
        if pre:
            r2 = 1 / norm(h.detach(), D).reshape(rows, 1)
            e, hh = ab(dn.double()) * ab(p["pre_weight"]), big_h * r2
            amp = 1 + (hh.pow(2).mean(-1, keepdim=True))      # h's own error through the norm
            G = G + r2 * (e + hh * (e * hh).mean(-1, keepdim=True)) * amp
            pre_big = (ab(dn.double()) * hh * amp).sum(0)
        dm = G * s
        big = {"dresidual": G}
        if z is not None:
            sg = torch.sigmoid(z)
            big["dgate"] = dm * u * (sg * (1 - sg) if act == "sigmoid" else sg * (1 + z.abs() * (1 - sg)))
        if W:
            mean = (dm * a * wp * yhat).reshape(rows, -1, W).mean(-1, keepdim=True)
            mean = mean.expand(rows, D // W, W).reshape(rows, D)
            big["dy"] = r1 * (dm * a * wp + yhat * mean)
            big["dpost_weight"] = (dm * a * yhat).reshape(-1, W).sum(0)
        else:
            big["dy"] = dm * a
        big["dres_vector"] = (G * u * a).sum(0) * abs(kw["res_scale"])
        if pre:
            big["dpre_weight"] = pre_big
    for name, t in names.items():
        if t is None:
            assert got[name] is None, name
        else:
            terms = 2 * D + 128 + (rows * (D // W if name == "dpost_weight" else 1)
                                   if got[name].dim() == 1 else 0)
            assert_close(got[name], want[name], terms, big[name], name)


def test_parts_left_out():
    """Ones for missing weights, zero for a missing residual, dh or dn alone."""
    y, kw, dh, dn = make(40, 96, 96, "silu", True, True, "f32", 3)
    bare = {**kw, "post_weight": None, "pre_weight": None, "res_vector": None, "residual": None}
    full = {**kw, "post_weight": torch.ones(96, device="cuda"), "pre_weight": torch.ones(96, device="cuda"),
            "res_vector": torch.ones(96, device="cuda"), "residual": torch.zeros_like(y)}
    for a, b in zip(ck.block_norm(y, **bare), ck.block_norm(y, **full)):
        assert torch.equal(a, b)
    zero = torch.zeros_like(y)
    for d1, d2 in ((dh, None), (None, dn)):
        a = ck.block_norm_bwd(y, d1, d2, **full)
        b = ck.block_norm_bwd(y, zero if d1 is None else d1, zero if d2 is None else d2, **full)
        for n in ("dy", "dgate", "dresidual", "dpost_weight", "dpre_weight", "dres_vector"):
            assert torch.allclose(a[n], b[n], rtol=0, atol=0), n
        c = ck.block_norm_bwd(y, d1, d2, **bare)
        assert torch.equal(c["dy"], a["dy"]) and torch.equal(c["dgate"], a["dgate"])
        assert all(c[n] is None for n in ("dresidual", "dpost_weight", "dpre_weight", "dres_vector"))


def test_in_place():
    y, kw, _, _ = make(70, 320, 64, "sigmoid", True, True, "bf16", 5)
    h, n = ck.block_norm(y, **kw)
    x2, y2 = kw["residual"].clone(), y.clone()
    a, b = ck.block_norm(y2, **{**kw, "residual": x2}, h=x2, n=y2)
    assert a is x2 and b is y2 and torch.equal(x2, h) and torch.equal(y2, n)


def test_extreme_values():
    """A row of zeros, gates that saturate, values whose squares are large or tiny."""
    D = 64
    y = torch.zeros(4, D, device="cuda")
    y[1], y[2], y[3] = 1e15, 1e-15, torch.linspace(-3, 3, D, device="cuda")
    gate = torch.full_like(y, -200.0)
    gate[:, ::2] = 200.0
    kw = dict(gate=gate, gate_act="silu", post_group=D, pre_norm=True, eps=EPS)
    h, n = ck.block_norm(y, **kw)
    wh, wn = formulas(y.double(), **in64(kw))
    assert torch.allclose(h.double(), wh, rtol=1e-5, atol=1e-30)
    assert torch.allclose(n.double(), wn, rtol=1e-5, atol=1e-30)
    g = ck.block_norm_bwd(y, torch.ones_like(y), torch.ones_like(y), **kw)
    assert all(bool(torch.isfinite(t).all()) for t in g.values() if t is not None)


def test_graph_replay():
    y, kw, dh, dn = make(300, 1024, 128, "silu", True, True, "bf16", 7)
    want, grads = ck.block_norm(y, **kw), ck.block_norm_bwd(y, dh, dn, **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, back = ck.block_norm(y, **kw), ck.block_norm_bwd(y, dh, dn, **kw)
    for x in (*out, *back.values()):
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert all(torch.equal(back[n], grads[n]) for n in grads)
