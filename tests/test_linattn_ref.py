"""The float64 restatement that the GPU tests compare with, itself checked on the CPU: against the
unrolled sum, against differentiation by torch, against differences, and for its majorants."""
import torch

import linattn_ref as ref


def _case(T=7, H=2, dk=4, dv=3, seed=0):
    d = ref.make((1, T), H, 1, dk, dv, torch.float32, states=1, seed=seed, grads=True)
    return {n: x.double() for n, x in d.items()}


def test_recurrence_is_the_unrolled_sum():
    d = _case()
    (o, S), _ = ref.forward(d["q"], d["k"], d["v"], d["g"], d["h0"], scale=0.3)
    q, k, g = ref.expand(d["q"][0], d["k"][0], d["g"][0], 2)
    G = g.cumsum(0)
    for h in range(2):
        for t in range(7):
            want = torch.exp(G[t, h]) * (d["h0"][0, h].T @ q[t, h])
            for j in range(t + 1):
                want = want + torch.exp(G[t, h] - G[j, h]) * (q[t, h] @ k[j, h]) * d["v"][0, j, h]
            assert torch.allclose(o[0, t, h], 0.3 * want, rtol=1e-12, atol=1e-12)


def test_gradients_are_the_derivatives():
    for per_token in (True, False):
        d = _case(seed=3)
        if not per_token:
            d["g"] = d["g"][0, 0].clone()
        leaves = {n: d[n].clone().requires_grad_() for n in ("q", "k", "v", "g", "h0")}
        q, k, g = ref.expand(leaves["q"][0], leaves["k"][0], leaves["g"][0] if per_token else leaves["g"], 2)
        S, loss = leaves["h0"][0], 0.0
        for t in range(7):
            S = torch.exp(g[t])[:, None, None] * S + k[t][:, :, None] * leaves["v"][0, t][:, None, :]
            loss = loss + ((q[t][:, :, None] * S).sum(1) * 0.5 * d["do"][0, t]).sum()
        loss = loss + (S * d["dhT"][0]).sum()
        want = torch.autograd.grad(loss, list(leaves.values()))
        got, big = ref.backward(d["q"], d["k"], d["v"], d["g"], d["h0"], d["do"], d["dhT"], scale=0.5)
        for name, w in zip(("dq", "dk", "dv", "dlog_decay", "dh0"), want):
            assert torch.allclose(got[name], w, rtol=1e-11, atol=1e-11), name
            assert bool((big[name] >= got[name].abs() - 1e-12).all()), name


def test_packed_is_each_sequence_alone():
    d = ref.make((9,), 2, 2, 4, 4, torch.float32, states=3, seed=1, grads=True)
    cu = [0, 4, 4, 9]
    (o, S), _ = ref.forward(d["q"], d["k"], d["v"], d["g"], d["h0"], cu)
    got, _ = ref.backward(d["q"], d["k"], d["v"], d["g"], d["h0"], d["do"], d["dhT"], cu)
    assert torch.equal(S[1], d["h0"][1].double()) and torch.equal(got["dh0"][1], d["dhT"][1].double())
    for s in (0, 2):
        at = slice(cu[s], cu[s + 1])
        one = [d[n][None, at] for n in ("q", "k", "v", "g")]
        (o1, S1), _ = ref.forward(*one, d["h0"][s:s + 1])
        assert torch.equal(o[at], o1[0]) and torch.equal(S[s], S1[0])


def test_an_error_in_the_decay_is_noticed():
    """A decay applied one token late misses the bound that the kernels are held to."""
    d = _case(T=40, seed=5)
    (o, _), (big, _) = ref.forward(d["q"], d["k"], d["v"], d["g"], d["h0"])
    late = torch.cat([torch.zeros_like(d["g"][:, :1]), d["g"][:, :-1]], 1)
    (o2, _), _ = ref.forward(d["q"], d["k"], d["v"], late, d["h0"])
    assert ref.off(o2, o, 120 * ref.F32 * big + ref.BF16 * (o.abs() + big)) > 1
