"""Plain float64 restatement of the decayed linear attention, token by token, for the tests:

    S_t = exp(g_t) S_{t-1} + k_t v_t^T,        o_t = scale S_t^T q_t

and its reverse mode, each with a majorant: the same sums over the absolute values of every
factor.  A kernel that rounds an operand of a sum by a relative e is off by at most e times the
majorant, and an fp32 evaluation of it by n 2^-23 times it, n the number of terms one value passes
through (2^-23 covers sums that truncate as well as those that round).
"""
import numpy as np
import torch

BF16 = 2.0 ** -8      # half a step of bf16, relative
F32 = 2.0 ** -23


def _d(x):
    return None if x is None else x.detach().double().cpu()


def expand(q, k, g, H):
    """q, k with a head per value head; g per token."""
    rep = H // q.shape[-2]
    return q.repeat_interleave(rep, -2), k.repeat_interleave(rep, -2), g.expand(*q.shape[:-2], H)


def recurrence(q, k, v, g, h0, scale):
    """out [T, H, dv], final state [H, dk, dv], of one sequence [T, H, d]."""
    T, H, dk = q.shape
    S = torch.zeros(H, dk, v.shape[-1], dtype=torch.float64) if h0 is None else h0.clone()
    a, o = torch.exp(g), torch.zeros_like(v)
    for t in range(T):
        S = a[t, :, None, None] * S + k[t, :, :, None] * v[t, :, None, :]
        o[t] = scale * (q[t, :, :, None] * S).sum(1)
    return o, S


def gradients(q, k, v, g, h0, do, dhT, scale):
    """dq, dk, dv, dg, dh0 of <do, out> + <dhT, hT> for one sequence; per value head and token."""
    T, H, dk = q.shape
    S = torch.zeros(H, dk, v.shape[-1], dtype=torch.float64) if h0 is None else h0.clone()
    a, states = torch.exp(g), [S]
    for t in range(T):
        S = a[t, :, None, None] * S + k[t, :, :, None] * v[t, :, None, :]
        states.append(S)
    R = torch.zeros_like(S) if dhT is None else dhT.clone()
    dq, dkk, dv, dg = (torch.zeros_like(x) for x in (q, k, v, g))
    for t in range(T - 1, -1, -1):
        R = R + scale * q[t, :, :, None] * do[t, :, None, :]
        dq[t] = scale * (states[t + 1] * do[t, :, None, :]).sum(2)
        dkk[t] = (R * v[t, :, None, :]).sum(2)
        dv[t] = (R * k[t, :, :, None]).sum(1)
        R = a[t, :, None, None] * R
        dg[t] = (R * states[t]).sum((1, 2))
    return dq, dkk, dv, dg, R


def sequences(q, cu):
    """Slices of the sequences: rows of a batch, or packed ones by their offsets."""
    if cu is None:
        return [(b,) for b in range(q.shape[0])]
    return [(slice(int(a), int(b)),) for a, b in zip(cu[:-1], cu[1:])]


def forward(q, k, v, g, h0=None, cu=None, scale=None):
    """(out, hT), and the majorants of both, in the layouts of the inputs (float64)."""
    q, k, v, g, h0 = map(_d, (q, k, v, g, h0))
    H = v.shape[-2]
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    q, k, g = expand(q, k, g, H)
    out, big = torch.zeros_like(v), torch.zeros_like(v)
    n = len(sequences(q, cu))
    hT = torch.zeros(n, H, q.shape[-1], v.shape[-1], dtype=torch.float64)
    hbig = torch.zeros_like(hT)
    for s, at in enumerate(sequences(q, cu)):
        i = None if h0 is None else h0[s]
        out[at], hT[s] = recurrence(q[at], k[at], v[at], g[at], i, scale)
        big[at], hbig[s] = recurrence(q[at].abs(), k[at].abs(), v[at].abs(), g[at],
                                      None if i is None else i.abs(), abs(scale))
    return (out, hT), (big, hbig)


def backward(q, k, v, g, h0, do, dhT=None, cu=None, scale=None):
    """Dicts of the gradients and of their majorants (float64, the library's layouts)."""
    per_token = g.dim() != 1
    Hk, dk = q.shape[-2:]
    q, k, v, g, h0, do, dhT = map(_d, (q, k, v, g, h0, do, dhT))
    H = v.shape[-2]
    scale = dk ** -0.5 if scale is None else scale
    qe, ke, ge = expand(q, k, g, H)
    ge = ge.contiguous()
    n = len(sequences(qe, cu))
    res, maj = ({"dq": torch.zeros_like(qe), "dk": torch.zeros_like(qe), "dv": torch.zeros_like(v),
                 "dlog_decay": torch.zeros_like(ge),
                 "dh0": torch.zeros(n, H, dk, v.shape[-1], dtype=torch.float64)} for _ in range(2))
    ab = lambda x: None if x is None else x.abs()
    for s, at in enumerate(sequences(qe, cu)):
        i, f = (None if x is None else x[s] for x in (h0, dhT))
        for to, args in ((res, (qe[at], ke[at], v[at], ge[at], i, do[at], f)),
                         (maj, (qe[at].abs(), ke[at].abs(), v[at].abs(), ge[at], ab(i),
                                do[at].abs(), ab(f)))):
            got = gradients(*args, scale)
            for name, x in zip(("dq", "dk", "dv", "dlog_decay"), got):
                to[name][at] = x
            to["dh0"][s] = got[4]
        # the library forms dg from sums over the later tokens of q.dq - k.dk: its error is
        # relative to the sum of their absolute values, not to dg's own terms
        rows = (qe[at].abs() * maj["dq"][at] + ke[at].abs() * maj["dk"][at]).sum(-1)
        tail = rows.flip(0).cumsum(0).flip(0)
        if f is not None:
            _, hbig = recurrence(qe[at].abs(), ke[at].abs(), v[at].abs(), ge[at], ab(i), scale)
            tail = tail + (hbig * f.abs()).sum((1, 2))
        maj["dlog_decay"][at] = torch.maximum(maj["dlog_decay"][at], tail)
    for to in (res, maj):
        for name in ("dq", "dk"):
            x = to[name]
            to[name] = x.reshape(*x.shape[:-2], Hk, H // Hk, dk).sum(-2)
        if not per_token:
            to["dlog_decay"] = to["dlog_decay"].reshape(-1, H).sum(0)
    return res, maj


def make(lead, H, Hk, dk, dv, dtype, *, per_token=True, states=0, seed=0, grads=False, strong=1.0,
         device="cpu"):
    """Inputs of one call; lead: (B, T) or (T,) for packed tokens."""
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen)
    unit = lambda x: x / (x.square().sum(-1, keepdim=True) + 1e-6).sqrt()
    rate = strong * torch.exp(-4 * torch.rand(H, generator=gen))
    d = {"q": unit(rn(*lead, Hk, dk)).to(dtype), "k": unit(rn(*lead, Hk, dk)).to(dtype),
         "v": rn(*lead, H, dv).to(dtype),
         "g": -rate * torch.nn.functional.softplus(rn(*lead, H)) if per_token else -rate,
         "h0": rn(states, H, dk, dv) * 0.2 if states else None}
    if grads:
        d["do"] = rn(*lead, H, dv).to(dtype)
        d["dhT"] = rn(states, H, dk, dv) * 0.2 if states else None
    return {n: None if x is None else x.to(device) for n, x in d.items()}


def off(got, want, bound) -> float:
    """Largest error in units of its bound (at most 1 passes)."""
    got, want = _d(got), _d(want)
    assert got.shape == want.shape
    if not got.numel():
        return 0.0
    err, bound = (got - want).abs(), _d(bound)
    assert bool(torch.isfinite(got).all()), "non-finite result"
    return float(np.nan_to_num((err / bound.clamp_min(1e-300)).numpy(), nan=0.0).max())
