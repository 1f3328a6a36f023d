"""Timed cases of the decayed linear attention and of the block norms, with their plain forms.

Linear attention with a decay for each head (scale s, log decay g <= 0, state S in R^{dk x dv}):

    S_t = exp(g_t) S_{t-1} + k_t v_t^T,        o_t = s S_t^T q_t

as a chunked form over prompts (batched or packed), its backward pass, and its single-token step on
a state that is updated in place.  Block norms (rows of D channels; RMS norm over groups of W or all D):

    m = norm_W(y) w_post act(gate),   h = x + s r m,   n = norm_D(h) w_pre

with any of norm, gate, residual x and second norm left out, and their backward pass.  `run` takes
the plain torch form, or this package's kernels where `own` is set.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------ the cases

def listed():
    return [
        # one attention layer of the benchmark's 1.3B-shaped model over a batch of two prompts
        dict(name="fwd_layer", kind="fwd", lens="2048,2048", packed=False, H=16, Hk=16, dk=128, dv=128,
             per_token=True, h0=False, dtype="bf16"),
        # the benchmark's long context, continued from a carried state
        dict(name="fwd_long", kind="fwd", lens="65536", packed=False, H=16, Hk=16, dk=128, dv=128,
             per_token=True, h0=True, dtype="bf16"),
        # serving: prompts of ragged lengths packed on one token axis (an empty one among them),
        # grouped heads, fixed decays, fp32
        dict(name="fwd_packed_f32", kind="fwd", lens="777,1,300,0,1500,63", packed=True, H=8, Hk=2, dk=64, dv=128,
             per_token=False, h0=True, dtype="f32"),
        # the training step of the layer above
        dict(name="bwd_layer", kind="bwd", lens="2048,2048", packed=False, H=16, Hk=16, dk=128, dv=128,
             per_token=True, h0=False, dtype="bf16"),
        # a small fp32 training step on an odd length with a carried state and grouped heads
        dict(name="bwd_f32", kind="bwd", lens="333,333,333", packed=False, H=6, Hk=3, dk=64, dv=64,
             per_token=False, h0=True, dtype="f32"),
        # the benchmark's batched decode: 256 sequences, 32 heads, 512 MiB of state
        dict(name="step_batch", kind="step", N=256, H=32, Hk=32, dk=128, dv=128, per_token=True, dtype="bf16"),
        # one sequence of the layer: latency
        dict(name="step_one", kind="step", N=1, H=16, Hk=16, dk=128, dv=128, per_token=True, dtype="bf16"),
        # the attention output of that layer: norm per head and the layer's output gate
        dict(name="norm_heads", kind="norm", rows=4096, D=2048, W=128, act="sigmoid", res=False, pre=False,
             dtype="bf16"),
        # a whole block boundary over a long context: norm after a block, its gate and scale, the
        # residual stream, and the norm before the next block
        dict(name="norm_block", kind="norm", rows=65536, D=2048, W=2048, act="silu", res=True, pre=True,
             dtype="bf16"),
        # the same for the single tokens of a few sequences, on an odd width
        dict(name="norm_tokens", kind="norm", rows=3, D=1001, W=1001, act="none", res=True, pre=True, dtype="f32"),
        # training step of the block boundary
        dict(name="norm_bwd_block", kind="norm_bwd", rows=4096, D=2048, W=2048, act="silu", res=True, pre=True,
             dtype="bf16"),
        # training step of the head norm in fp32, ragged row count
        dict(name="norm_bwd_heads", kind="norm_bwd", rows=1999, D=1024, W=64, act="sigmoid", res=False, pre=False,
             dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["fwd", "fwd", "bwd", "step", "norm", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind in ("fwd", "bwd"):
        dk, dv = rng.choice([16, 32, 64, 128, 128]), rng.choice([16, 32, 64, 128, 128])
        Hk = rng.choice([1, 2, 3, 4, 8, 16])
        H = Hk * rng.choice([1, 1, 2, 4])
        packed = rng.random() < 0.4
        most = (1 << 20 if kind == "fwd" else 1 << 16) // H   # tokens: token-heads of the listed ones
        if packed:
            n = rng.randint(1, 9)
            lens = [0 if rng.random() < 0.05 else _log_int(rng, 1, max(2, min(8192, most // n))) for _ in range(n)]
            lens[rng.randrange(n)] += 1
        else:
            n = rng.choice([1, 1, 2, 3, 5])
            lens = [_log_int(rng, 1, max(2, min(40000, most // n)))] * n
        return dict(kind=kind, lens=",".join(map(str, lens)), packed=packed, H=H, Hk=Hk, dk=dk, dv=dv,
                    per_token=rng.random() < 0.6, h0=rng.random() < 0.5, dtype=dtype)
    if kind == "step":
        Hk = rng.choice([1, 3, 4, 8, 16, 32])
        H = Hk * rng.choice([1, 1, 2])
        return dict(kind="step", N=_log_int(rng, 1, 8192 // H), H=H, Hk=Hk, dk=rng.choice([16, 32, 64, 128, 128]),
                    dv=rng.choice([16, 32, 64, 128, 128]), per_token=rng.random() < 0.6, dtype=dtype)
    W = rng.choice([0, 1, 1, 16, 32, 64, 128])   # 0: no first norm, 1: over the row, else groups
    D = W * rng.choice([1, 2, 5, 8, 16, 32]) if W > 1 else _log_int(rng, 1, 8192)
    if W <= 1 and rng.random() < 0.5:
        D = max(8, D // 8 * 8)
    rows = _log_int(rng, 1, min(100000, (1 << 27 if kind == "norm" else 1 << 23) // (D + 256)))
    return dict(kind=kind, rows=rows, D=D, W=D if W == 1 else W, act=rng.choice(["none", "sigmoid", "silu"]),
                res=rng.random() < 0.6, pre=rng.random() < 0.6, dtype=dtype)


# ----------------------------------------------------------------------------------- the inputs

def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def _offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _unit(x):
    return x / (x.square().sum(-1, keepdim=True) + 1e-6).sqrt()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = TYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device=dev) * std

    s = {"case": case}
    if case["kind"] in ("norm", "norm_bwd"):
        R, D, W = case["rows"], case["D"], case["W"]
        s["y"] = normal(R, D, std=2.0).to(dt)
        s["gate"] = None if case["act"] == "none" else normal(R, D).to(dt)
        s["x"] = normal(R, D).to(dt) if case["res"] else None
        s["w_post"] = 1 + normal(W, std=0.1) if W else None
        s["w_pre"] = 1 + normal(D, std=0.1) if case["pre"] else None
        s["r"] = normal(D, std=0.1).exp() if case["res"] else None   # per-channel residual scale
        s["scale"] = 0.5 if case["res"] else 1.0
        if case["kind"] == "norm_bwd":
            s["dh"] = normal(R, D).to(dt)
            s["dn"] = normal(R, D).to(dt) if case["pre"] else None
        return s

    H, Hk, dk, dv = (case[n] for n in ("H", "Hk", "dk", "dv"))
    if case["kind"] == "step":
        lead, states = (case["N"],), case["N"]
    else:
        lens = _lens(case)
        lead, states = ((sum(lens),) if case["packed"] else (len(lens), lens[0])), len(lens)
        s["cu"] = s["cu_cpu"] = None
        if case["packed"]:
            s["cu_cpu"] = torch.tensor(_offsets(lens), dtype=torch.int32)
            s["cu"] = s["cu_cpu"].to(dev)
    # q and k as the q/k prologue leaves them: unit length per head
    s["q"] = _unit(normal(*lead, Hk, dk)).to(dt)
    s["k"] = _unit(normal(*lead, Hk, dk)).to(dt)
    s["v"] = normal(*lead, H, dv).to(dt)
    # log decays: per token -rate_h softplus(z), with rates that give each head a memory of its
    # own (a token to some hundreds), or a fixed one per head
    rate = torch.exp(torch.rand(H, generator=gen, device=dev) * math.log(256.0)) / 256.0
    if case["per_token"]:
        s["g"] = -rate * torch.nn.functional.softplus(normal(*lead, H))
    else:
        s["g"] = -rate
    if case["kind"] == "step":
        s["state"] = normal(states, H, dk, dv, std=0.2)
        return s
    s["h0"] = normal(states, H, dk, dv, std=0.2) if case["h0"] else None
    if case["kind"] == "bwd":
        s["do"] = normal(*lead, H, dv).to(dt)
        s["dhT"] = normal(states, H, dk, dv, std=0.2) if case["h0"] else None
    return s


# -------------------------------------------------------------------------------- the plain form

CHUNK = 128


def _heads_first(x, H):
    """[B, T, Hx, d] -> fp32 [B, H, T, d], each of the Hx heads repeated H / Hx times."""
    return x.float().transpose(1, 2).repeat_interleave(H // x.shape[2], dim=1)


def _attend(q, k, v, g, h0):
    """Unscaled linear attention of [B, H, T, d] in chunks, without loops; g fp64 [B, H, T].
    Returns (o, state after the last token)."""
    B, H, T, dk = q.shape
    dv, N = v.shape[-1], -(-T // CHUNK)
    pad = N * CHUNK - T

    def split(x):
        return torch.nn.functional.pad(x, (0, 0, 0, pad)).reshape(B, H, N, CHUNK, x.shape[-1])

    qc, kc, vc = split(q), split(k), split(v)
    G = torch.nn.functional.pad(g, (0, pad)).reshape(B, H, N, CHUNK).cumsum(-1)
    tri = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    D = torch.where(tri, G[..., :, None] - G[..., None, :], -math.inf).float().exp()
    o = ((qc @ kc.transpose(-1, -2)) * D) @ vc
    # chunk summaries, and the state entering every chunk as one product over the chunk axis
    E = (kc * (G[..., -1:] - G).float().exp()[..., None]).transpose(-1, -2) @ vc
    after = G[..., -1].cumsum(-1)                       # [B, H, N]
    low = torch.ones(N + 1, N, dtype=torch.bool, device=q.device).tril(-1)
    before = torch.nn.functional.pad(after, (1, 0))      # [B, H, N + 1]
    Wc = torch.where(low, before[..., :, None] - after[..., None, :], -math.inf).float().exp()
    S = (Wc @ E.reshape(B, H, N, dk * dv)).reshape(B, H, N + 1, dk, dv)
    if h0 is not None:
        S = S + before.float().exp()[..., None, None] * h0[:, :, None]
    o = o + (qc * G.float().exp()[..., None]) @ S[:, :, :N]
    return o.reshape(B, H, N * CHUNK, dv)[:, :, :T], S[:, :, N]


def _padded(s):
    """The token axis as a batch: index [n, Tmax] and mask of packed sequences, or None."""
    if s["cu"] is None:
        return None
    cu = s["cu"].long()
    lens = cu[1:] - cu[:-1]
    t = torch.arange(max(_lens(s["case"])), device=cu.device)
    live = t < lens[:, None]
    return torch.where(live, cu[:-1, None] + t, 0), live


def _batch(x, at):
    """[tokens, ..] -> [n, Tmax, ..], zero behind a sequence's end."""
    if at is None:
        return x
    idx, live = at
    return x[idx] * live.reshape(live.shape + (1,) * (x.dim() - 1)).to(x.dtype)


def _tokens(x, at):
    return x if at is None else x[at[1]]


def _gates(s, at):
    g, lead = s["g"], s["v"].shape[:-2]
    return _batch(g.double().expand(*lead, g.shape[-1]), at).transpose(1, 2)   # [B, H, T]


def _plain_fwd(s):
    H, at = s["case"]["H"], _padded(s)
    q, k, v = (_heads_first(_batch(s[n], at), H) for n in "qkv")
    o, hT = _attend(q, k, v, _gates(s, at), s["h0"])
    o = (o * s["case"]["dk"] ** -0.5).transpose(1, 2)
    return _tokens(o, at).to(s["v"].dtype), hT


def _plain_bwd(s):
    """dS_t = exp(g_{t+1}) dS_{t+1} + scale q_t do_t^T backwards in time; dq = scale S do,
    dk = dS v, dv = dS^T k, and dg from dg_t - dg_{t+1} = q_t.dq_t - k_t.dk_t."""
    c = s["case"]
    H, Hk, dt, at = c["H"], c["Hk"], s["v"].dtype, _padded(s)
    q, k, v, do = (_heads_first(_batch(s[n], at), H) for n in ("q", "k", "v", "do"))
    do = do * c["dk"] ** -0.5
    g, h0, dhT = _gates(s, at), s["h0"], s["dhT"]
    dq, ST = _attend(do, v, k, g, None if h0 is None else h0.transpose(-1, -2))
    # time reversed: the decay of a step is applied one token later, the first one not at all
    back = torch.nn.functional.pad(g[..., 1:].flip(-1), (1, 0))
    dv, dS = _attend(k.flip(2), q.flip(2), do.flip(2), back, dhT)
    dk, _ = _attend(v.flip(2), do.flip(2), q.flip(2), back, None if dhT is None else dhT.transpose(-1, -2))
    dv, dk = dv.flip(2), dk.flip(2)
    rows = ((q * dq).double() - (k * dk).double()).sum(-1)
    dg = rows.flip(-1).cumsum(-1).flip(-1)
    if dhT is not None:
        dg = dg + (dhT * ST.transpose(-1, -2)).double().sum((-1, -2))[..., None]
    dh0 = g[..., 0].exp().float()[..., None, None] * dS

    def tokens(x, heads):   # [B, H, T, d] -> the inputs' layout, summed over a group of heads
        x = x.reshape(x.shape[0], heads, H // heads, *x.shape[2:]).sum(2).transpose(1, 2)
        return _tokens(x, at).to(dt)

    if at is not None:      # (a padded token has no gradient)
        dg = dg * at[1][:, None]
    dg = _tokens(dg.transpose(1, 2), at) if c["per_token"] else dg.sum((0, 2))
    return tokens(dq, Hk), tokens(dk, Hk), tokens(dv, H), dg.float(), dh0


def _plain_step(s):
    H = s["case"]["H"]
    q, k, v = (s[n].float().repeat_interleave(H // s[n].shape[1], dim=1) for n in "qkv")
    S = s["g"].exp()[..., None, None] * s["state"] + k[..., :, None] * v[..., None, :]
    s["state"].copy_(S)
    o = (S * q[..., :, None]).sum(-2) * s["case"]["dk"] ** -0.5
    return o.to(s["v"].dtype), s["state"]


EPS = 1e-5


def _norm_parts(s):
    """fp32 pieces of the block norm's forward."""
    c = s["case"]
    R, D, W = c["rows"], c["D"], c["W"]
    y, p = s["y"].float(), {}
    if W:
        yg = y.reshape(R, D // W, W)
        p["r1"] = (yg.square().mean(-1, keepdim=True) + EPS).rsqrt()
        p["yhat"] = yg * p["r1"]
        p["u"] = (p["yhat"] * s["w_post"]).reshape(R, D)
    else:
        p["u"] = y
    z = None if s["gate"] is None else s["gate"].float()
    p["a"] = 1.0 if z is None else z.sigmoid() * (z if c["act"] == "silu" else 1.0)
    p["m"] = p["u"] * p["a"]
    p["s"] = s["scale"] * (1.0 if s["r"] is None else s["r"])
    p["h"] = p["m"] * p["s"] + (0.0 if s["x"] is None else s["x"].float())
    if c["pre"]:
        p["r2"] = (p["h"].square().mean(-1, keepdim=True) + EPS).rsqrt()
        p["hhat"] = p["h"] * p["r2"]
    return p


def _plain_norm(s):
    p, dt = _norm_parts(s), s["y"].dtype
    n = (p["hhat"] * s["w_pre"]).to(dt) if s["case"]["pre"] else None
    return p["h"].to(dt), n


def _plain_norm_bwd(s):
    c, p, dt = s["case"], _norm_parts(s), s["y"].dtype
    R, D, W = c["rows"], c["D"], c["W"]
    dh, dw_pre, dw_post, dgate, dr = s["dh"].float(), None, None, None, None
    if c["pre"]:
        dn = s["dn"].float()
        e = dn * s["w_pre"]
        dw_pre = (dn * p["hhat"]).sum(0)
        dh = dh + p["r2"] * (e - p["hhat"] * (e * p["hhat"]).mean(-1, keepdim=True))
    if s["r"] is not None:
        dr = (dh * p["m"]).sum(0) * s["scale"]
    dm = dh * p["s"]
    du = dm * p["a"]
    if s["gate"] is not None:
        sg = s["gate"].float().sigmoid()
        slope = sg * (1 - sg)
        if c["act"] == "silu":
            slope = sg + s["gate"].float() * slope
        dgate = (dm * p["u"] * slope).to(dt)
    dy = du
    if W:
        dug = du.reshape(R, D // W, W)
        dw_post = (dug * p["yhat"]).sum((0, 1))
        e = dug * s["w_post"]
        dy = (p["r1"] * (e - p["yhat"] * (e * p["yhat"]).mean(-1, keepdim=True))).reshape(R, D)
    return {"dx": dh.to(dt) if c["res"] else None, "dy": dy.to(dt), "dgate": dgate, "dw_post": dw_post,
            "dw_pre": dw_pre, "dr": dr}


# ------------------------------------------------------------------------------ the framework's

def _own(s):
    import gated_delta_rule_82_b200 as ck
    c = s["case"]
    if c["kind"] == "fwd":
        return ck.linattn_fwd_chunked(s["q"], s["k"], s["v"], s["g"], s["h0"], cu_seqlens=s["cu"],
                                      cu_seqlens_cpu=s["cu_cpu"])
    if c["kind"] == "bwd":
        g = ck.linattn_bwd_chunked(s["q"], s["k"], s["v"], s["g"], s["h0"], s["do"], s["dhT"],
                                   cu_seqlens=s["cu"], cu_seqlens_cpu=s["cu_cpu"])
        return g["dq"], g["dk"], g["dv"], g["dlog_decay"], g["dh0"]
    if c["kind"] == "step":
        return ck.linattn_decode_step(s["q"], s["k"], s["v"], s["g"], s["state"]), s["state"]
    args = dict(gate=s["gate"], gate_act=c["act"], residual=s["x"], post_group=c["W"], post_weight=s["w_post"],
                res_scale=s["scale"], res_vector=s["r"], pre_norm=c["pre"], pre_weight=s["w_pre"], eps=EPS)
    if c["kind"] == "norm":
        return ck.block_norm(s["y"], **args)
    g = ck.block_norm_bwd(s["y"], s["dh"], s["dn"], **args)
    return {"dx": g["dresidual"], "dy": g["dy"], "dgate": g["dgate"], "dw_post": g["dpost_weight"],
            "dw_pre": g["dpre_weight"], "dr": g["dres_vector"]}


PLAIN = {"fwd": _plain_fwd, "bwd": _plain_bwd, "step": _plain_step, "norm": _plain_norm, "norm_bwd": _plain_norm_bwd}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["kind"]](state)


# ------------------------------------------------------------------------------------- the work

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["kind"] in ("norm", "norm_bwd"):
        n, c = case["rows"] * case["D"], case
        fwd = 1 + (c["act"] != "none") + c["res"]                   # y, gate, x
        if c["kind"] == "norm":
            return {"bytes": n * e * (fwd + 1 + c["pre"]), "flops": n * (4 + 4 * c["pre"] + 6 * (c["act"] != "none"))}
        grads = 1 + (c["act"] != "none") + c["res"]                 # dy, dgate, dx
        return {"bytes": n * e * (fwd + 1 + c["pre"] + grads), "flops": n * (14 + 10 * c["pre"] + 12 * (c["act"] != "none"))}
    H, Hk, dk, dv = (case[n] for n in ("H", "Hk", "dk", "dv"))
    if case["kind"] == "step":
        N = case["N"]
        vecs = N * (2 * Hk * dk + 2 * H * dv) * e + 4 * (N * H if case["per_token"] else H)
        return {"bytes": 8 * N * H * dk * dv + vecs, "flops": 5 * N * H * dk * dv}
    lens = _lens(case)
    tok, states = sum(lens), 4 * len(lens) * H * dk * dv
    g = 4 * (tok * H if case["per_token"] else H)
    qkv = tok * (2 * Hk * dk + H * dv) * e
    if case["kind"] == "fwd":
        # (update and read-out of the recurrence: 2 dk dv each)
        return {"bytes": qkv + tok * H * dv * e + g + states * (1 + case["h0"]), "flops": 4 * tok * H * dk * dv}
    # (states again, their gradients, dq, dk, dv: 2 dk dv each)
    return {"bytes": 2 * qkv + tok * H * dv * e + 2 * g + states * (1 + 2 * case["h0"]), "flops": 10 * tok * H * dk * dv}


# ---------------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """The recurrence token by token, and the norms by their formulas, in 64 bits."""
    s = prepare(case, seed)
    f = {k: (v.double() if torch.is_tensor(v) and v.is_floating_point() else v) for k, v in s.items()}
    if case["kind"] == "norm":
        return _exact_norm(case, f, False)
    if case["kind"] == "norm_bwd":
        return _exact_norm(case, f, True)
    H, dk = case["H"], case["dk"]
    rep = H // case["Hk"]
    if case["kind"] == "step":
        q, k = (f[n].repeat_interleave(rep, 1) for n in "qk")
        S = torch.exp(f["g"]).reshape(-1, H, 1, 1) * f["state"] + torch.einsum("nhi,nhj->nhij", k, f["v"])
        return torch.einsum("nhij,nhi->nhj", S, q) / math.sqrt(dk), S
    lens = _lens(case)
    if not case["packed"]:
        lens = lens[:1]
    steps = sum(lens)
    cost = steps * len(lens if case["packed"] else _lens(case)) * H * dk * case["dv"] * 8
    if steps > 70000 or (case["kind"] == "bwd" and (steps > 20000 or cost > 4e10)):
        return None
    q, k = (f[n].repeat_interleave(rep, -2) for n in "qk")
    v, do = f["v"], f.get("do")
    g = f["g"].expand(*v.shape[:-1])
    if case["packed"]:        # one sequence after the other, each a batch of one
        parts, cu = [], _offsets(lens)
        for i in range(len(lens)):
            at = slice(cu[i], cu[i + 1])
            parts.append(_exact_sequence(case, *(None if x is None else x[None, at] for x in (q, k, v, g, do)),
                                         *(None if f.get(n) is None else f[n][i:i + 1] for n in ("h0", "dhT"))))
        last = len(parts[0]) - 1   # (the states, or their gradients: a row for each sequence)
        outs = [torch.cat([p[j] if j == last else p[j][0] for p in parts]) for j in range(last + 1)]
    else:
        outs = list(_exact_sequence(case, q, k, v, g, do, f["h0"], f.get("dhT")))
    if case["kind"] == "bwd":
        for j in (0, 1):      # a q/k head gathers the gradients of its value heads
            x = outs[j]
            outs[j] = x.reshape(*x.shape[:-2], H // rep, rep, dk).sum(-2)
        if not case["per_token"]:
            outs[3] = outs[3].reshape(-1, H).sum(0)
    return tuple(outs)


def _exact_sequence(case, q, k, v, g, do, h0, dhT):
    """(o, state) of [B, T, H, d], or the gradients (dq, dk, dv, dg, dh0)."""
    B, T, H, dk = q.shape
    S = q.new_zeros(B, H, dk, v.shape[-1]) if h0 is None else h0.clone()
    a = torch.exp(g)[..., None, None]
    scale, states, o = 1 / math.sqrt(dk), [S], torch.zeros_like(v)
    for t in range(T):
        S = torch.addcmul(a[:, t] * S, k[:, t, :, :, None], v[:, t, :, None, :])
        if do is None:
            o[:, t] = (q[:, t, :, None] @ S)[:, :, 0] * scale
        else:
            states.append(S)
    if do is None:
        return o, S
    dS = torch.zeros_like(S) if dhT is None else dhT
    dq, dk_, dv, dg = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v), torch.zeros_like(g)
    for t in range(T - 1, -1, -1):
        dS = torch.addcmul(dS, q[:, t, :, :, None], do[:, t, :, None, :], value=scale)
        dq[:, t] = (states[t + 1] @ do[:, t, :, :, None])[..., 0] * scale
        dk_[:, t] = (dS @ v[:, t, :, :, None])[..., 0]
        dv[:, t] = (k[:, t, :, None] @ dS)[:, :, 0]
        dS = a[:, t] * dS
        dg[:, t] = (dS * states[t]).sum((-1, -2))
    return dq, dk_, dv, dg, dS


def _exact_norm(case, f, back):
    """By differentiating the 64-bit formulas."""
    names = [n for n in ("x", "y", "gate", "w_post", "w_pre", "r") if f[n] is not None]
    if back:
        for n in names:
            f[n].requires_grad_()
    R, D, W = case["rows"], case["D"], case["W"]
    m = f["y"]
    if W:
        yg = m.view(R, D // W, W)
        m = (yg / torch.sqrt(yg.pow(2).sum(-1, keepdim=True) / W + EPS) * f["w_post"]).view(R, D)
    if f["gate"] is not None:
        m = m / (1 + torch.exp(-f["gate"]))
        if case["act"] == "silu":
            m = m * f["gate"]
    h = f["scale"] * m
    if f["r"] is not None:
        h = h * f["r"]
    if f["x"] is not None:
        h = h + f["x"]
    n = h / torch.sqrt(h.pow(2).sum(-1, keepdim=True) / D + EPS) * f["w_pre"] if case["pre"] else None
    if not back:
        return h, n
    loss = (h * f["dh"]).sum() + ((n * f["dn"]).sum() if case["pre"] else 0)
    got = dict(zip(names, torch.autograd.grad(loss, [f[n] for n in names])))
    return {"dx": got.get("x"), "dy": got["y"], "dgate": got.get("gate"), "dw_post": got.get("w_post"),
            "dw_pre": got.get("w_pre"), "dr": got.get("r")}
