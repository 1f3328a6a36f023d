"""Block norms where a user has them (GPU): gradients over their own inputs, as the C ABI allows, and the
norms behind a CKDA forward, with the gradients of both."""
import ctypes

import numpy as np
import pytest
import torch

import gated_delta_rule_82_b200 as ck
import oracle
from helpers import fwd_case, oracle_fwd, rel_err
from test_gpu_block_norm import formulas, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from gated_delta_rule_82_b200 import build
    build.build()


# dy, dgate and dresidual over: the forward's inputs; the gradients that came in
@pytest.mark.parametrize("places", [("y", "gate", "residual"), ("dh", "dn", None), ("dn", None, "dh"),
                                    ("y", "dh", "dn"), (None, "gate", "dh")])
# (rows in turn and requested ahead; odd rows, one at a time; rows of one CTA)
@pytest.mark.parametrize("rows,D,W,dtype", [(3000, 512, 64, "bf16"), (1500, 250, 250, "f32"), (400, 8192, 8192, "bf16")])
def test_gradients_in_place(places, rows, D, W, dtype):
    y, kw, dh, dn = make(rows, D, W, "silu", True, True, dtype, rows)
    want = ck.block_norm_bwd(y, dh, dn, **kw)
    at = {"y": y.clone(), "gate": kw["gate"].clone(), "residual": kw["residual"].clone(), "dh": dh.clone(),
          "dn": dn.clone()}
    out = [torch.full_like(y, float("nan")) if p is None else at[p] for p in places]
    sums = [torch.empty_like(kw[n]) for n in ("post_weight", "res_vector", "pre_weight")]
    ws = torch.empty(ck.block_norm_bwd_workspace_bytes(rows, D, W), dtype=torch.uint8, device="cuda")
    st = ck._load().ckda_block_norm_bwd(
        *(t.data_ptr() for t in (at["y"], at["gate"], at["residual"], kw["post_weight"], kw["res_vector"],
                                 kw["pre_weight"], at["dh"], at["dn"], *out, *sums)),
        rows, D, ck._NormFlags(W, 2, kw["res_scale"], kw["eps"]), ck._dtype_code(y), ws.data_ptr(), ws.numel(),
        ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert st == 0
    torch.cuda.synchronize()
    for got, name in zip(out + sums, ("dy", "dgate", "dresidual", "dpost_weight", "dres_vector", "dpre_weight")):
        assert torch.equal(got, want[name]), name


def test_norms_behind_a_ckda_forward():
    """fp32 CKDA, then the norm per head with its gate: outputs and gradients of both against the oracle
    and float64 formulas.  CKDA is held to 1e-4 of the largest value by its own tests, the norm to
    (D + 64) 2^-23 < 1e-5 of its terms; a norm of values of about its root's size passes an error on with a
    factor of a few, and the gradients through both add theirs: 1e-3."""
    B, T, H, d = 2, 130, 3, 32
    D = H * d
    data, g = fwd_case(B, T, H, d, d, kind="ckda", dtype="f32", h0_std=0.3, seed=11)
    args = (g["q"], g["k"], g["v"], g["alpha"], g["beta"], g["h0"])
    gen = torch.Generator().manual_seed(3)
    rn = lambda *s: torch.randn(*s, generator=gen).cuda()
    kw = dict(gate=rn(B, T, D), gate_act="sigmoid", residual=rn(B, T, D), post_group=d, post_weight=1 + 0.1 * rn(d),
              res_scale=0.5, pre_norm=True, pre_weight=1 + 0.1 * rn(D), eps=1e-2)
    dh, dn, dhT = rn(B, T, D), rn(B, T, D), 0.1 * rn(B, H, d, d)

    out, hT = ck.fwd_chunked(*args)
    h, n = ck.block_norm(out.flatten(-2), **kw)
    back = ck.block_norm_bwd(out.flatten(-2), dh, dn, **kw)
    grads = ck.bwd_chunked(*args, back["dy"].view(B, T, H, d), dhT)

    o_ref, s_ref = oracle_fwd(data)
    y = torch.from_numpy(np.ascontiguousarray(o_ref)).reshape(B * T, D).requires_grad_()
    p = {k: (v.double().cpu().reshape(-1, D) if k in ("gate", "residual") else v.double().cpu())
         if torch.is_tensor(v) else v for k, v in kw.items()}
    leaves = [y, p["gate"], p["residual"], p["post_weight"], p["pre_weight"]]
    for t in leaves[1:]:
        t.requires_grad_()
    wh, wn = formulas(y, **p)
    in64 = lambda t: t.double().cpu().reshape(-1, D)
    want = torch.autograd.grad((wh * in64(dh)).sum() + (wn * in64(dn)).sum(), leaves)
    for got, ref in ((hT, s_ref), (h.reshape(-1, D), wh.detach().numpy()), (n.reshape(-1, D), wn.detach().numpy())):
        assert rel_err(got, ref) < 1e-3
    for name, ref in zip(("dy", "dgate", "dresidual", "dpost_weight", "dpre_weight"), want):
        got = back[name]
        assert rel_err(got.reshape(ref.shape), ref.numpy()) < 1e-3, name
    ref = oracle.bwd(data["q"], data["k"], data["v"], data["alpha"], data["beta"], data["h0"],
                     want[0].reshape(B, T, H, d).numpy(), dhT.double().cpu().numpy())
    for name in ("dq", "dk", "dv", "dalpha", "dbeta", "dh0"):
        assert rel_err(grads[name], ref[name]) < 1e-3, name
