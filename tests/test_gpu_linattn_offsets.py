"""Packed linear attention whose offsets in device memory are not the host's (GPU; a captured call whose
offsets are rewritten between replays): the results are undefined, but nothing outside the outputs is
written, no wait runs out, and the next call is right."""
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


def _guarded(shape, dtype):
    """A tensor with 4 KB of a known pattern on both sides."""
    n, pad = int(torch.Size(shape).numel()), 4096 // dtype.itemsize
    buf = torch.full((n + 2 * pad,), 7.0, dtype=dtype, device="cuda")
    return buf[pad:pad + n].view(shape), lambda: bool((buf[:pad] == 7).all() and (buf[pad + n:] == 7).all())


# sequences of one unit (no summaries) and of several; units that belong to another sequence, or to none
@pytest.mark.parametrize("host,device", [
    ([0, 64, 128], [0, 128, 128]), ([0, 64, 128], [0, 0, 128]), ([0, 64, 128], [0, 0, 0]),
    ([0, 10, 20, 300], [0, 300, 300, 300]), ([0, 300, 300], [0, 100, 300]),
    ([0, 700, 701, 1500], [0, 1500, 1500, 1500]), ([0, 700, 701, 1500], [0, 3, 701, 900]),
    ([0, 700, 701, 1500], [-5, 2000, 1, 1500]),
])
@pytest.mark.parametrize("H,Hk,dk,dv,dtype", [(2, 2, 128, 128, "bf16"), (4, 2, 64, 32, "f32")])
def test_offsets_that_disagree_stay_inside(host, device, H, Hk, dk, dv, dtype):
    T, n = host[-1], len(host) - 1
    cpu, dev = (torch.tensor(x, dtype=torch.int32) for x in (host, device))
    d = ref.make((T,), H, Hk, dk, dv, DT[dtype], states=n, seed=T, grads=True, device="cuda")
    args = (d["q"], d["k"], d["v"], d["g"], d["h0"])
    out, out_ok = _guarded((T, H, dv), DT[dtype])
    hT, hT_ok = _guarded((n, H, dk, dv), torch.float32)
    ws = {}
    for name, need in (("fwd", ck.linattn_fwd_workspace_bytes(1, T, H, dk, dv, cpu)),
                       ("bwd", ck.linattn_bwd_workspace_bytes(1, T, H, Hk, dk, dv, cpu))):
        ws[name] = _guarded((need,), torch.uint8)
    kw = dict(cu_seqlens=dev.cuda(), cu_seqlens_cpu=cpu)
    ck.linattn_fwd_chunked(*args, **kw, out=out, hT=hT, workspace=ws["fwd"][0])
    ck.linattn_bwd_chunked(*args, d["do"], d["dhT"], **kw, workspace=ws["bwd"][0])
    torch.cuda.synchronize()
    assert out_ok() and hT_ok() and ws["fwd"][1]() and ws["bwd"][1]()
    assert ck.last_device_status() == 0
    kw["cu_seqlens"].copy_(cpu)
    got = ck.linattn_fwd_chunked(*args, **kw)
    (o, S), (ob, Sb) = ref.forward(*args, cpu)
    for x, want, big in ((got[0], o, ob), (got[1], S, Sb)):
        bound = (T + dk + dv + 64) * ref.F32 * big + 1e-30
        if x.dtype == torch.bfloat16:
            bound = bound + ref.BF16 * (want.abs() + big)
        assert ref.off(x, want, bound) <= 1


def test_workspaces_given_are_checked():
    """One that repeats a byte, lies on the host, or is one byte short is refused by every call; one of
    exactly the bytes asked for serves."""
    T, H, d = 900, 4, 128
    x = ref.make((1, T), H, H, d, d, torch.bfloat16, seed=1, grads=True, device="cuda")
    args, y = (x["q"], x["k"], x["v"], x["g"]), x["v"].view(T, H * d)
    w = torch.ones(H * d, device="cuda")
    f32 = [t.float() for t in args]
    calls = [
        (ck.linattn_fwd_workspace_bytes(1, T, H, d, d),
         lambda ws: [ck.linattn_fwd_chunked(*a, workspace=ws)[0] for a in (args, f32)]),
        (ck.linattn_bwd_workspace_bytes(1, T, H, H, d, d),
         lambda ws: [ck.linattn_bwd_chunked(*a, None, x["do"].to(a[0].dtype), workspace=ws)["dq"]
                     for a in (args, f32)]),
        (ck.block_norm_bwd_workspace_bytes(T, H * d),
         lambda ws: [ck.block_norm_bwd(y, y, y, pre_norm=True, pre_weight=w, workspace=ws)["dy"]]),
    ]
    for need, call in calls:
        one = torch.empty(1, dtype=torch.uint8, device="cuda")
        for bad in (one.expand(need), torch.empty(need, dtype=torch.uint8)):
            with pytest.raises(ValueError):
                call(bad)
        buf = torch.empty(need, dtype=torch.uint8, device="cuda")
        # (the query is the need of the type that takes more: for that one a byte less is too little)
        with pytest.raises(ck.CkdaError) as e:
            call(buf[:need - 1])
        assert e.value.status == 5
        for got, want in zip(call(buf), call(None)):
            assert torch.equal(got, want)
