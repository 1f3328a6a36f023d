"""How the linear attention is cut into units and launches (GPU): one to many units a sequence, summed
up by the runs or by a scan, dq, dk and dv in one launch or two, narrow heads several to an SM, all
against the float64 reference with the bounds of the operators' other tests.

Bounds: every result is a sum of products over at most T tokens and two channel axes, so its fp32 error
is at most (T + dk + dv + 64) 2^-24 times the sum of the terms' absolute values; results that come out
in bf16 add a rounding of the value, 2^-8 of it, and one of each of the state's elements, 2^-8 of the sum.
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


def _check(got, want, big, n):
    for name, x in got.items():
        if x is not None:
            bound = n * ref.F32 * big[name] + 1e-30
            if x.dtype == torch.bfloat16:
                bound = bound + ref.BF16 * (want[name].abs() + big[name])
            assert ref.off(x, want[name], bound) <= 1, name


# (H, Hk, dk, dv, type): tcgen05, warp tiles of every width, grouped heads, dk != dv
SHAPES = [(2, 2, 128, 128, "bf16"), (16, 16, 128, 128, "bf16"), (4, 2, 64, 64, "bf16"),
          (3, 3, 32, 32, "f32"), (2, 1, 128, 128, "f32"), (2, 2, 16, 64, "bf16")]


@pytest.mark.parametrize("T", [64, 128, 129, 192, 257, 640])
@pytest.mark.parametrize("H,Hk,dk,dv,dtype", SHAPES)
def test_units(T, H, Hk, dk, dv, dtype):
    d = ref.make((2, T), H, Hk, dk, dv, DT[dtype], states=2, seed=T + H, grads=True, device="cuda")
    args, n = (d["q"], d["k"], d["v"], d["g"], d["h0"]), T + dk + dv + 64
    (o, S), (ob, Sb) = ref.forward(*args)
    out, hT = ck.linattn_fwd_chunked(*args)
    _check(dict(out=out, hT=hT), dict(out=o, hT=S), dict(out=ob, hT=Sb), n)
    want, big = ref.backward(*args, d["do"], d["dhT"])
    _check(ck.linattn_bwd_chunked(*args, d["do"], d["dhT"]), want, big, n)
    _check(ck.linattn_bwd_chunked(*args, d["do"], d["dhT"], want_dlog_decay=False), want, big, n)
    assert ck.last_device_status() == 0


def test_workspace_serves_either_type():
    """The queries know no type: their size is enough for both, and one byte less than a call's need
    is refused."""
    for dk, dv in ((128, 128), (32, 64)):
        for dtype in DT.values():
            d = ref.make((1, 900), 4, 4, dk, dv, dtype, seed=1, grads=True, device="cuda")
            args = (d["q"], d["k"], d["v"], d["g"])
            for need, call in (
                    (ck.linattn_fwd_workspace_bytes(1, 900, 4, dk, dv),
                     lambda w: ck.linattn_fwd_chunked(*args, workspace=w)[0]),
                    (ck.linattn_bwd_workspace_bytes(1, 900, 4, 4, dk, dv),
                     lambda w: ck.linattn_bwd_chunked(*args, None, d["do"], workspace=w)["dq"])):
                pad = torch.full((need + 4096,), 7, dtype=torch.uint8, device="cuda")
                with_it, own = call(pad[:need]), call(None)
                assert torch.equal(with_it, own) and bool((pad[need:] == 7).all())
                with pytest.raises(ck.CkdaError):
                    call(pad[:256])


def test_fixed_decays_over_packed_gaps():
    """Fixed decays' gradients sum over every chunk of sequences that end anywhere in a chunk, empty
    ones between them, after a call that left other values in the same workspace."""
    lens = [0, 63, 64, 0, 0, 65, 1, 130, 0, 128, 0]
    cu = torch.tensor([0, *torch.tensor(lens).cumsum(0)], dtype=torch.int32)
    d = ref.make((sum(lens),), 3, 3, 32, 32, torch.float32, states=len(lens), per_token=False, seed=8,
                 grads=True, device="cuda")
    args = (d["q"], d["k"], d["v"], d["g"], d["h0"], d["do"], d["dhT"])
    need = ck.linattn_bwd_workspace_bytes(0, 0, 3, 3, 32, 32, cu)
    ws = torch.full((need // 8,), float("nan"), dtype=torch.float64, device="cuda")
    want, big = ref.backward(*args, cu)
    got = ck.linattn_bwd_chunked(*args, cu_seqlens=cu.cuda(), cu_seqlens_cpu=cu, workspace=ws)
    _check(got, want, big, max(lens) + 128)


def _same(a, b, steps):
    """bf16 values that differ by rounding only: `steps` times 2^-8 of the largest."""
    return float((a.float() - b.float()).abs().max()) <= steps * 2 ** -8 * float(b.float().abs().max())


def test_offsets_past_32_bits():
    """More than 2^31 elements in an array: the last tokens, rows and sequences are those of a call on
    the tail alone (decays of e^-0.05 a token on average forget what lies 3000 tokens back)."""
    torch.cuda.empty_cache()
    T, H, d, tail = 1_060_001, 16, 128, 5000
    rand = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda").normal_().mul_(s[-1] ** -0.5)
    q, k, v, do = (rand(1, T, H, d) for _ in range(4))
    g = -0.1 * torch.rand(1, T, H, device="cuda")
    part = [x[:, -tail - 3000:].contiguous() for x in (q, k, v, g)]
    out, hT = ck.linattn_fwd_chunked(q, k, v, g)
    o2, h2 = ck.linattn_fwd_chunked(*part)
    assert _same(out[:, -tail:], o2[:, 3000:], 2) and float((hT - h2).abs().max()) < 1e-5
    grads = ck.linattn_bwd_chunked(q, k, v, g, None, do)
    less = ck.linattn_bwd_chunked(*part, None, do[:, -tail - 3000:].contiguous())
    for n in ("dq", "dk", "dv", "dlog_decay"):
        assert _same(grads[n][:, -tail:], less[n][:, 3000:], 2), n
    del grads, out, do
    rows = q.view(-1, 2048), k.view(-1, 2048), v.view(-1, 2048)
    kw = dict(gate_act="silu", post_group=2048, pre_norm=True)
    h, n = ck.block_norm(rows[0], gate=rows[1], residual=rows[2], **kw)
    last = [r[-9:].contiguous() for r in rows]
    h2, n2 = ck.block_norm(last[0], gate=last[1], residual=last[2], **kw)
    assert torch.equal(h[-9:], h2) and torch.equal(n[-9:], n2)
    del h, n, q, k, v, rows
    N = 4200
    state = torch.empty(N, 32, 128, 128, device="cuda").normal_()
    q, k, v = (rand(N, 32, 128) for _ in range(3))
    g = -torch.rand(N, 32, device="cuda")
    end = state[-3:].clone()
    o = ck.linattn_decode_step(q, k, v, g, state)
    o2 = ck.linattn_decode_step(*(x[-3:].contiguous() for x in (q, k, v, g)), end)
    assert torch.equal(o[-3:], o2) and torch.equal(state[-3:], end)
    del state
    torch.cuda.empty_cache()
