"""Precision of the linear attention's bf16 calls (GPU): what its operands may lose, and that neither the
size of the call nor the gradients asked for beside it change a result.

With `big` the sum of the absolute values of a result's terms (linattn_ref), n = T + dk + dv + 64:
  scores, state  two bf16 terms each: the first leaves at most 2^-8 of a value, the second 2^-8 of that;
                 2^-16 of the terms that pass through one of them, 2^-15 with room for both
  fp32 sums      n 2^-23 big (as in the operators' other tests)
  output         half a step of bf16, 2^-8 of the value
A state of one term would add 2^-9 of each of its elements, at random signs 2^-9 of a result's usual
size: beyond the bound wherever a result is small.
"""
import pytest
import torch

import gated_delta_rule_82_b200 as ck
import linattn_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from gated_delta_rule_82_b200 import build
    build.build()


def _bound(want, big, n):
    return ref.BF16 * want.abs() + (2.0 ** -15 + n * ref.F32) * big + 1e-30


# (heads, head sizes: tcgen05 and warp tiles; tokens: one to many units)
@pytest.mark.parametrize("B,T,H,Hk,dk,dv", [
    (1, 320, 16, 16, 128, 128), (2, 700, 16, 8, 128, 128), (20, 100, 4, 4, 128, 128),
    (1, 320, 16, 16, 64, 64), (2, 200, 32, 32, 32, 128), (1, 320, 16, 16, 128, 16),
])
def test_outputs_are_rounded_once(B, T, H, Hk, dk, dv):
    d = ref.make((B, T), H, Hk, dk, dv, torch.bfloat16, states=B, seed=T + dv, grads=True, strong=0.1,
                 device="cuda")
    args, n = (d["q"], d["k"], d["v"], d["g"], d["h0"]), T + dk + dv + 64
    (o, _), (big, _) = ref.forward(*args)
    assert ref.off(ck.linattn_fwd_chunked(*args)[0], o, _bound(o, big, n)) <= 1
    want, big = ref.backward(*args, d["do"], d["dhT"])
    got = ck.linattn_bwd_chunked(*args, d["do"], d["dhT"])
    for name in ("dq", "dk", "dv"):
        assert ref.off(got[name], want[name], _bound(want[name], big[name], n)) <= 1, name


@pytest.mark.parametrize("B,T,H,Hk,dk,dv", [
    (1, 700, 16, 16, 128, 128), (1, 700, 16, 8, 128, 128), (1, 700, 16, 16, 64, 64), (3, 100, 8, 4, 32, 16),
])
def test_other_gradients_do_not_change_dq_and_dk(B, T, H, Hk, dk, dv):
    """Whether the gradients of the decays and of h0 are asked for: the same dq, dk, dv bit for bit."""
    d = ref.make((B, T), H, Hk, dk, dv, torch.bfloat16, states=B, seed=T, grads=True, device="cuda")
    args = (d["q"], d["k"], d["v"], d["g"], d["h0"], d["do"], d["dhT"])
    got = ck.linattn_bwd_chunked(*args)
    less = ck.linattn_bwd_chunked(*args, want_dlog_decay=False, want_dh0=False)
    for name in ("dq", "dk", "dv"):
        assert torch.equal(got[name], less[name]), name


@pytest.mark.parametrize("T,H,dk,dv", [(100, 2, 128, 128), (1, 16, 128, 128), (77, 4, 64, 64), (128, 2, 32, 128)])
def test_a_sequence_alone_is_the_sequence_in_a_batch(T, H, dk, dv):
    """Up to two chunks are one unit in any batch: the same results bit for bit, however large the call."""
    B = 48
    d = ref.make((B, T), H, H, dk, dv, torch.bfloat16, states=B, seed=T, grads=True, device="cuda")
    args = [d[n] for n in ("q", "k", "v", "g", "h0")]
    out, hT = ck.linattn_fwd_chunked(*args)
    grads = ck.linattn_bwd_chunked(*args, d["do"], d["dhT"])
    for b in (0, 7, B - 1):
        one = [x[b:b + 1].contiguous() for x in (*args, d["do"], d["dhT"])]
        o, h = ck.linattn_fwd_chunked(*one[:5])
        assert torch.equal(o, out[b:b + 1]) and torch.equal(h, hT[b:b + 1])
        for name, x in ck.linattn_bwd_chunked(*one).items():
            assert torch.equal(x, grads[name][b:b + 1]), name


def _neighbours(B, T, H, d):
    """q_t = do_t = e_{t-1}, k_t = v_t = e_t: the only products are those of a token with the one before
    it, and dlog_decay_t is the decay between them."""
    eye = torch.eye(d, dtype=torch.bfloat16, device="cuda")
    rows = lambda first: eye[(torch.arange(T) + first) % d].view(1, T, 1, d).expand(B, T, H, d).contiguous()
    return rows(d - 1), rows(0), rows(0), rows(d - 1)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("forget", [-float("inf"), -80.0])
@pytest.mark.parametrize("T,at", [(16, range(12)), (16, [3, 4, 5, 6, 9]), (60, [0, 17, 18, 19, 20, 35, 36, 37, 38])])
def test_decays_behind_resets(T, at, forget, d):
    """Decays behind resets (or behind tokens that forget all but e^-80) of the same 16 tokens.  Every
    product has one term that is not zero, so a row of q.dq or k.dk has the roundings of its decay alone: of
    the exponent (2^-24 of at most 2), of 2^x (2^-22) and of three-term operands (2^-24), together below
    4 2^-23; 8 2^-23 of the sum of the later rows bounds their differences.  (Differences of single floats
    of -1000 were off by 1e-4.)"""
    B, H = 24, 2
    q, k, v, do = _neighbours(B, T, H, d)
    g = -torch.rand(B, T, H, generator=torch.Generator().manual_seed(T)).cuda()
    g[:, list(at)] = forget
    want, big = ref.backward(q, k, v, g, None, do, None, scale=1.0)
    got = ck.linattn_bwd_chunked(q, k, v, g, None, do, scale=1.0)
    assert ref.off(got["dlog_decay"], want["dlog_decay"], 8 * ref.F32 * big["dlog_decay"] + 1e-30) <= 1


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
def test_sums_of_the_decay_gradient(d, dtype):
    """Whole numbers, no decay: rows of q.dq and k.dk stay below 2^24 and are exact, their sums over a chunk
    pass 2^27, and the gradients, differences of those, come out exactly (0 before the first key)."""
    T, H = 128, 3
    gen = torch.Generator().manual_seed(d)
    q, k, v, do = (torch.randint(0, 4, (1, T, H, d), generator=gen).to(dtype) for _ in range(4))
    for x in (q, k, v, do):
        x[:, :63] = 0
    for x in (k, v):
        x[:, 63] = 0
        x[:, 63, :, 0] = 1
    q, k, v, do = (x.cuda() for x in (q, k, v, do))
    g = torch.zeros(1, T, H, device="cuda")
    want, _ = ref.backward(q, k, v, g, None, do, None, scale=1.0)
    rows = (ref.expand(q, k, g, H)[0].double().cpu() * want["dq"]).sum(-1)
    assert float(rows.max()) < 2 ** 24 and (d < 128 or float(rows.sum(1).max()) > 2 ** 27)
    got = ck.linattn_bwd_chunked(q, k, v, g, None, do, scale=1.0)
    assert torch.equal(got["dlog_decay"].cpu(), want["dlog_decay"].float())


def test_sums_of_the_decay_gradient_past_32_bits():
    """The same behind 2^31 elements: tokens of zeros, then some of whole numbers; the gradients of the last
    tokens are exact, and 0 on all before them."""
    torch.cuda.empty_cache()
    T, H, d, tail = 1_060_001, 16, 128, 150
    gen = torch.Generator().manual_seed(1)
    part = [torch.randint(0, 4, (1, tail, H, d), generator=gen).bfloat16() for _ in range(4)]
    full = [torch.zeros(1, T, H, d, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    for x, p in zip(full, part):
        x[:, -tail:] = p.cuda()
    q, k, v, do = full
    want, _ = ref.backward(*part[:3], torch.zeros(1, tail, H), None, part[3], None, scale=1.0)
    got = ck.linattn_bwd_chunked(q, k, v, torch.zeros(1, T, H, device="cuda"), None, do, scale=1.0)
    rows = [(part[0].double() * want["dq"]).sum(-1), (part[1].double() * want["dk"]).sum(-1)]
    assert float(max(x.max() for x in rows)) < 2 ** 24
    dg = got["dlog_decay"]
    assert torch.equal(dg[:, -tail:].cpu(), want["dlog_decay"].float())
    assert bool((dg[:, :-tail] == 0).all())
    for n in ("dq", "dk", "dv"):
        assert torch.equal(got[n][:, -tail:].cpu(), want[n].to(torch.bfloat16)), n
        assert not bool(got[n][:, :-tail].any()), n
    del full, q, k, v, do, got
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_of_the_decay_gradient(dtype):
    """Whole numbers again, enough of them for rows of q.dq and k.dk past 2^24 (each of their elements, and
    the products of 32 channels, below): the rows are sums in fp64 too, and the gradients exact."""
    T, H, d = 230, 2, 128
    gen = torch.Generator().manual_seed(3)
    q, k, v, do = (torch.randint(0, 4, (1, T, H, d), generator=gen).to(dtype).cuda() for _ in range(4))
    g = torch.zeros(1, T, H, device="cuda")
    want, _ = ref.backward(q, k, v, g, None, do, None, scale=1.0)
    parts = [(x.double().cpu() * want[n]).reshape(1, T, H, 4, 32).sum(-1) for x, n in ((q, "dq"), (k, "dk"))]
    assert all(2 ** 22 < float(p.max()) < 2 ** 24 < float(p.sum(-1).max()) for p in parts)
    got = ck.linattn_bwd_chunked(q, k, v, g, None, do, scale=1.0)
    assert torch.equal(got["dlog_decay"].cpu(), want["dlog_decay"].float())
