"""Refusals of the decayed linear attention and of the block norms: the C ABI on the host (fake
addresses, never dereferenced: every call is invalid in exactly the stated way and is rejected before
any launch), and the Python binding.  CPU only."""
import ctypes

import pytest
import torch

import gated_delta_rule_82_b200 as ck
from gated_delta_rule_82_b200 import build as ckbuild

OK, NULL, SHAPE, UNSUP, ALIGN, WORKSPACE, CUDA, ARG, DEVICE_STATUS = range(9)
P = 0x100000       # 1 MiB apart: the arrays of the small calls below do not touch
BAD = ctypes.c_size_t(-1).value


@pytest.fixture(scope="module")
def lib():
    ckbuild.build()
    return ck._load()


def flags(l2norm=0, rope_theta=0.0, scale=0.0, gate_logits=0, qk_heads=0):
    return ck._Flags(l2norm, rope_theta, 0, scale, 0, 0, gate_logits, 0, qk_heads)


def offsets(*cu):
    return (ctypes.c_int * len(cu))(*cu)


FWD = dict(q=P, k=2 * P, v=3 * P, g=4 * P, per_token=1, h0=5 * P, out=6 * P, hT=7 * P, B=1, T=40,
           cu=None, cu_host=None, n=0, H=2, dk=16, dv=32, fl=flags(), dtype=1, ws=8 * P, wsb=1 << 20)


def fwd(lib, **kw):
    a = {**FWD, **kw}
    return lib.ckda_linattn_fwd_chunked(a["q"], a["k"], a["v"], a["g"], a["per_token"], a["h0"], a["out"],
                                        a["hT"], a["B"], a["T"], a["cu"], a["cu_host"], a["n"], a["H"],
                                        a["dk"], a["dv"], a["fl"], a["dtype"], a["ws"], a["wsb"], None)


PACKED = dict(cu=9 * P, n=2)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(g=None), NULL),
    (dict(out=None), NULL),
    (dict(cu=9 * P, n=2), NULL),                                   # device offsets alone
    (dict(cu_host=offsets(0, 20, 40), n=2), NULL),                 # host offsets alone
    (dict(B=0), SHAPE), (dict(T=0), SHAPE), (dict(H=0), SHAPE), (dict(T=-3), SHAPE),
    (dict(B=1 << 16, T=1 << 16, H=1 << 10), SHAPE),                # more elements than any device holds
    (dict(T=0x7fffffff), SHAPE),                                   # whole chunks would pass 2^31
    ({**PACKED, "n": 0, "cu_host": offsets(0)}, SHAPE),
    ({**PACKED, "cu_host": offsets(1, 20, 40)}, ARG),              # does not start at 0
    ({**PACKED, "cu_host": offsets(0, 30, 20)}, ARG),              # decreasing
    ({**PACKED, "cu": 9 * P + 2, "cu_host": offsets(0, 20, 40)}, ALIGN),
    (dict(dk=24), UNSUP), (dict(dv=256), UNSUP), (dict(dtype=2), UNSUP),
    (dict(per_token=2), ARG),
    (dict(fl=flags(l2norm=1)), ARG), (dict(fl=flags(rope_theta=1e4)), ARG),
    (dict(fl=flags(gate_logits=1)), ARG), (dict(fl=flags(qk_heads=-1)), ARG),
    (dict(H=3, fl=flags(qk_heads=2)), ARG),
    (dict(q=P + 8), ALIGN), (dict(hT=7 * P + 4), ALIGN), (dict(g=4 * P + 2), ALIGN),
    (dict(ws=8 * P + 8), ALIGN),
    (dict(out=3 * P), ARG),                                        # out is v
    (dict(hT=6 * P), ARG),                                         # hT is out
    (dict(hT=5 * P + 16), ARG),                                    # hT overlaps h0 in part
    (dict(T=4096, ws=None), WORKSPACE), (dict(T=4096, wsb=64), WORKSPACE),
    (dict(T=4096, q=P, k=2 * P, v=3 * P, out=8 * P + 64, ws=8 * P, wsb=1 << 30), ARG),   # workspace on out
])
def test_forward_refusals(lib, kw, want):
    assert fwd(lib, **kw) == want


BWD = dict(q=P, k=2 * P, v=3 * P, g=4 * P, per_token=1, h0=5 * P, do=6 * P, dhT=7 * P, dq=10 * P,
           dk=11 * P, dv=12 * P, dg=13 * P, dh0=14 * P, B=1, T=40, cu=None, cu_host=None, n=0, H=2, dk_=16,
           dv_=32, fl=flags(), dtype=1, ws=16 * P, wsb=1 << 24)


def bwd(lib, **kw):
    a = {**BWD, **kw}
    return lib.ckda_linattn_bwd_chunked(a["q"], a["k"], a["v"], a["g"], a["per_token"], a["h0"], a["do"],
                                        a["dhT"], a["dq"], a["dk"], a["dv"], a["dg"], a["dh0"], a["B"],
                                        a["T"], a["cu"], a["cu_host"], a["n"], a["H"], a["dk_"], a["dv_"],
                                        a["fl"], a["dtype"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(do=None), NULL), (dict(dq=None), NULL), (dict(dk=None), NULL), (dict(dv=None), NULL),
    (dict(q=None), NULL), (dict(T=0), SHAPE), (dict(dk_=8), UNSUP), (dict(dtype=3), UNSUP),
    (dict(per_token=-1), ARG), (dict(fl=flags(l2norm=1)), ARG), (dict(H=3, fl=flags(qk_heads=2)), ARG),
    (dict(dq=10 * P + 8), ALIGN), (dict(dg=13 * P + 1), ALIGN), (dict(dh0=14 * P + 4), ALIGN),
    (dict(ws=None), WORKSPACE), (dict(wsb=16), WORKSPACE),
    (dict(dq=P), ARG), (dict(dv=6 * P), ARG), (dict(dk=10 * P), ARG), (dict(dh0=7 * P), ARG),
    (dict(dg=16 * P + 256), ARG),                                  # a gradient inside the workspace
])
def test_backward_refusals(lib, kw, want):
    assert bwd(lib, **kw) == want


STEP = dict(q=P, k=2 * P, v=3 * P, g=4 * P, per_token=1, state=5 * P, out=6 * P, N=2, H=2, dk=16, dv=32,
            fl=flags(), dtype=1)


def step(lib, **kw):
    a = {**STEP, **kw}
    return lib.ckda_linattn_decode_step(a["q"], a["k"], a["v"], a["g"], a["per_token"], a["state"], a["out"],
                                        a["N"], a["H"], a["dk"], a["dv"], a["fl"], a["dtype"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(state=None), NULL), (dict(g=None), NULL), (dict(N=0), SHAPE), (dict(H=-1), SHAPE),
    (dict(N=1 << 26, H=4), SHAPE), (dict(dv=8), UNSUP), (dict(dtype=-1), UNSUP), (dict(per_token=3), ARG),
    (dict(state=5 * P + 8), ALIGN), (dict(g=4 * P + 3), ALIGN), (dict(out=5 * P), ARG), (dict(out=3 * P), ARG),
    (dict(state=2 * P), ARG), (dict(fl=flags(rope_theta=1.0)), ARG), (dict(H=3, fl=flags(qk_heads=2)), ARG),
])
def test_step_refusals(lib, kw, want):
    assert step(lib, **kw) == want


def test_linattn_workspace_queries(lib):
    f, b = lib.ckda_linattn_fwd_workspace_bytes, lib.ckda_linattn_bwd_workspace_bytes
    assert f(1, 100, None, 0, 4, 128, 128) == 0                    # one unit: nothing to keep
    assert 0 < f(1, 65536, None, 0, 16, 128, 128) < 1 << 30
    assert f(0, 0, offsets(0, 5, 5, 4000), 3, 4, 64, 64) > 0
    assert f(1, 65536, None, 0, 4096, 16, 16) == 0                 # heads enough to fill the device
    for bad in ((0, 5, None, 0, 1, 16, 16), (1, 5, None, 0, 1, 17, 16), (1, 5, offsets(0, 3, 2), 2, 1, 16, 16),
                (1, 5, None, 0, 0, 16, 16)):
        assert f(*bad) == BAD
    assert b(1, 1, None, 0, 1, 0, 16, 16) > 0
    assert b(2, 300, None, 0, 4, 2, 64, 64) > b(2, 300, None, 0, 4, 4, 64, 64)   # shared heads are summed
    assert b(1, 5, None, 0, 3, 2, 16, 16) == BAD


NORM = dict(y=P, gate=2 * P, x=3 * P, wp=4 * P, r=5 * P, wn=6 * P, h=7 * P, n=8 * P, rows=4, D=64, group=64,
            act=1, scale=1.0, eps=1e-5, dtype=1)


def norm(lib, **kw):
    a = {**NORM, **kw}
    return lib.ckda_block_norm(a["y"], a["gate"], a["x"], a["wp"], a["r"], a["wn"], a["h"], a["n"], a["rows"],
                               a["D"], ck._NormFlags(a["group"], a["act"], a["scale"], a["eps"]), a["dtype"],
                               None)


NORM_BAD = [
    (dict(y=None), NULL), (dict(rows=0), SHAPE), (dict(D=0), SHAPE),
    (dict(D=8193, group=0), UNSUP), (dict(group=24), UNSUP), (dict(group=128), UNSUP), (dict(group=-1), UNSUP),
    (dict(dtype=5), UNSUP),
    (dict(act=0), ARG), (dict(gate=None), ARG), (dict(act=3), ARG), (dict(eps=0.0), ARG),
    (dict(eps=float("nan")), ARG), (dict(eps=-1.0), ARG), (dict(scale=float("inf")), ARG),
    (dict(y=P + 8), ALIGN), (dict(wp=4 * P + 2), ALIGN), (dict(x=3 * P + 4), ALIGN),
]


@pytest.mark.parametrize("kw,want", NORM_BAD + [
    (dict(h=None), NULL), (dict(n=8 * P + 2), ALIGN),
    (dict(h=P + 16), ARG),              # shifted by part of a row: rows would be read after being written
    (dict(n=7 * P), ARG),               # n is h
    (dict(h=4 * P), ARG),               # h over a weight
])
def test_block_norm_refusals(lib, kw, want):
    assert norm(lib, **kw) == want


NORM_B = {**NORM, "dh": 9 * P, "dn": 10 * P, "dy": 11 * P, "dz": 12 * P, "dx": 13 * P, "dwp": 14 * P,
          "dr": 15 * P, "dwn": 16 * P, "ws": 17 * P, "wsb": 1 << 20}


def norm_bwd(lib, **kw):
    a = {**NORM_B, **kw}
    return lib.ckda_block_norm_bwd(a["y"], a["gate"], a["x"], a["wp"], a["r"], a["wn"], a["dh"], a["dn"],
                                   a["dy"], a["dz"], a["dx"], a["dwp"], a["dr"], a["dwn"], a["rows"], a["D"],
                                   ck._NormFlags(a["group"], a["act"], a["scale"], a["eps"]), a["dtype"],
                                   a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,want", NORM_BAD + [
    (dict(dy=None), NULL), (dict(dh=None, dn=None), NULL), (dict(dz=None), NULL),
    (dict(gate=None, act=0), ARG),                   # dgate without a gate
    (dict(group=0), ARG),                            # dpost_weight without a first norm
    (dict(dn=None), ARG),                            # dpre_weight without dn
    (dict(ws=None), WORKSPACE), (dict(wsb=8), WORKSPACE), (dict(ws=17 * P + 4), ALIGN),
    (dict(dwp=14 * P + 2), ALIGN), (dict(dx=13 * P + 8), ALIGN),
    (dict(dy=12 * P), ARG), (dict(dx=P + 64), ARG), (dict(dr=17 * P + 64), ARG), (dict(dwn=9 * P), ARG),
])
def test_block_norm_bwd_refusals(lib, kw, want):
    assert norm_bwd(lib, **kw) == want


def test_block_norm_workspace_query(lib):
    f = lib.ckda_block_norm_bwd_workspace_bytes
    assert 0 < f(4096, 2048, 128) < 1 << 27
    for bad in ((0, 8, 0), (4, 0, 0), (4, 9000, 0), (4, 64, 24)):
        assert f(*bad) == BAD


# ------------------------------------------------------------------------------------- the binding

def test_binding_refuses_before_the_library():
    t = torch.zeros(1, 4, 2, 16)
    g = torch.zeros(1, 4, 2)
    with pytest.raises(ValueError, match="CUDA"):
        ck.linattn_fwd_chunked(t, t, t, g)
    with pytest.raises(ValueError, match="CUDA"):
        ck.linattn_bwd_chunked(t, t, t, g, None, t)
    with pytest.raises(ValueError, match="CUDA"):
        ck.linattn_decode_step(t[:, 0], t[:, 0], t[:, 0], g[:, 0], torch.zeros(1, 2, 16, 16))
    with pytest.raises(ValueError, match="CUDA"):
        ck.block_norm(t)
    with pytest.raises(ValueError, match="CUDA"):
        ck.block_norm_bwd(t, t)
    with pytest.raises(TypeError, match="torch.Tensor"):
        ck.block_norm([1.0])
    with pytest.raises(ValueError, match="unsupported"):
        ck.linattn_fwd_workspace_bytes(1, 8, 1, 24, 16)
    with pytest.raises(ValueError, match="unsupported"):
        ck.linattn_bwd_workspace_bytes(1, 8, 3, 2, 16, 16)
    with pytest.raises(ValueError, match="unsupported"):
        ck.block_norm_bwd_workspace_bytes(4, 10000)
