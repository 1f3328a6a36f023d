"""Block norms called from several host threads at once (GPU): rows of one width with one, two or three
weight vectors are the same kernel with different amounts of shared memory.  The calls are made from C++,
where nothing serialises them."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import gated_delta_rule_82_b200 as ck

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from gated_delta_rule_82_b200 import build
    build.build()


@pytest.mark.parametrize("D", [4096, 8192])
def test_threads_do_not_disturb_each_other(D, tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    so = str(tmp_path / "norm_threads.so")
    subprocess.run([gxx, "-O2", "-std=c++17", "-shared", "-fPIC", "-pthread", "-I",
                    os.path.join(os.path.dirname(HERE), "include"), os.path.join(HERE, "norm_threads.cpp"), "-o", so],
                   check=True)
    run = ctypes.CDLL(so).norm_threads
    P = ctypes.c_void_p
    run.restype = ctypes.c_long
    run.argtypes = [P, P, P, ctypes.POINTER(P), ctypes.POINTER(P), ctypes.c_longlong, ctypes.c_int, ctypes.c_int,
                    ctypes.c_long]
    torch.manual_seed(D)
    y = torch.randn(2, D, device="cuda", dtype=torch.bfloat16)
    w = 1 + 0.1 * torch.randn(D, device="cuda")
    h, n = (torch.full((3, 2, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    torch.cuda.synchronize()
    at = lambda x: (P * 3)(*(x[i].data_ptr() for i in range(3)))
    call = ctypes.cast(ck._load().ckda_block_norm, P)
    assert run(call, y.data_ptr(), w.data_ptr(), at(h), at(n), 2, D, 3, 20000) == 0
    torch.cuda.synchronize()
    for i, kw in enumerate((dict(), dict(post_group=D, post_weight=w), dict(post_group=D, post_weight=w,
                                                                            res_vector=w))):
        want = ck.block_norm(y, residual=y, pre_norm=True, pre_weight=w, eps=1e-5, **kw)
        assert torch.equal(h[i], want[0]) and torch.equal(n[i], want[1])
