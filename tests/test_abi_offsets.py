"""Host offsets of packed sequences, which the library reads on the host: those that do not lie there, or
are no offsets, are refused by the workspace queries too.  CPU only."""
import pytest
import torch

import gated_delta_rule_82_b200 as ck

QUERIES = [lambda cu: ck.linattn_fwd_workspace_bytes(1, 500, 2, 16, 32, cu),
           lambda cu: ck.linattn_bwd_workspace_bytes(1, 500, 2, 2, 16, 32, cu),
           lambda cu: ck.varlen_workspace_bytes(cu, 2, 16, 32, 64, torch.float32)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_delta_rule_82_b200 import build
    build.build()


@pytest.mark.parametrize("query", QUERIES)
@pytest.mark.parametrize("cu,error", [
    (torch.empty(3, dtype=torch.int32, device="meta"), ValueError),      # not host memory
    (torch.empty(0, dtype=torch.int32), ValueError), (torch.tensor([0], dtype=torch.int32), ValueError),
    ([0, 3, 9], TypeError),
])
def test_offsets_that_are_not_on_the_host(query, cu, error):
    with pytest.raises(error):
        query(cu)


@pytest.mark.parametrize("query", QUERIES)
def test_offsets_of_any_integer_type(query):
    want = query(torch.tensor([0, 300, 301, 900], dtype=torch.int32))
    wide = torch.tensor([0, 7, 300, 7, 301, 7, 900], dtype=torch.int64)[::2]     # (strided, too)
    assert query(wide) == want


@pytest.mark.parametrize("workspace,error", [
    (torch.empty(1, dtype=torch.uint8).expand(1 << 20), ValueError),      # a million elements of one byte
    (torch.empty(64, dtype=torch.uint8)[::2], ValueError),
    (torch.empty(64, dtype=torch.uint8, device="meta"), ValueError), (bytearray(64), TypeError),
])
def test_workspaces_that_are_not_what_they_count(workspace, error):
    with pytest.raises(error):
        ck._room(workspace, torch.device("cpu"))


def test_workspace_bytes():
    w = torch.empty(10, dtype=torch.float64)
    assert ck._room(w, torch.device("cpu")) == (w.data_ptr(), 80) and ck._room(None, torch.device("cpu")) == (None, 0)


def test_device_status_is_read_on_the_device_asked_for(monkeypatch):
    """(with a fake library and fake devices: the word belongs to the device that is current)"""
    current, seen = [0], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before = current[0]
            current[0] = current[0] if self.index is None else self.index

        def __exit__(self, *error):
            current[0] = self.before

    class Library:
        @staticmethod
        def ckda_last_device_status(stream, code):
            seen.append((current[0], stream))
            return 0

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(ck, "_load", lambda: Library)
    monkeypatch.setattr(ck, "_stream", lambda device: f"stream of {current[0] if device is None else device}")
    assert ck.last_device_status(2) == 0 and ck.last_device_status() == 0
    assert seen == [(2, "stream of 2"), (0, "stream of 0")] and current == [0]
