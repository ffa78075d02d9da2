"""Workspace.scratch on host tensors: which calls share a buffer."""
import pytest

torch = pytest.importorskip("torch")

import lossless_bit_weights_gb300 as w12


def test_streams_do_not_share_a_buffer():
    ws = w12.Workspace(torch.device("cpu"))
    a, b = ws.scratch(1000, None, 1), ws.scratch(1000, None, 2)
    assert a.data_ptr() != b.data_ptr()
    assert ws.scratch(500, None, 1).data_ptr() == a.data_ptr()
    assert ws.scratch(1000, None, 2).data_ptr() == b.data_ptr()
    assert ws.scratch(5000, None, 1).numel() >= 5000
    assert ws.scratch(1000, None, 2).data_ptr() == b.data_ptr()
