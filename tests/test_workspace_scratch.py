"""Workspace.scratch on host tensors: which calls share a buffer."""
import weakref

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


def test_outgrown_buffers_stay():
    """A graph may still write to them."""
    ws = w12.Workspace(torch.device("cpu"))
    grown, sizes = [], [300, 400, 5000, 5001, 100000, 99999, 1 << 20]
    for n in sizes:
        t = ws.scratch(n, None, 7)
        assert t.numel() >= n
        grown.append(weakref.ref(t))
        del t
    assert all(r() is not None for r in grown)
    kept = {r().data_ptr(): r().numel() for r in grown}
    assert sum(kept.values()) <= 2 * max(kept.values())
