"""What the binding takes as a device pointer: tensors, addresses and None.  Host objects that
ctypes would turn into host addresses are refused before the library is reached."""
import ctypes

import numpy as np
import pytest

from tree_speculative_verify_tv_gb300 import binding


class Recorder:
    """A library of which every function notes its arguments and succeeds."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append((name, a)) or 0


@pytest.fixture()
def lib(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(binding, "_lib", r)
    return r


def calls(x):
    yield lambda: binding.tv_qcache_write(1, 1, 1, 64, 1, 1, 16, 16, 16, x, 16, 64, 16, 16, stream=0)
    yield lambda: binding.tv_qcache_read(1, 1, 1, 64, 1, 1, 16, 16, 16, 16, x, 16, 16, 64, 16, stream=0)
    yield lambda: binding.tv_tree_attention(1, 1, 1, 1, 1, 64, 1, 16, 16, 16, 16, 16, x, 16, 16, 1.0,
                                            16, 0, 0, 16, stream=0)
    yield lambda: binding.tv_accept_greedy(1, 1, 1, 1, x, 16, 16, 16, 16, 16, 16, 16, 16, stream=0)


@pytest.mark.parametrize("x", [
    b"sixteen bytes...", bytearray(16), "text", ctypes.create_string_buffer(16), (ctypes.c_int32 * 4)(),
    ctypes.c_void_p(4096), np.zeros(4, np.int32), [0], object()], ids=lambda x: type(x).__name__)
def test_host_objects_are_not_device_pointers(lib, x):
    for call in calls(x):
        with pytest.raises((AttributeError, TypeError)):
            call()
    assert lib.calls == []


def test_tensors_addresses_and_none_are(lib):
    torch = pytest.importorskip("torch")
    t = torch.zeros(8)
    for x, seen in ((t, t.data_ptr()), (4096, 4096), (None, None)):
        del lib.calls[:]
        for call in calls(x):
            assert call() == 0
        assert len(lib.calls) == 4 and all(seen in a for _, a in lib.calls)
