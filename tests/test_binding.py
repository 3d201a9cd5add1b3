"""The ctypes binding's own conversions (no GPU, no library call)."""
import ctypes

import numpy as np
import pytest

from paged_kv_cache_458_b200 import pa


@pytest.mark.parametrize("x", [b"\0" * 64, "address", 4096.0, (ctypes.c_float * 4)(), np.zeros(4, np.float32),
                               np.zeros(4, np.float32).ctypes, [4096], ctypes.c_void_p(4096)],
                         ids=["bytes", "str", "float", "ctypes array", "ndarray", "ndarray.ctypes", "list", "c_void_p"])
def test_what_is_no_tensor_and_no_address_is_refused(x):
    """A host buffer passed by mistake must not travel to a kernel as a device address."""
    with pytest.raises(AttributeError):
        pa._ptr(x)


def test_tensors_addresses_and_none_pass():
    torch = pytest.importorskip("torch")
    t = torch.zeros(4)
    assert pa._ptr(t) == t.data_ptr() and pa._ptr(4096) == 4096 and pa._ptr(None) is None


@pytest.mark.parametrize("fast", [True, False])
def test_current_stream_with_and_without_the_fast_query(monkeypatch, fast):
    """Without a stream the call goes to torch's current one, also where torch lacks the calls that ask for its handle."""
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(pa, "_current_stream", None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: type("Stream", (), {"cuda_stream": 77})())
    if fast:
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 1000 + device, raising=False)
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 3, raising=False)
    else:
        monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
        monkeypatch.delattr(torch._C, "_cuda_getDevice", raising=False)
    for _ in range(2):
        assert pa._stream(None) == (1003 if fast else 77)
    assert pa._stream(5) == 5
