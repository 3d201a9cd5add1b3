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
