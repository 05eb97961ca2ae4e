"""Host-side rules of the serving binding that need no GPU: calls without rows,
import on a PyTorch without the CUDA bindings, workspaces sized for the tensors'
own device."""

import ctypes

import pytest


@pytest.fixture(scope="module")
def sf():
    import quantized_gemv_kv_b200 as sf
    return sf


def test_append_without_rows_needs_no_pointers(sf):
    """T = 0 is nothing to do, also with queries: tensors without elements have no address."""
    from quantized_gemv_kv_b200.serving import _AppendArgs, _PagedKV
    kv = _PagedKV(256, 256, 256, 256, 8, 2, 16, 128, 0)
    for theta, Hq in ((0.0, 0), (1e4, 0), (1e4, 4)):
        args = _AppendArgs(ctypes.pointer(kv), None, None, None, None, None, None, None, None, 256, 256, 512, 512, theta,
                           0, Hq, 0)
        assert sf._lib.sf_paged_append(ctypes.byref(args), None) == sf.SF_OK
    args = _AppendArgs(ctypes.pointer(kv), None, None, None, None, None, None, None, None, 256, 256, 512, 512, 0.0, 0, 4, 0)
    assert sf._lib.sf_paged_append(ctypes.byref(args), None) == sf.SF_EINVAL   # queries without a rotation all the same
