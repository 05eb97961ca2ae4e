"""Host-side rules of the serving binding that need no GPU: calls without rows,
import on a PyTorch without the CUDA bindings, workspaces sized for the tensors'
own device."""

import ctypes
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


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


def test_import_without_torch_cuda_bindings():
    """A PyTorch built without CUDA lacks the raw bindings: the package imports, and only calls need them."""
    code = ("import torch\n"
            "for n in ('_cuda_getCurrentRawStream', '_cuda_getDevice'):\n"
            "    if hasattr(torch._C, n): delattr(torch._C, n)\n"
            "import quantized_gemv_kv_b200 as sf\n"
            "assert sf.attn_paged_workspace_size(3, 2, 4, 2, 128) > 0\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
