"""Host-side rules of the serving binding that need no GPU: calls without rows,
import on a PyTorch without the CUDA bindings, workspaces sized for the tensors'
own device, integers that the C interface cannot hold."""

import contextlib
import ctypes
import os
import subprocess
import sys

import pytest
import torch

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


def test_workspace_is_sized_on_the_tensors_device(sf, monkeypatch):
    """The workspace goes by the number of SMs of the device that the call runs on, not of the current one."""
    from quantized_gemv_kv_b200 import serving
    at = [torch.device("cuda", 0)]
    asked = []

    @contextlib.contextmanager
    def device(d):
        at.append(torch.device(d))
        yield
        at.pop()

    def size(T, R, Hq, Hkv, d, out):
        asked.append(at[-1])
        ctypes.cast(out, ctypes.POINTER(ctypes.c_size_t))[0] = 4096
        return 0

    class Lib:
        sf_attn_paged_workspace_size = staticmethod(size)

    monkeypatch.setattr(serving, "_lib", Lib)
    monkeypatch.setattr(serving, "_dev", lambda t, name: None)
    monkeypatch.setattr(serving, "_same_device", lambda first, **t: torch.device("cuda", 1))
    monkeypatch.setattr(torch.cuda, "device", device)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    param = torch.zeros((4, 2, 16, 2), dtype=torch.float16)
    kv = serving.PagedKV(i32(4, 2, 16, 16), param, i32(4, 2, 16, 16), param)
    q = torch.zeros((3, 4, 128), dtype=torch.bfloat16)
    job = serving.PagedAttention(q, kv, i32(3), i32(2), i32(2, 4))
    assert job.workspace.numel() == 4096 and job.device == torch.device("cuda", 1)
    assert asked and all(d == torch.device("cuda", 1) for d in asked)
    asked.clear()
    assert serving.attn_paged_workspace_size(3, 2, 4, 2, 128, device="cuda:1") == 4096
    assert serving.attn_paged_workspace_size(3, 2, 4, 2, 128) == 4096
    assert asked == [torch.device("cuda", 1), torch.device("cuda", 0)]


@pytest.mark.parametrize("big", [2 ** 32 + 16, 2 ** 31, -(2 ** 32) + 16])
def test_integers_beyond_32_bits_are_refused(sf, big):
    """ctypes would cut them: a window of 2^32 + 16 would come out as one of 16 tokens."""
    from quantized_gemv_kv_b200 import serving
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    plan = dict(lens=i32(3), add=i32(3), block_table=i32(3, 4), free_list=i32(9), n_free=i32(1), page_size=16,
                max_rows=4)
    for name in ("page_size", "max_rows"):
        with pytest.raises(ValueError, match=name):
            sf.PagedPlan(**{**plan, name: big})
    with pytest.raises(ValueError, match="T must fit"):
        sf.attn_paged_workspace_size(big, 2, 4, 2, 128)
    param = torch.zeros((4, 2, 16, 2), dtype=torch.float16)
    with pytest.MonkeyPatch.context() as mp:
        mp.setattr(serving, "_dev", lambda t, name: None)
        kv = serving.PagedKV(i32(4, 2, 16, 16), param, i32(4, 2, 16, 16), param)
        with pytest.raises(ValueError, match="window must fit"):
            serving.PagedAttention(torch.zeros((3, 4, 128), dtype=torch.bfloat16), kv, i32(3), i32(2), i32(2, 4),
                                   window=big)
