"""The entry points for a step of many requests refuse bad arguments on the
host, with a status and a message, before any device work (so this runs
without a GPU); the binding refuses tensors of the wrong shape, type or device
before it reaches the library."""

import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def sf():
    import quantized_gemv_kv_b200 as sf
    return sf


def _err(sf):
    buf = ctypes.create_string_buffer(512)
    sf._lib.sf_last_error(buf, len(buf))
    return buf.value.decode()


def _refused(sf, call, args, match):
    assert call(ctypes.byref(args), None) == sf.SF_EINVAL
    assert match in _err(sf), _err(sf)


def _kv(**kw):
    from quantized_gemv_kv_b200.serving import _PagedKV
    a = dict(k_codes=256, k_param=256, v_codes=256, v_param=256, num_pages=8, Hkv=2, page_size=16, d=128, page_rows=0)
    a.update(kw)
    return _PagedKV(*a.values())


BAD_KV = [(dict(k_codes=None), "null"), (dict(v_param=260), "aligned"), (dict(d=96), "d must be"),
          (dict(page_size=24), "page_size"), (dict(page_size=8), "page_size"), (dict(page_size=512), "page_size"),
          (dict(Hkv=0), "Hkv"), (dict(num_pages=0), "num_pages"), (dict(num_pages=1 << 27), "num_pages"),
          (dict(page_rows=31), "page_rows"), (dict(page_rows=34), "page_rows")]


def test_plan_refusals(sf):
    from quantized_gemv_kv_b200.serving import _PlanArgs
    good = dict(len=256, keep=None, add=256, block_table=256, free_list=256, n_free=256, len_out=256, n_free_out=256,
                cu_rows=256, slots=256, positions=256, row_request=256, status=256, table_stride=4, R=2, page_size=16,
                max_pages=4, max_rows=8, free_cap=8)
    for bad, match in ((dict(len=None), "null"), (dict(status=None), "null"), (dict(R=0), "R must"),
                       (dict(R=8193), "R must"), (dict(page_size=20), "page_size"), (dict(max_pages=0), "max_pages"),
                       (dict(max_pages=1 << 27, table_stride=1 << 27), "max_pages"), (dict(table_stride=3), "stride"),
                       (dict(max_rows=0), "max_rows"), (dict(free_cap=0), "free_cap"),
                       (dict(max_rows=2 ** 30 + 1), "max_rows"), (dict(free_cap=2 ** 31 - 1), "free_cap")):
        _refused(sf, sf._lib.sf_paged_plan, _PlanArgs(*{**good, **bad}.values()), match)
    assert sf._lib.sf_paged_plan(None, None) == sf.SF_EINVAL


def test_append_refusals(sf):
    from quantized_gemv_kv_b200.serving import _AppendArgs

    def args(kv=None, **kw):
        a = dict(kv=ctypes.pointer(kv if kv is not None else _kv()), k=256, v=256, q=256, q_out=256, k_val=None,
                 v_val=None, slots=256, positions=256, k_stride=256, v_stride=256, q_stride=512, q_out_stride=512,
                 theta=1e4, T=3, Hq=4, src_type=0)
        a.update(kw)
        return _AppendArgs(*a.values())

    call = sf._lib.sf_paged_append
    for bad, match in BAD_KV:
        _refused(sf, call, args(_kv(**bad)), match)
    for bad, match in ((dict(T=-1), "T must"), (dict(src_type=2), "src_type"), (dict(Hq=-1), "Hq"),
                       (dict(Hq=2000), "Hq"), (dict(theta=-1.0), "theta"), (dict(theta=float("nan")), "theta"),
                       (dict(theta=0.0), "theta"), (dict(q=None), "Hq > 0"), (dict(q_out=None), "Hq > 0"),
                       (dict(slots=None), "null"), (dict(positions=None), "positions"), (dict(k_stride=255), "stride"),
                       (dict(q_stride=511), "stride"), (dict(k=264), "aligned"), (dict(v_stride=258), "aligned"),
                       (dict(q_out=260), "aligned"), (dict(k_val=258), "aligned")):
        _refused(sf, call, args(**bad), match)
    assert call(None, None) == sf.SF_EINVAL
    assert call(ctypes.byref(args(T=0)), None) == sf.SF_OK       # nothing to do


def test_attention_refusals(sf):
    from quantized_gemv_kv_b200.serving import _AttnArgs

    def args(kv=None, **kw):
        a = dict(kv=ctypes.pointer(kv if kv is not None else _kv()), q=256, cu_rows=256, len=256, block_table=256,
                 out=256, workspace=256, ws_bytes=1 << 40, q_stride=512, out_stride=512, table_stride=4, scale=0.1,
                 T=3, R=2, Hq=4, max_pages=4, window=0, out_type=0)
        a.update(kw)
        return _AttnArgs(*a.values())

    call = sf._lib.sf_attn_paged
    for bad, match in BAD_KV:
        _refused(sf, call, args(_kv(**bad)), match)
    for bad, match in ((dict(T=-1), "T >= 0"), (dict(R=0), "R in"), (dict(R=8193), "R in"), (dict(Hq=5), "Hq"),
                       (dict(Hq=0), "Hq"), (dict(Hq=130), "Hq"), (dict(max_pages=0), "max_pages"),
                       (dict(table_stride=3), "stride"), (dict(window=-1), "window"),
                       (dict(scale=float("inf")), "scale"), (dict(out_type=7), "out_type"), (dict(q=None), "null"),
                       (dict(workspace=None), "null"), (dict(q_stride=504), "stride"), (dict(q=264), "aligned"),
                       (dict(q_stride=516), "aligned"), (dict(out_stride=514), "aligned"),
                       (dict(workspace=264), "aligned"), (dict(ws_bytes=0), "too small"), (dict(T=1 << 25), "2^26")):
        _refused(sf, call, args(**bad), match)
    assert call(None, None) == sf.SF_EINVAL
    assert call(ctypes.byref(args(T=0)), None) == sf.SF_OK
    out = ctypes.c_size_t()
    assert sf._lib.sf_attn_paged_workspace_size(3, 2, 4, 2, 96, ctypes.byref(out)) == sf.SF_EINVAL
    assert sf._lib.sf_attn_paged_workspace_size(3, 2, 4, 2, 128, None) == sf.SF_EINVAL
    assert sf._lib.sf_attn_paged_workspace_size(3, 2, 4, 2, 128, ctypes.byref(out)) == sf.SF_OK and out.value > 0


def test_lora_refusals(sf):
    from quantized_gemv_kv_b200.serving import _LoraArgs

    def args(**kw):
        a = dict(x=256, A=256, B=256, scale=256, ids=256, row_of=None, y=256, out=256, x_stride=64, y_stride=40,
                 out_stride=40, T=3, n_ids=3, n_adapters=2, K=64, N=40, rank=16)
        a.update(kw)
        return _LoraArgs(*a.values())

    call = sf._lib.sf_lora_add
    for bad, match in ((dict(T=-1), "T >= 0"), (dict(n_ids=-1), "n_ids"), (dict(n_adapters=0), "n_adapters"),
                       (dict(N=0), "N >= 1"), (dict(K=0), "K must"), (dict(K=60), "K must"), (dict(rank=0), "rank"),
                       (dict(N=2 ** 30 + 1), "N <= 2^30"), (dict(K=2 ** 31 - 8), "K must"),
                       (dict(rank=12), "rank"), (dict(rank=136), "rank"), (dict(x=None), "null"),
                       (dict(ids=None), "null"), (dict(scale=None), "null"), (dict(x_stride=56), "stride"),
                       (dict(y_stride=39), "stride"), (dict(out_stride=39), "stride"), (dict(out_stride=44), "another row stride"), (dict(A=264), "aligned"),
                       (dict(x_stride=68), "aligned"), (dict(x=258), "aligned")):
        _refused(sf, call, args(**bad), match)
    assert call(None, None) == sf.SF_EINVAL
    assert call(ctypes.byref(args(T=0)), None) == sf.SF_OK


def test_binding_refuses_wrong_tensors(sf):
    """Everything is checked before the device is touched: CPU tensors get as
    far as the device check when their shapes are right, and no further."""
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        sf.PagedKV.empty(2, 2, 16, 128, device="cpu")
    with pytest.raises(ValueError, match="k_codes must be"):
        sf.PagedKV(i32(2, 16, 16), i32(1), i32(1), i32(1))
    plan = dict(lens=i32(3), add=i32(3), block_table=i32(3, 4), free_list=i32(9), n_free=i32(1), page_size=16,
                max_rows=4)
    for bad, match in ((dict(add=i32(2)), "add must have 3"), (dict(lens=i32(3).long()), "lens must be"),
                       (dict(keep=i32(4)), "keep must"), (dict(block_table=i32(2, 4)), "block_table"),
                       (dict(block_table=i32(4, 3).t()), "block_table"), (dict(n_free=i32(2)), "n_free"),
                       (dict(max_rows=0), "max_rows"), (dict(), "CUDA")):
        with pytest.raises(ValueError, match=match):
            sf.PagedPlan(**{**plan, **bad})
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    lora = dict(x=bf(3, 16), A=bf(2, 8, 16), B=bf(2, 5, 8), scale=torch.zeros(2), ids=i32(3))
    for bad, match in ((dict(x=torch.zeros(3, 16)), "x must be"), (dict(A=bf(2, 8, 8)), "A must be"),
                       (dict(B=bf(1, 5, 8)), "B must be"), (dict(scale=torch.zeros(3)), "scale"),
                       (dict(y=torch.zeros(3, 6)), "y must be"), (dict(out=bf(3, 5)), "out must be"),
                       (dict(row_of=i32(2)), "row_of"), (dict(x=bf(16, 3).t()), "contiguous"), (dict(), "CUDA")):
        with pytest.raises(ValueError, match=match):
            sf.LoraAdd(**{**lora, **bad})
