"""Binding of the operators for a step of many requests: the paged 4-bit KV
cache (``sf_paged_plan``, ``sf_paged_append``, ``sf_attn_paged``) and the
per-request adapters (``sf_lora_add``).

Each operator is a class that checks its tensors, allocates what is missing
and builds the C arguments once; ``run()`` is then one library call on the
same buffers, so a step loop (or a captured CUDA graph) pays for neither.  The
function of the same name makes one such object and runs it.  Shapes, dtypes,
devices and strides are checked here, everything else by the library.
"""

from __future__ import annotations

import contextlib
import ctypes
import math
from dataclasses import dataclass

import torch

from . import _check, _dev, _i, _lib, _p, _sz

SF_F32, SF_BF16 = 0, 1
PLAN_OK, PLAN_LENGTH, PLAN_ROWS, PLAN_PAGES = range(4)
_DTYPES = {torch.float32: SF_F32, torch.bfloat16: SF_BF16}
_i64 = ctypes.c_int64


class _PagedKV(ctypes.Structure):
    _fields_ = [("k_codes", _p), ("k_param", _p), ("v_codes", _p), ("v_param", _p), ("num_pages", _i), ("Hkv", _i),
                ("page_size", _i), ("d", _i), ("page_rows", _i64)]


class _PlanArgs(ctypes.Structure):
    _fields_ = [("len", _p), ("keep", _p), ("add", _p), ("block_table", _p), ("free_list", _p), ("n_free", _p),
                ("len_out", _p), ("n_free_out", _p), ("cu_rows", _p), ("slots", _p), ("positions", _p),
                ("row_request", _p), ("status", _p), ("table_stride", _i64), ("R", _i), ("page_size", _i),
                ("max_pages", _i), ("max_rows", _i), ("free_cap", _i)]


class _AppendArgs(ctypes.Structure):
    _fields_ = [("kv", ctypes.POINTER(_PagedKV)), ("k", _p), ("v", _p), ("q", _p), ("q_out", _p), ("k_val", _p),
                ("v_val", _p), ("slots", _p), ("positions", _p), ("k_stride", _i64), ("v_stride", _i64),
                ("q_stride", _i64), ("q_out_stride", _i64), ("theta", ctypes.c_double), ("T", _i), ("Hq", _i),
                ("src_type", _i)]


class _AttnArgs(ctypes.Structure):
    _fields_ = [("kv", ctypes.POINTER(_PagedKV)), ("q", _p), ("cu_rows", _p), ("len", _p), ("block_table", _p),
                ("out", _p), ("workspace", _p), ("ws_bytes", _sz), ("q_stride", _i64), ("out_stride", _i64),
                ("table_stride", _i64), ("scale", ctypes.c_float), ("T", _i), ("R", _i), ("Hq", _i),
                ("max_pages", _i), ("window", _i), ("out_type", _i)]


class _LoraArgs(ctypes.Structure):
    _fields_ = [("x", _p), ("A", _p), ("B", _p), ("scale", _p), ("ids", _p), ("row_of", _p), ("y", _p), ("out", _p),
                ("x_stride", _i64), ("y_stride", _i64), ("out_stride", _i64), ("T", _i), ("n_ids", _i),
                ("n_adapters", _i), ("K", _i), ("N", _i), ("rank", _i)]


# ---- argument checks -----------------------------------------------------------


def _same_device(first: str, **tensors) -> torch.device:
    """The one device of the given tensors (None entries left out)."""
    dev = tensors[first].device
    for name, t in tensors.items():
        if t is None:
            continue
        _dev(t, name)
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, {first} on {dev}")
    return dev


def _fit(**values: int) -> None:
    """Whole numbers that go to the library as C ints, which ctypes would cut
    to 32 bits without a word."""
    for name, v in values.items():
        if not -2 ** 31 <= v < 2 ** 31:
            raise ValueError(f"{name} must fit 32 bits, it is {v}")


def _ints(name: str, t: torch.Tensor, n: int | None = None) -> None:
    """A contiguous int32 vector, of n entries where n is given."""
    if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 vector")
    if n is not None and t.numel() != n:
        raise ValueError(f"{name} must have {n} entries, it has {t.numel()}")


def _matrix(name: str, t: torch.Tensor, dtype, shape) -> int:
    """A 2-D or 3-D tensor whose rows are contiguous and apart from one
    another; returns the row stride in elements."""
    dtypes = dtype if isinstance(dtype, tuple) else (dtype,)
    if t.dtype not in dtypes or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {' or '.join(str(x) for x in dtypes)} of shape {tuple(shape)}, it is "
                         f"{t.dtype} of {tuple(t.shape)}")
    row = math.prod(shape[1:])
    inner = 1
    for size, stride in zip(reversed(shape[1:]), reversed(t.stride()[1:])):
        if size > 1 and stride != inner:
            raise ValueError(f"{name}'s rows must be contiguous")
        inner *= size
    if shape[0] > 1:
        if t.stride(0) < row:
            raise ValueError(f"{name}'s rows overlap")
        return t.stride(0)
    return -(-row // 8) * 8  # one row: any stride does


def _table(t: torch.Tensor, R: int) -> int:
    if t.dtype != torch.int32 or t.dim() != 2 or t.shape[0] != R or t.shape[1] < 1 or \
            (t.shape[1] > 1 and t.stride(1) != 1) or (R > 1 and t.stride(0) < t.shape[1]):
        raise ValueError(f"block_table must be int32 [{R}][max_pages] with contiguous rows")
    return t.stride(0) if R > 1 else t.shape[1]


class _Job:
    """One library call on fixed buffers."""

    _call = None

    def _bind(self, args: ctypes.Structure, device: torch.device, keep) -> None:
        self._args = args
        self._ref = ctypes.byref(args)
        self._keep = keep          # the tensors whose addresses the arguments hold
        self.device = device
        self._index = device.index

    def run(self, stream: torch.cuda.Stream | None = None) -> None:
        """Enqueues the call on ``stream`` (default: the current stream of
        the tensors' device).  What the object allocated belongs to the
        stream that was current then: order ``stream`` behind it, and keep
        the object until the call's work has ended."""
        if stream is None:
            raw = torch._C._cuda_getCurrentRawStream(self._index)  # the current stream, without a Stream object
        elif stream.device != self.device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {self.device}")
        else:
            raw = stream.cuda_stream
        if torch._C._cuda_getDevice() == self._index:
            status = self._call(self._ref, raw)
        else:
            with torch.cuda.device(self.device):
                status = self._call(self._ref, raw)
        if status:
            _check(status)


def _on(stream: torch.cuda.Stream | None):
    """What is allocated inside belongs to the stream that the call runs on."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


# ---- the pool ------------------------------------------------------------------


@dataclass
class PagedKV:
    """A pool of pages of 4-bit K and V (``sf_paged_kv``).  ``*_codes`` int32
    [num_pages][Hkv][page_size][d/8]; ``*_param`` float16 [num_pages][Hkv]
    [page_size][2], a token-head's scale and zero point.  Pages may be apart
    from one another (a slice of a larger allocation), by the same number of
    token-heads in all four tensors."""
    k_codes: torch.Tensor
    k_param: torch.Tensor
    v_codes: torch.Tensor
    v_param: torch.Tensor

    def __post_init__(self):
        c = self.k_codes
        if c.dim() != 4 or c.dtype != torch.int32:
            raise ValueError("k_codes must be int32 [num_pages][Hkv][page_size][d/8]")
        self.num_pages, self.Hkv, self.page_size, words = c.shape
        self.d = words * 8
        self.device = _same_device("k_codes", k_codes=c, k_param=self.k_param, v_codes=self.v_codes,
                                   v_param=self.v_param)
        rows = None
        for name, dtype, last in (("k_codes", torch.int32, words), ("v_codes", torch.int32, words),
                                  ("k_param", torch.float16, 2), ("v_param", torch.float16, 2)):
            t = getattr(self, name)
            s = _matrix(name, t, dtype, (self.num_pages, self.Hkv, self.page_size, last))
            if self.num_pages == 1:
                continue
            if s % last or (rows is not None and s // last != rows):
                raise ValueError("the four arrays must have the same number of token-heads from page to page")
            rows = s // last
        _fit(num_pages=self.num_pages, Hkv=self.Hkv, page_size=self.page_size, d=self.d)
        self._c = _PagedKV(self.k_codes.data_ptr(), self.k_param.data_ptr(), self.v_codes.data_ptr(),
                           self.v_param.data_ptr(), self.num_pages, self.Hkv, self.page_size, self.d, rows or 0)

    @classmethod
    def empty(cls, num_pages: int, Hkv: int, page_size: int, d: int, device="cuda") -> "PagedKV":
        """A pool whose tokens do not exist yet (their scales are 0)."""
        def codes():
            return torch.zeros((num_pages, Hkv, page_size, d // 8), dtype=torch.int32, device=device)

        def param():
            return torch.zeros((num_pages, Hkv, page_size, 2), dtype=torch.float16, device=device)

        return cls(codes(), param(), codes(), param())


# ---- sf_paged_plan ---------------------------------------------------------------


class PagedPlan(_Job):
    """``sf_paged_plan``: from ``lens`` (int32 [R], tokens held), ``keep`` (int32
    [R] or None: all) and ``add`` (int32 [R], rows of this step) the pages, slots
    and positions of a step.  ``block_table`` (int32 [R][max_pages]) and
    ``free_list`` (int32) are updated in place; ``lens_out`` and ``n_free_out``
    default to ``lens`` and ``n_free`` themselves.  Outputs, allocated here:
    ``cu_rows`` [R + 1], ``slots``, ``positions``, ``row_request`` [max_rows] and
    ``status`` [1] (PLAN_OK, or the reason why nothing changed)."""

    _call = _lib.sf_paged_plan

    def __init__(self, lens: torch.Tensor, add: torch.Tensor, block_table: torch.Tensor, free_list: torch.Tensor,
                 n_free: torch.Tensor, page_size: int, max_rows: int, keep: torch.Tensor | None = None,
                 lens_out: torch.Tensor | None = None, n_free_out: torch.Tensor | None = None):
        lens_out = lens if lens_out is None else lens_out
        n_free_out = n_free if n_free_out is None else n_free_out
        _ints("lens", lens)
        R = lens.numel()
        for name, t in (("add", add), ("keep", keep), ("lens_out", lens_out)):
            if t is not None:
                _ints(name, t, R)
        _ints("free_list", free_list)
        _ints("n_free", n_free, 1)
        _ints("n_free_out", n_free_out, 1)
        stride = _table(block_table, R)
        _fit(R=R, page_size=page_size, max_pages=block_table.shape[1], max_rows=max_rows, free_cap=free_list.numel())
        if max_rows < 1:
            raise ValueError("max_rows must be >= 1")
        dev = _same_device("lens", lens=lens, add=add, keep=keep, lens_out=lens_out, block_table=block_table,
                           free_list=free_list, n_free=n_free, n_free_out=n_free_out)
        self.lens_out, self.n_free_out = lens_out, n_free_out
        self.block_table, self.free_list = block_table, free_list
        self.cu_rows = torch.empty(R + 1, dtype=torch.int32, device=dev)
        self.slots, self.positions, self.row_request = (
            torch.empty(max_rows, dtype=torch.int32, device=dev) for _ in range(3))
        self.status = torch.empty(1, dtype=torch.int32, device=dev)
        a = _PlanArgs(lens.data_ptr(), keep.data_ptr() if keep is not None else None, add.data_ptr(),
                      block_table.data_ptr(), free_list.data_ptr(), n_free.data_ptr(), lens_out.data_ptr(),
                      n_free_out.data_ptr(), self.cu_rows.data_ptr(), self.slots.data_ptr(),
                      self.positions.data_ptr(), self.row_request.data_ptr(), self.status.data_ptr(), stride, R,
                      page_size, block_table.shape[1], max_rows, free_list.numel())
        self._bind(a, dev, (lens, add, keep, n_free))


def paged_plan(lens, add, block_table, free_list, n_free, page_size, max_rows, keep=None, lens_out=None,
               n_free_out=None, stream=None) -> PagedPlan:
    """One ``sf_paged_plan`` call; returns the ``PagedPlan`` with its outputs."""
    with _on(stream):
        job = PagedPlan(lens, add, block_table, free_list, n_free, page_size, max_rows, keep, lens_out, n_free_out)
        job.run(stream)
    return job


# ---- sf_paged_append --------------------------------------------------------------


class PagedAppend(_Job):
    """``sf_paged_append``: rows k and v (fp32 or bf16 [T][Hkv][d], rows may be
    strided) quantized to 4 bits into their ``slots`` (int32 [T]).  With theta >
    0 the keys, and q [T][Hq][d] into ``q_out`` (bf16, allocated when None), are
    rotated to ``positions`` (int32 [T]) first.  ``k_val`` / ``v_val`` (bf16
    [T][Hkv][d]) receive the values the pages then hold."""

    _call = _lib.sf_paged_append

    def __init__(self, kv: PagedKV, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
                 positions: torch.Tensor | None = None, theta: float = 0.0, q: torch.Tensor | None = None,
                 q_out: torch.Tensor | None = None, k_val: torch.Tensor | None = None,
                 v_val: torch.Tensor | None = None):
        if k.dim() != 3 or k.dtype not in _DTYPES:
            raise ValueError("k must be float32 or bfloat16 [T][Hkv][d]")
        T, d = k.shape[0], kv.d
        ks = _matrix("k", k, k.dtype, (T, kv.Hkv, d))
        vs = _matrix("v", v, k.dtype, (T, kv.Hkv, d))
        _ints("slots", slots, T)
        Hq = qs = qos = 0
        if theta > 0.0:
            if positions is None:
                raise ValueError("the rotation needs positions")
            _ints("positions", positions, T)
        elif q is not None or q_out is not None:
            raise ValueError("q is only rotated: it needs theta > 0")
        if q is not None:
            if q.dim() != 3:
                raise ValueError("q must be [T][Hq][d]")
            Hq = q.shape[1]
            qs = _matrix("q", q, k.dtype, (T, Hq, d))
            if q_out is None:
                q_out = torch.empty((T, Hq, d), dtype=torch.bfloat16, device=q.device)
            qos = _matrix("q_out", q_out, torch.bfloat16, (T, Hq, d))
        elif q_out is not None:
            raise ValueError("q_out needs q")
        _fit(T=T, Hq=Hq)
        for name, t in (("k_val", k_val), ("v_val", v_val)):
            if t is not None and (t.dtype != torch.bfloat16 or t.shape != (T, kv.Hkv, d) or not t.is_contiguous()):
                raise ValueError(f"{name} must be contiguous bfloat16 {(T, kv.Hkv, d)}")
        dev = _same_device("k_codes", k_codes=kv.k_codes, k=k, v=v, slots=slots, positions=positions, q=q,
                           q_out=q_out, k_val=k_val, v_val=v_val)
        self.q_out, self.k_val, self.v_val = q_out, k_val, v_val

        def ptr(t):
            return t.data_ptr() if t is not None else None

        a = _AppendArgs(ctypes.pointer(kv._c), k.data_ptr(), v.data_ptr(), ptr(q), ptr(q_out), ptr(k_val),
                        ptr(v_val), slots.data_ptr(), ptr(positions), ks, vs, qs, qos, theta, T, Hq, _DTYPES[k.dtype])
        self._bind(a, dev, (kv, k, v, slots, positions, q))


def paged_append(kv, k, v, slots, positions=None, theta=0.0, q=None, q_out=None, k_val=None, v_val=None,
                 stream=None) -> torch.Tensor | None:
    """One ``sf_paged_append`` call; returns q_out (None without q)."""
    with _on(stream):
        job = PagedAppend(kv, k, v, slots, positions, theta, q, q_out, k_val, v_val)
        job.run(stream)
    return job.q_out


# ---- sf_attn_paged ----------------------------------------------------------------


def attn_paged_workspace_size(T: int, R: int, Hq: int, Hkv: int, d: int, device=None) -> int:
    """Bytes of workspace that ``attn_paged`` needs on ``device`` (default:
    the current one); it goes by the device's number of SMs."""
    _fit(T=T, R=R, Hq=Hq, Hkv=Hkv, d=d)
    out = _sz()
    with contextlib.nullcontext() if device is None else torch.cuda.device(device):
        _check(_lib.sf_attn_paged_workspace_size(T, R, Hq, Hkv, d, ctypes.byref(out)))
    return out.value


class PagedAttention(_Job):
    """``sf_attn_paged``: q (bf16 [T][Hq][d], rows may be strided) over the
    pages of each row's request, into ``out`` (fp32 or bf16 [T][Hq][d], fp32 and
    zero-filled when None; rows behind the last request stay as they are).
    cu_rows int32 [R + 1], lens int32 [R] (this step's rows included),
    block_table int32 [R][max_pages]; scale defaults to 1/sqrt(d); window 0 means
    all tokens.  ``workspace`` (uint8, allocated when None) belongs to the call
    while it runs: calls that may overlap need one each."""

    _call = _lib.sf_attn_paged

    def __init__(self, q: torch.Tensor, kv: PagedKV, cu_rows: torch.Tensor, lens: torch.Tensor,
                 block_table: torch.Tensor, out: torch.Tensor | None = None, scale: float | None = None,
                 window: int = 0, workspace: torch.Tensor | None = None):
        if q.dim() != 3:
            raise ValueError("q must be bfloat16 [T][Hq][d]")
        T, Hq, d = q.shape
        if d != kv.d:
            raise ValueError(f"q has head dim {d}, the cache {kv.d}")
        qs = _matrix("q", q, torch.bfloat16, (T, Hq, d))
        _ints("lens", lens)
        R = lens.numel()
        _ints("cu_rows", cu_rows, R + 1)
        stride = _table(block_table, R)
        _fit(T=T, R=R, Hq=Hq, max_pages=block_table.shape[1], window=window)
        if out is None:
            out = torch.zeros((T, Hq, d), dtype=torch.float32, device=q.device)
        os_ = _matrix("out", out, tuple(_DTYPES), (T, Hq, d))
        dev = _same_device("q", q=q, k_codes=kv.k_codes, cu_rows=cu_rows, lens=lens, block_table=block_table,
                           out=out, workspace=workspace)
        need = attn_paged_workspace_size(T, R, Hq, kv.Hkv, d, device=dev)
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        self.out, self.workspace = out, workspace
        a = _AttnArgs(ctypes.pointer(kv._c), q.data_ptr(), cu_rows.data_ptr(), lens.data_ptr(),
                      block_table.data_ptr(), out.data_ptr(), workspace.data_ptr(),
                      workspace.numel() * workspace.element_size(), qs, os_, stride,
                      1.0 / math.sqrt(d) if scale is None else scale, T, R, Hq, block_table.shape[1], window,
                      _DTYPES[out.dtype])
        self._bind(a, dev, (q, kv, cu_rows, lens, block_table))


def attn_paged(q, kv, cu_rows, lens, block_table, out=None, scale=None, window=0, workspace=None,
               stream=None) -> torch.Tensor:
    """One ``sf_attn_paged`` call; returns out."""
    with _on(stream):
        job = PagedAttention(q, kv, cu_rows, lens, block_table, out, scale, window, workspace)
        job.run(stream)
    return job.out


# ---- sf_lora_add ------------------------------------------------------------------


class LoraAdd(_Job):
    """``sf_lora_add``: out[t] = y[t] + scale[a] B[a] (A[a] x[t]) with a =
    ids[row_of[t]] (row_of None: ids[t]).  x bf16 [T][K], A bf16 [n][rank][K], B
    bf16 [n][N][rank], scale fp32 [n], ids int32 (outside [0, n): no adapter), y
    fp32 [T][N] (None: 0), out fp32 [T][N] (None: y itself, or a new tensor
    without y)."""

    _call = _lib.sf_lora_add

    def __init__(self, x: torch.Tensor, A: torch.Tensor, B: torch.Tensor, scale: torch.Tensor, ids: torch.Tensor,
                 out: torch.Tensor | None = None, y: torch.Tensor | None = None,
                 row_of: torch.Tensor | None = None):
        if x.dim() != 2 or A.dim() != 3 or B.dim() != 3:
            raise ValueError("x must be [T][K], A [n][rank][K] and B [n][N][rank]")
        T, K = x.shape
        n, rank, _ = A.shape
        N = B.shape[1]
        _fit(T=T, n_ids=ids.numel(), n_adapters=n, K=K, N=N, rank=rank)
        xs = _matrix("x", x, torch.bfloat16, (T, K))
        for name, t, shape in (("A", A, (n, rank, K)), ("B", B, (n, N, rank))):
            if t.dtype != torch.bfloat16 or tuple(t.shape) != shape or not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous bfloat16 of shape {shape}, it is {t.dtype} of "
                                 f"{tuple(t.shape)}")
        if scale.dtype != torch.float32 or tuple(scale.shape) != (n,) or not scale.is_contiguous():
            raise ValueError(f"scale must be contiguous float32 with {n} entries")
        _ints("ids", ids)
        if row_of is not None:
            _ints("row_of", row_of, T)
        ys = 0
        if y is not None:
            ys = _matrix("y", y, torch.float32, (T, N))
        if out is None:
            out = y if y is not None else torch.empty((T, N), dtype=torch.float32, device=x.device)
        os_ = _matrix("out", out, torch.float32, (T, N))
        dev = _same_device("x", x=x, A=A, B=B, scale=scale, ids=ids, row_of=row_of, y=y, out=out)
        self.out = out
        a = _LoraArgs(x.data_ptr(), A.data_ptr(), B.data_ptr(), scale.data_ptr(), ids.data_ptr(),
                      row_of.data_ptr() if row_of is not None else None, y.data_ptr() if y is not None else None,
                      out.data_ptr(), xs, ys, os_, T, ids.numel(), n, K, N, rank)
        self._bind(a, dev, (x, A, B, scale, ids, row_of, y))


def lora_add(x, A, B, scale, ids, out=None, y=None, row_of=None, stream=None) -> torch.Tensor:
    """One ``sf_lora_add`` call; returns out."""
    with _on(stream):
        job = LoraAdd(x, A, B, scale, ids, out, y, row_of)
        job.run(stream)
    return job.out
