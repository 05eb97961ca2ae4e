"""A step of many requests over a paged 4-bit KV cache, and per-request
low-rank adapters (oracle; test infrastructure).

S1  pages: a request's tokens lie in pages of P tokens, page j of request i is
    table[i][j]; token t has slot table[i][t // P] * P + t % P.
S2  plan: request i keeps keep_i of its len_i tokens and adds add_i.  The free
    list is a stack; first every page behind ceil((keep + add) / P) is pushed
    (requests in order, a request's pages in order), then the missing pages
    are popped (same order).  A page outside [0, 2^31 / P) gives slots of -1.  Lengths out of range, more rows than there is
    room for, or too few pages: nothing changes and the step has no rows.
S3  a token-head's K or V row is quantized as one group with b = 4 (Q1-Q4 of
    the nested quantizer); its value is scale (code - zero).
S4  row j of a request with n rows in the step and len tokens is the token at
    p = len - n + j; it attends to tokens [max(0, p - window + 1), p] (all from 0
    without a window) that lie in pages of the pool, fp64 softmax; a row
    without tokens gives zeros.
S5  adapters: y_t + scale_a B_a (A_a x_t), fp64, a the adapter of row t.
"""

from __future__ import annotations

import math

import numpy as np

from .quant import quantize_nested

PLAN_OK, PLAN_LENGTH, PLAN_ROWS, PLAN_PAGES = range(4)


def plan(lens, keep, add, table, free, free_cap: int, P: int, max_rows: int) -> dict:
    """S2 with plain lists.  table: [R][max_pages]; free: the free list's
    live part.  Returns the new lens, table and free list, cu_rows, the per-row
    slots, positions and requests, and the status."""
    R, room = len(lens), len(table[0]) * P
    table = [list(r) for r in table]
    free = list(free)

    def refuse(status):
        return dict(status=status, lens=list(lens), table=table, free=free, cu=[0] * (R + 1), slots=[-1] * max_rows,
                    positions=[0] * max_rows, request=[-1] * max_rows)

    for n, k, a in zip(lens, keep, add):
        if n < 0 or n > room or k < 0 or k > n or a < 0 or k + a > room:
            return refuse(PLAN_LENGTH)
    if sum(add) > max_rows:
        return refuse(PLAN_ROWS)
    have = [math.ceil(n / P) for n in lens]
    want = [math.ceil((k + a) / P) for k, a in zip(keep, add)]
    stack = free + [table[i][j] for i in range(R) for j in range(want[i], have[i])]
    if len(stack) > free_cap or sum(max(0, w - h) for w, h in zip(want, have)) > len(stack):
        return refuse(PLAN_PAGES)
    for i in range(R):
        for j in range(have[i], want[i]):
            table[i][j] = stack.pop()
    cu, slots, positions, request = [0], [], [], []
    for i in range(R):
        cu.append(cu[-1] + add[i])
        for p in range(keep[i], keep[i] + add[i]):
            page = table[i][p // P]
            slots.append(page * P + p % P if 0 <= page < 2 ** 31 // P else -1)
            positions.append(p)
            request.append(i)
    pad = max_rows - len(slots)
    return dict(status=PLAN_OK, lens=[k + a for k, a in zip(keep, add)], table=table, free=stack, cu=cu,
                slots=slots + [-1] * pad, positions=positions + [0] * pad, request=request + [-1] * pad)


def rope_rows(x: np.ndarray, positions, theta: float) -> np.ndarray:
    """RoPE of x [T][H][d] to a position per row (rotate-half pairs), fp64."""
    x = np.asarray(x, dtype=np.float64)
    d = x.shape[-1]
    ang = np.asarray(positions, dtype=np.float64)[:, None] * theta ** (-2.0 * np.arange(d // 2) / d)
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    lo, hi = x[..., :d // 2], x[..., d // 2:]
    return np.concatenate([lo * c - hi * s, hi * c + lo * s], axis=-1)


def quantize_rows(x: np.ndarray) -> tuple[np.ndarray, np.ndarray, np.ndarray]:
    """S3 for x [..., d] fp32: codes uint8 [..., d], scale and zero fp16 [...]."""
    x = np.ascontiguousarray(x, dtype=np.float32)
    d = x.shape[-1]
    z = quantize_nested(x.reshape(-1, d), d, 2, 2)
    return z["q"].reshape(x.shape), z["scale"][0].reshape(x.shape[:-1]), z["zero"][0].reshape(x.shape[:-1])


def values(codes: np.ndarray, scale: np.ndarray, zero: np.ndarray) -> np.ndarray:
    """S3, fp64."""
    return scale.astype(np.float64)[..., None] * (codes.astype(np.float64) - zero.astype(np.float64)[..., None])


def attention(q: np.ndarray, k_pool: np.ndarray, v_pool: np.ndarray, cu, lens, table, scale: float | None = None,
              window: int = 0, out: np.ndarray | None = None) -> np.ndarray:
    """S4.  q fp64 [T][Hq][d]; pools: values fp64 [pages][Hkv][P][d]; out: what
    rows behind the last request keep (zeros when None).  Returns fp64 [T][Hq][d]."""
    T, Hq, d = q.shape
    pages, Hkv, P, _ = k_pool.shape
    g = Hq // Hkv
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    res = np.zeros((T, Hq, d)) if out is None else np.array(out, dtype=np.float64)
    for i, n in enumerate(lens):
        rows = range(cu[i], min(cu[i + 1], T))
        if not len(rows):
            continue
        toks = [t for t in range(n) if 0 <= table[i][t // P] < pages]
        at = [(table[i][t // P], t % P) for t in toks]
        pg, off = (np.array([a[c] for a in at], dtype=np.int64) for c in (0, 1))
        toks = np.array(toks, dtype=np.int64)
        for r in rows:
            p = int(n - (cu[i + 1] - cu[i]) + (r - cu[i]))
            see = (toks <= p) & ((toks > p - window) if window > 0 else True)
            for h in range(Hkv):
                if not see.any():
                    res[r, h * g:(h + 1) * g] = 0.0
                    continue
                s = scale * (q[r, h * g:(h + 1) * g] @ k_pool[pg[see], h, off[see]].T)
                w = np.exp(s - s.max(-1, keepdims=True))
                res[r, h * g:(h + 1) * g] = (w / w.sum(-1, keepdims=True)) @ v_pool[pg[see], h, off[see]]
    return res


def lora(x: np.ndarray, A: np.ndarray, B: np.ndarray, scale, ids, y: np.ndarray | None) -> np.ndarray:
    """S5.  ids: the adapter of each row (outside [0, len(A)): none)."""
    out = np.zeros((x.shape[0], B.shape[1])) if y is None else np.array(y, dtype=np.float64)
    for t, a in enumerate(ids):
        if 0 <= a < len(A):
            out[t] += float(scale[a]) * (B[a].astype(np.float64) @ (A[a].astype(np.float64) @ x[t].astype(np.float64)))
    return out
