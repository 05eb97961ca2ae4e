"""Pins of the serving oracle (oracle.serving) to things other than itself:
hand-worked plans, library softmax over values assembled token by token, a
dense matmul with the merged weight for the adapters, the relative-position
identity of RoPE."""

import numpy as np
from scipy.special import softmax

from oracle import serving as os_


def test_plan_by_hand():
    # P = 4.  Request 0: 5 tokens in pages 7, 2, keeps 3 and adds 1: page 2 goes back.  Request 1: 4 tokens in
    # page 5, adds 5 (9 tokens, 3 pages): pops 2 (just given back), then 8.  Request 2: empty, adds 1: pops 1.
    r = os_.plan([5, 4, 0], [3, 4, 0], [1, 5, 1], [[7, 2, -1], [5, -1, -1], [-1, -1, -1]], [3, 1, 8], 8, 4, 9)
    assert r["status"] == os_.PLAN_OK
    assert r["table"] == [[7, 2, -1], [5, 2, 8], [1, -1, -1]]
    assert r["free"] == [3] and r["lens"] == [4, 9, 1] and r["cu"] == [0, 1, 6, 7]
    assert r["slots"] == [7 * 4 + 3, 2 * 4, 2 * 4 + 1, 2 * 4 + 2, 2 * 4 + 3, 8 * 4, 1 * 4, -1, -1]
    assert r["positions"] == [3, 4, 5, 6, 7, 8, 0, 0, 0]
    assert r["request"] == [0, 1, 1, 1, 1, 1, 2, -1, -1]


def test_plan_refusals_change_nothing():
    table = [[0, -1], [1, -1]]
    for lens, keep, add, free, cap, rows, want in (
            ([3, 2], [4, 2], [0, 0], [2], 4, 8, os_.PLAN_LENGTH),      # keeps more than it has
            ([3, 2], [3, 2], [0, 7], [2], 4, 8, os_.PLAN_LENGTH),      # 9 tokens in 2 pages of 4
            ([3, 2], [3, 2], [4, 5], [2, 3], 4, 8, os_.PLAN_ROWS),
            ([3, 2], [3, 2], [2, 3], [2], 4, 8, os_.PLAN_PAGES),
            ([3, 2], [0, 0], [0, 0], [2], 2, 8, os_.PLAN_PAGES)):       # two pages back, room for one
        r = os_.plan(lens, keep, add, table, free, cap, 4, rows)
        assert r["status"] == want and r["lens"] == lens and r["table"] == table and r["free"] == free
        assert set(r["slots"]) == {-1} and r["cu"] == [0, 0, 0]


def test_plan_keeps_every_page_once():
    rng = np.random.default_rng(5)
    P, R, MP = 4, 6, 8
    lens, table, free = [0] * R, [[-1] * MP for _ in range(R)], list(range(20))
    for _ in range(200):
        keep = [int(rng.integers(0, n + 1)) for n in lens]
        add = [int(rng.integers(0, 6)) for _ in lens]
        r = os_.plan(lens, keep, add, table, free, 20, P, 64)
        lens, table, free = r["lens"], r["table"], r["free"]
        held = [table[i][j] for i in range(R) for j in range(-(-lens[i] // P))]
        assert sorted(held + free) == list(range(20))


def test_rope_rows_relative_position():
    rng = np.random.default_rng(1)
    a, b = rng.standard_normal((1, 1, 64)), rng.standard_normal((1, 1, 64))
    dots = [(os_.rope_rows(a, [p + 17], 10000.0) * os_.rope_rows(b, [p], 10000.0)).sum() for p in (0, 5, 4000)]
    np.testing.assert_allclose(dots, dots[0], rtol=1e-10)
    np.testing.assert_array_equal(os_.rope_rows(a, [0], 10000.0), a)


def test_quantize_rows_error_and_values():
    x = np.random.default_rng(2).standard_normal((7, 3, 64)).astype(np.float32)
    c, s, z = os_.quantize_rows(x)
    assert c.max() <= 15
    # half a step, the scale's fp16 rounding (15 steps at most, 2^-11 each) and the zero point's own half step
    assert np.all(np.abs(os_.values(c, s, z) - x) <= s[..., None].astype(np.float64) * (1.0 + 15 * 2.0 ** -11))


def test_attention_against_library_softmax():
    rng = np.random.default_rng(3)
    P, Hkv, g, d = 4, 2, 3, 8
    k, v = rng.standard_normal((2, 5, Hkv, P, d))
    table, lens, cu = [[4, 1, 0], [3, 9, -1]], [9, 6], [0, 2, 5]   # page 9 does not exist: tokens 4, 5 of request 1
    q = rng.standard_normal((6, Hkv * g, d))
    out = os_.attention(q, k, v, cu, lens, table, window=4, out=np.full((6, Hkv * g, d), 7.0))
    assert np.all(out[5] == 7.0)
    for r, toks in ((0, [4, 5, 6, 7]), (1, [5, 6, 7, 8]), (2, [0, 1, 2, 3]), (3, [1, 2, 3]), (4, [2, 3])):
        i = 0 if r < 2 else 1
        kk = np.stack([k[table[i][t // P], :, t % P] for t in toks])
        vv = np.stack([v[table[i][t // P], :, t % P] for t in toks])
        for h in range(Hkv * g):
            w = softmax(kk[:, h // g] @ q[r, h] / np.sqrt(d))
            np.testing.assert_allclose(out[r, h], w @ vv[:, h // g], rtol=1e-12)


def test_attention_rows_without_tokens():
    k = v = np.ones((1, 1, 4, 8))
    out = os_.attention(np.ones((3, 1, 8)), k, v, [0, 3], [2], [[0]])     # three rows, two tokens: the first sees none
    assert np.all(out[0] == 0.0) and np.all(out[1:] == 1.0)
    assert np.all(os_.attention(np.ones((3, 1, 8)), k, v, [0, 3], [3], [[1]]) == 0.0)


def test_lora_against_merged_weight():
    rng = np.random.default_rng(4)
    x, y = rng.standard_normal((4, 16)), rng.standard_normal((4, 5))
    A, B, s = rng.standard_normal((2, 3, 16)), rng.standard_normal((2, 5, 3)), [2.0, 0.5]
    out = os_.lora(x, A, B, s, [1, -1, 0, 2], y)
    np.testing.assert_allclose(out[0], y[0] + x[0] @ (0.5 * B[1] @ A[1]).T, rtol=1e-12)
    np.testing.assert_allclose(out[2], y[2] + x[2] @ (2.0 * B[0] @ A[0]).T, rtol=1e-12)
    np.testing.assert_array_equal(out[[1, 3]], y[[1, 3]])
