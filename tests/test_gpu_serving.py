"""Parity of the operators for a step of many requests (paged 4-bit cache,
per-request adapters) with the fp64 oracle, at the sizes and masks where they
can go wrong.

Tolerances.  Plans, codes, scales and zero points are exact.  bf16 outputs: half
a step, 2^-8 of the value, over the fp32 bound below.
Attention: a score is scale ks (sum q (c - z)); q enters in 22-bit fixed point
(2^-22 of its row's maximum), the sums and products in fp32, so with S the
largest scale ks sum |q| 15 of the call a score is within 2^-20 S and a softmax
weight within 2^-19 S relatively.  Weights enter the value product with 2^-22,
and a chain of L/16 products with 16 terms each is summed in fp32, so with V
the largest |v|: |out - exact| <= 2 V (2^-19 S + 2^-21 + (64 + L/16) 2^-24).
For bf16 outputs q enters in 15-bit fixed point: an entry is off by up to
2^-15 qmax (uniform, sigma 2^-15.8 qmax), so a score by a sum of d such errors
times scale ks |c - z| (rms at most 8): six sigma of that is E = 6 2^-15.8 qmax
8 sqrt(d) scale ks, a weight is off by 2 E + 2^-11 relatively, and 2 V (2 E +
2^-11) is added; over all outputs the errors are independent, so their 2-norm
is within 2^-8 of the outputs'.
Adapters: fp32 sums of at most K + rank + 40 terms, in chains of 16, so
|out - exact| <= 2^-24 (|out| + (K/8 + rank/8 + 40) M), M = scale |B| (|A| |x|).
"""

import numpy as np
import pytest
import torch

from oracle import attn as oattn
from oracle import decode as odec
from oracle import serving as osv

pytestmark = pytest.mark.gpu

BF16 = 2.0 ** -8


@pytest.fixture(scope="module")
def sf():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import quantized_gemv_kv_b200 as sf
    return sf


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _i32(a):
    return _dev(np.asarray(a, dtype=np.int32))


def _f64(t):
    return t.detach().double().cpu().numpy()


# ---- plan ------------------------------------------------------------------------


def _random_state(rng, R, P, MP, pages, max_rows, calm=False):
    lens, table, used = [], np.full((R, MP), -1, np.int64), 0
    perm = rng.permutation(pages)
    for i in range(R):
        n = int(rng.integers(0, MP * P // 2 + 1))
        h = -(-n // P)
        if used + h > pages // 2:
            n = h = 0
        lens.append(n)
        table[i, :h] = perm[used:used + h]
        used += h
    keep = [n if calm or rng.random() < 0.5 else int(rng.integers(0, n + 1)) for n in lens]
    add = [1 if calm else int(rng.choice([0, 1, 1, 5, 40])) for _ in lens]
    add = [min(a, MP * P - k) for a, k in zip(add, keep)]
    while sum(add) > max_rows:
        add[int(np.argmax(add))] //= 2
    return lens, keep, add, table, [int(p) for p in perm[used:]]


def _run_plan(sf, lens, keep, add, table, free, cap, P, max_rows, in_place=False, stride=None, use_keep=True):
    R, MP = table.shape
    d_lens, d_n = _i32(lens), _i32([len(free)])
    buf = torch.full((R, stride or MP), -9, dtype=torch.int32, device="cuda")
    tab = buf[:, :MP]
    tab.copy_(_i32(table))
    lst = torch.full((cap,), -9, dtype=torch.int32, device="cuda")
    lst[:len(free)] = _i32(free)
    kw = {} if in_place else dict(lens_out=torch.full_like(d_lens, -9), n_free_out=torch.full_like(d_n, -9))
    job = sf.paged_plan(d_lens, _i32(add), tab, lst, d_n, P, max_rows, keep=_i32(keep) if use_keep else None, **kw)
    torch.cuda.synchronize()
    return job, buf


def _check_plan(job, buf, want, R, MP, free_before):
    n = int(job.n_free_out.item())
    assert int(job.status.item()) == want["status"]
    assert job.lens_out.tolist() == want["lens"] and job.cu_rows.tolist() == want["cu"]
    assert job.slots.tolist() == want["slots"] and job.positions.tolist() == want["positions"]
    assert job.row_request.tolist() == want["request"]
    assert n == len(want["free"]) and job.free_list[:n].tolist() == want["free"]
    np.testing.assert_array_equal(buf[:, :MP].cpu().numpy(), np.array(want["table"]))
    assert torch.all(buf[:, MP:] == -9)


@pytest.mark.parametrize("R,P,MP,max_rows,in_place", [
    (1, 16, 1, 1, True), (1, 16, 3, 40, False), (3, 32, 4, 64, True), (16, 64, 64, 16, True), (129, 16, 9, 700, False),
    (1000, 16, 20, 20000, True), (257, 256, 5, 4097, True), (8192, 16, 4, 60000, True)])
def test_plan(sf, R, P, MP, max_rows, in_place):
    rng = np.random.default_rng(R + P)
    pages = max(4, 2 * R * MP // 3 + 3)
    st = _random_state(rng, R, P, MP, pages, max_rows)
    want = osv.plan(*st[:4], st[4], pages, P, max_rows)
    assert want["status"] == osv.PLAN_OK
    job, buf = _run_plan(sf, *st, pages, P, max_rows, in_place, stride=MP + 3)
    _check_plan(job, buf, want, R, MP, st[4])


def test_plan_without_keep(sf):
    rng = np.random.default_rng(8)
    lens, _, add, table, free = _random_state(rng, 40, 16, 6, 300, 400)
    add = [min(a, 6 * 16 - n) for a, n in zip(add, lens)]
    want = osv.plan(lens, lens, add, table, free, 300, 16, 400)
    job, buf = _run_plan(sf, lens, lens, add, table, free, 300, 16, 400, use_keep=False)
    _check_plan(job, buf, want, 40, 6, free)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("what", ["len", "keep", "negative", "room", "huge", "rows", "pages", "cap", "n_free"])
def test_plan_refusals_on_the_device(sf, what, in_place):
    """Nothing changes, and the step has no rows."""
    lens, keep, add, table, free, cap, P, rows = [40, 20, 0], [40, 20, 0], [1, 1, 1], np.array(
        [[3, 5, 1, -1], [0, 2, -1, -1], [-1] * 4]), [4, 6], 9, 16, 8
    if what == "len":
        lens[1] = 65
    elif what == "keep":
        keep[1] = 21
    elif what == "negative":
        add[2] = -1
    elif what == "room":
        add[0] = 25
    elif what == "huge":
        add[0] = 2 ** 31 - 1
    elif what == "rows":
        add[:] = [4, 4, 1]
    elif what == "pages":
        add[2] = 49
        rows = 64
    elif what == "cap":
        keep, add, cap = [0, 0, 0], [0, 0, 0], 6
    if what == "n_free":
        job_free = [4, 6, 7]
        want = dict(status=osv.PLAN_PAGES, lens=lens, table=table.tolist(), free=job_free, cu=[0] * 4,
                    slots=[-1] * rows, positions=[0] * rows, request=[-1] * rows)
        d_n = _i32([-1])
        job = sf.paged_plan(_i32(lens), _i32(add), _i32(table), _i32(job_free), d_n, P, rows)
        assert int(job.status.item()) == osv.PLAN_PAGES and int(d_n.item()) == -1 and job.cu_rows.tolist() == [0] * 4
        return
    want = osv.plan(lens, keep, add, table, free, cap, P, rows) if what != "huge" else dict(
        status=osv.PLAN_LENGTH, lens=lens, table=table.tolist(), free=free, cu=[0] * 4, slots=[-1] * rows,
        positions=[0] * rows, request=[-1] * rows)
    assert want["status"] != osv.PLAN_OK
    job, buf = _run_plan(sf, lens, keep, add, table, free, cap, P, rows, in_place)
    _check_plan(job, buf, want, 3, 4, free)


def test_plan_many_steps_in_a_graph(sf):
    """In-place steps from one captured graph, as a decode loop replays it."""
    rng = np.random.default_rng(3)
    R, P, MP, pages, rows = 12, 16, 8, 60, 64
    lens, table, free = [0] * R, np.full((R, MP), -1), list(range(pages))
    d_lens, d_n, d_keep, d_add = _i32(lens), _i32([pages]), _i32(lens), _i32(lens)
    tab, lst = _i32(table), _i32(free)
    job = sf.PagedPlan(d_lens, d_add, tab, lst, d_n, P, rows, keep=d_keep)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        job.run()
    table = table.tolist()
    for step in range(40):
        keep = [int(rng.integers(max(0, n - 9), n + 1)) if rng.random() < 0.9 else 0 for n in lens]
        add = [int(rng.integers(0, 6)) for _ in lens]
        d_keep.copy_(_i32(keep))
        d_add.copy_(_i32(add))
        g.replay()
        torch.cuda.synchronize()
        want = osv.plan(lens, keep, add, table, free, pages, P, rows)
        assert int(job.status.item()) == want["status"]
        lens, table, free = want["lens"], want["table"], want["free"]
        assert d_lens.tolist() == lens and tab.tolist() == table and int(d_n.item()) == len(free)
        assert lst[:len(free)].tolist() == free and job.slots.tolist() == want["slots"]


# ---- append ----------------------------------------------------------------------


def _pool_np(kv):
    c = kv.k_codes.cpu().numpy().view(np.uint32), kv.v_codes.cpu().numpy().view(np.uint32)
    return [((x[..., None] >> (4 * np.arange(8, dtype=np.uint32))) & 15).reshape(*x.shape[:-1], -1) for x in c] + \
        [kv.k_param.cpu().numpy(), kv.v_param.cpu().numpy()]


@pytest.mark.parametrize("T,Hq,Hkv,d,P,src,rope", [
    (1, 32, 8, 128, 64, "fp32", True), (16, 32, 8, 128, 64, "fp32", True), (37, 3, 1, 64, 16, "fp32", True),
    (301, 8, 8, 256, 32, "bf16", True), (5, 0, 2, 128, 16, "fp32", True), (130, 0, 8, 128, 256, "bf16", False),
    (700, 0, 3, 64, 128, "fp32", False), (2, 0, 256, 64, 16, "fp32", False),
    # enough rows for a block to take several at a time (4, 8 and 2), odd head counts
    (2403, 3, 1, 128, 64, "fp32", True), (4801, 1, 1, 64, 64, "bf16", True), (1203, 2, 3, 256, 32, "fp32", True)])
def test_append(sf, T, Hq, Hkv, d, P, src, rope):
    rng = np.random.default_rng(T + d)
    pages = -(-T // P) + 2
    dt = torch.float32 if src == "fp32" else torch.bfloat16
    width = (Hq + 2 * Hkv) * d + 8                       # a fused projection's output with a gap behind each row
    x = torch.randn((T, width), generator=torch.Generator().manual_seed(T)).to(dt).cuda()
    q = x[:, :Hq * d].unflatten(1, (Hq, d)) if Hq else None
    k, v = (x[:, (Hq + o) * d:(Hq + o + Hkv) * d].unflatten(1, (Hkv, d)) for o in (0, Hkv))
    x[0, Hq * d:(Hq + Hkv) * d] = 0.5                    # a constant row: a scale of zero becomes 1 without a rotation
    slots = rng.permutation(pages * P)[:T].astype(np.int32)
    if T > 4:
        slots[1], slots[2], slots[3] = -1, pages * P, 2 ** 31 - 1
    pos = rng.integers(0, 1 << 20, T).astype(np.int32)
    kv = sf.PagedKV.empty(pages, Hkv, P, d)
    for t in (kv.k_codes, kv.v_codes):
        t.fill_(0x5A5A5A5A)
    q_out = torch.full((T, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda") if Hq else None
    val = [torch.full((T, Hkv, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    got = sf.paged_append(kv, k, v, _i32(slots), _i32(pos) if rope else None, 500000.0 if rope else 0.0, q, q_out,
                          *val)
    torch.cuda.synchronize()
    assert got is q_out
    live = (slots >= 0) & (slots < pages * P)
    kc, vc, kp, vp = _pool_np(kv)
    free = np.ones((pages, P), bool)
    free[slots[live] // P, slots[live] % P] = False
    for name, xs, c, p, vals in (("k", k, kc, kp, val[0]), ("v", v, vc, vp, val[1])):
        rows = _f64(xs)
        if name == "k" and rope:
            rows = osv.rope_rows(rows, pos, 500000.0)
        wc, ws, wz = osv.quantize_rows(rows.astype(np.float32))
        at = slots[live] // P, slots[live] % P
        np.testing.assert_array_equal(c[at[0], :, at[1]], wc[live])
        np.testing.assert_array_equal(p[at[0], :, at[1], 0], ws[live])
        np.testing.assert_array_equal(p[at[0], :, at[1], 1], wz[live])
        assert np.all(p.transpose(0, 2, 1, 3)[free] == 0)
        assert np.all(c.transpose(0, 2, 1, 3)[free].reshape(-1, 8)[:, ::2] == 0xA)
        want = osv.values(wc, ws, wz)
        err = np.abs(_f64(vals) - want)[live]
        assert np.all(err <= BF16 * np.abs(want[live]))
        assert np.all(_f64(vals)[~live] == 7.0)
    if Hq:
        want = osv.rope_rows(_f64(q), pos, 500000.0)
        # the rotation is rounded once; its fp64 error counts where terms cancel
        assert np.all(np.abs(_f64(q_out) - want)[live] <= BF16 * np.abs(want[live]) + 1e-12)
        assert np.all(_f64(q_out)[~live] == 7.0)


def test_append_equals_sf_rope(sf):
    """The rotation is the stand-alone operator's, bit for bit."""
    q = torch.randn((1, 4, 128), generator=torch.Generator().manual_seed(1)).cuda()
    kv = sf.PagedKV.empty(1, 1, 16, 128)
    k = torch.zeros((1, 1, 128), device="cuda")
    got = sf.paged_append(kv, k, k, _i32([3]), _i32([98765]), 500000.0, q)
    want = sf.rope(q[0].clone(), 98765, 500000.0, y=torch.empty((4, 128), dtype=torch.bfloat16, device="cuda"))
    assert torch.equal(got[0], want)


def test_append_to_interleaved_layers(sf):
    """Pages of two layers in one allocation: only the layer's own rows change."""
    Hkv, P, d, pages = 2, 16, 128, 5
    codes = [torch.full((pages, 2, Hkv, P, d // 8), 0x77777777, dtype=torch.int32, device="cuda") for _ in range(2)]
    param = [torch.full((pages, 2, Hkv, P, 2), 3.0, dtype=torch.float16, device="cuda") for _ in range(2)]
    kv = sf.PagedKV(codes[0][:, 1], param[0][:, 1], codes[1][:, 1], param[1][:, 1])
    plain = sf.PagedKV.empty(pages, Hkv, P, d)
    x = torch.randn((2, 9, Hkv, d), generator=torch.Generator().manual_seed(2)).cuda()
    slots = _i32([0, 17, 79, 40, 41, 42, 5, 6, 64])
    for target in (kv, plain):
        sf.paged_append(target, x[0], x[1], slots)
    for c, p, a, b in ((codes[0], param[0], plain.k_codes, plain.k_param),
                       (codes[1], param[1], plain.v_codes, plain.v_param)):
        assert torch.all(c[:, 0] == 0x77777777) and torch.all(p[:, 0] == 3.0)
        page, off = slots.long() // P, slots.long() % P
        assert torch.equal(c[:, 1][page, :, off], a[page, :, off])
        assert torch.equal(p[:, 1][page, :, off], b[page, :, off])


# ---- attention -------------------------------------------------------------------


class _Case:
    """Requests with their pages, in a pool whose unused tokens hold garbage
    (NaN scales among them)."""

    def __init__(self, sf, seed, n, lens, Hq, Hkv, d, P, extra_rows=2, layers=1, gain=10.0, v_gain=1.0):
        rng = np.random.default_rng(seed)
        self.lens, self.n, self.P, self.Hkv = list(lens), list(n), P, Hkv
        used = [-(-x // P) for x in lens]
        pages = sum(used) + 2
        perm = rng.permutation(pages)
        self.table = np.full((len(lens), max(used + [0]) + 2), pages + 5, np.int32)
        at = 0
        for i, u in enumerate(used):
            self.table[i, :u] = perm[at:at + u]
            at += u
        self.cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        self.T = int(self.cu[-1]) + extra_rows
        self.codes = rng.integers(0, 2 ** 32, (2, pages, layers, Hkv, P, d // 8), dtype=np.uint32)
        self.param = rng.integers(0, 2 ** 16, (2, pages, layers, Hkv, P, 2), dtype=np.uint16)
        self.param[..., 0] |= 0x7E00 * (rng.random(self.param.shape[:-1]) < 0.5).astype(np.uint16)  # many NaN
        self.val = np.zeros((2, pages, Hkv, P, d))
        g = np.ones((Hkv, d))
        g[:, :4] = gain
        for i, x in enumerate(lens):
            for j in range(used[i]):
                m, page = min(P, x - j * P), self.table[i, j]
                for w, by in ((0, g[:, None]), (1, v_gain)):
                    c, s, z = osv.quantize_rows((rng.standard_normal((Hkv, m, d)) * by).astype(np.float32))
                    packed = (c.reshape(Hkv, m, -1, 8).astype(np.uint32) << (4 * np.arange(8, dtype=np.uint32)))
                    self.codes[w, page, -1, :, :m] = packed.sum(-1, dtype=np.uint32)
                    self.param[w, page, -1, :, :m, 0] = s.view(np.uint16)
                    self.param[w, page, -1, :, :m, 1] = z.view(np.uint16)
                    self.val[w, page, :, :m] = osv.values(c, s, z)
        self.q = torch.from_numpy(rng.standard_normal((self.T, Hq, d)).astype(np.float32)).to(torch.bfloat16)
        codes, param = _dev(self.codes.view(np.int32)), _dev(self.param.view(np.int16)).view(torch.float16)
        self.kv = sf.PagedKV(codes[0, :, -1], param[0, :, -1], codes[1, :, -1], param[1, :, -1])

    def run(self, sf, out_type=torch.float32, **kw):
        out = torch.full(self.q.shape, 7.0, dtype=out_type, device="cuda")
        sf.attn_paged(self.q.cuda(), self.kv, _i32(self.cu), _i32(self.lens), _i32(self.table), out, **kw)
        torch.cuda.synchronize()
        return out

    def check(self, sf, out_type=torch.float32, out=None, **kw):
        out = _f64(self.run(sf, out_type, **kw) if out is None else out)
        q = _f64(self.q)[:len(out)]
        want = osv.attention(q, self.val[0], self.val[1], self.cu, self.lens, self.table, out=np.full(q.shape, 7.0),
                             **kw)
        scale = kw.get("scale") or 1.0 / np.sqrt(q.shape[-1])
        ks = np.abs(self.val[0]).max() / 7.0              # the largest key scale: values reach at least 7 steps
        S = scale * ks * np.abs(q).sum(-1).max() * 15
        V = np.abs(self.val[1]).max()
        tol = 2 * V * (2.0 ** -19 * S + 2.0 ** -21 + (64 + max(self.lens) / 16) * 2.0 ** -24)
        err = np.abs(out - want)
        if out_type == torch.bfloat16:
            E = 6 * 2.0 ** -15.8 * np.abs(q).max() * 8 * np.sqrt(q.shape[-1]) * scale * ks
            tol = tol + BF16 * np.abs(want) + 2 * V * (2 * E + 2.0 ** -11)
            rows = slice(0, self.cu[-1])
            assert np.linalg.norm(err[rows]) <= 2.0 ** -8 * np.linalg.norm(want[rows])
        assert np.all(err <= tol), (err.max(), np.max(tol))
        assert np.all(out[self.cu[-1]:] == 7.0)
        return err.max()


@pytest.mark.parametrize("Hq,Hkv,d,P", [(32, 8, 128, 64), (1, 1, 128, 16), (8, 8, 64, 16), (8, 1, 128, 32),
                                        (10, 2, 128, 128), (16, 1, 64, 256), (4, 2, 256, 16), (8, 1, 256, 64),
                                        (33, 3, 128, 16), (64, 1, 128, 16)])
@pytest.mark.parametrize("out_type", [torch.float32, torch.bfloat16])
def test_attention_head_layouts(sf, Hq, Hkv, d, P, out_type):
    _Case(sf, Hq + d, [1, 1, 1], [37, 300, 129], Hq, Hkv, d, P).check(sf, out_type)


@pytest.mark.parametrize("P", [16, 64])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attention_lengths(sf, d, P):
    """Lengths around a page's and a tile's end; requests without rows or without tokens."""
    lens = [1, 2, 15, 16, 17, 0, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 0, 513]
    n = [1] * len(lens)
    n[5], n[7], n[18] = 0, 0, 0
    _Case(sf, d + P, n, lens, 8, 2, d, P).check(sf)


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 128), (8, 8, 64), (5, 1, 128), (4, 1, 256)])
@pytest.mark.parametrize("window,out_type", [(0, torch.float32), (1, torch.float32), (16, torch.float32),
                                             (70, torch.float32), (0, torch.bfloat16), (70, torch.bfloat16)])
def test_attention_rows_and_windows(sf, Hq, Hkv, d, window, out_type):
    """Several rows per request (causal), more rows than tokens (the first rows see none), sliding windows."""
    _Case(sf, 5 + window, [4, 1, 7, 20, 3, 33], [200, 70, 7, 65, 1, 300], Hq, Hkv, d, 16).check(
        sf, out_type, window=window)


@pytest.mark.parametrize("out_type", [torch.float32, torch.bfloat16])
def test_attention_long(sf, out_type):
    """One long request beside short ones: its cache is split over many blocks."""
    _Case(sf, 11, [1, 2, 1], [20011, 5, 700], 8, 2, 128, 64).check(sf, out_type)


def test_attention_many_requests(sf):
    rng = np.random.default_rng(12)
    lens = rng.integers(0, 40, 700).tolist()
    _Case(sf, 13, [int(x > 0) for x in lens], lens, 4, 1, 64, 16, gain=1.0).check(sf)


@pytest.mark.parametrize("v_gain,scale", [(1e-4, None), (3000.0, None), (1.0, 0.5), (1.0, 1e-3), (1.0, -0.1)])
def test_attention_ranges(sf, v_gain, scale):
    """Small and large values, sharp and flat weights."""
    kw = {} if scale is None else dict(scale=scale)
    if scale == -0.1:
        c = _Case(sf, 17, [1, 1], [100, 500], 4, 2, 128, 32)
        q = _f64(c.q)
        want = osv.attention(q, c.val[0], c.val[1], c.cu, c.lens, c.table, scale=-0.1, out=np.full(q.shape, 7.0))
        assert np.abs(_f64(c.run(sf, scale=-0.1)) - want).max() <= 1e-3
        return
    _Case(sf, 17, [1, 1], [100, 500], 4, 2, 128, 32, v_gain=v_gain).check(sf, **kw)


def test_attention_value_scales_that_grow(sf):
    """Value scales that differ by 2^20 along the cache, growing and falling: the weights' f16 pairs follow them."""
    c = _Case(sf, 19, [1, 1], [400, 400], 4, 2, 128, 16)
    for i, sign in ((0, 1), (1, -1)):
        for j in range(25):
            f = 2.0 ** (sign * (j - 12) * 20 / 24)
            page = c.table[i, j]
            s = (c.param[1, page, -1, :, :, 0].view(np.float16).astype(np.float64) * f).astype(np.float16)
            ratio = s.astype(np.float64) / c.param[1, page, -1, :, :, 0].view(np.float16).astype(np.float64)
            c.param[1, page, -1, :, :, 0] = s.view(np.uint16)
            c.val[1, page] *= ratio[..., None]
    c.kv.v_param.copy_(_dev(c.param[1].view(np.int16)).view(torch.float16)[:, -1])
    c.check(sf)


@pytest.mark.parametrize("P", [16, 128])
def test_attention_leaves_bad_pages_out(sf, P):
    """Pages outside the pool, inside a request and for all of it."""
    c = _Case(sf, 23, [2, 1, 1, 1], [500, 300, 40, 129], 8, 2, 128, P)
    pages = c.val.shape[1]
    c.table[0, 1], c.table[1, 0], c.table[2, :] = -1, pages, 2 ** 31 - 1
    c.table[3, (129 + P - 1) // P - 1] = -(2 ** 31)
    c.check(sf)
    c.check(sf, window=100)


def test_attention_key_scale_zero_is_no_token(sf):
    c = _Case(sf, 29, [1], [200], 4, 1, 128, 16)
    page, off = c.table[0, 3], 5                          # token 53
    c.kv.k_param[page, :, off, 0] = 0.0
    out = _f64(c.run(sf))
    keep = [t for t in range(200) if t != 53]
    k, v = (np.stack([c.val[w, c.table[0, t // 16], 0, t % 16] for t in keep]) for w in (0, 1))
    q = _f64(c.q)[0]
    s = q @ k.T / np.sqrt(128)
    w = np.exp(s - s.max(-1, keepdims=True))
    assert np.abs(out[0] - (w / w.sum(-1, keepdims=True)) @ v).max() <= 1e-3


def test_attention_nonfinite_queries_stay_in_their_head(sf):
    c = _Case(sf, 31, [1, 3], [150, 90], 8, 2, 128, 16)
    clean = c.run(sf)
    c.q[0, 3, 5], c.q[2, 6, 0] = float("nan"), float("inf")
    out = c.run(sf)
    bad = torch.zeros(out.shape[:2], dtype=torch.bool, device="cuda")
    bad[0, 3] = bad[2, 6] = True
    assert torch.all(torch.isnan(out[bad])) and torch.equal(out[~bad], clean[~bad])
    c.q[2, 6] = 0.0                                       # a zero query: the plain mean
    out = _f64(c.run(sf))
    v = np.stack([c.val[1, c.table[1, t // 16], 1, t % 16] for t in range(89)])
    assert np.abs(out[2, 6] - v.mean(0)).max() <= 1e-5


def test_attention_strides_and_layers(sf):
    """Strided q and out rows, a strided block table, pages of two layers interleaved."""
    c = _Case(sf, 37, [1, 2, 1], [100, 64, 33], 8, 2, 128, 16, layers=2)
    want = c.run(sf)
    T = c.T
    q = torch.full((T, 3, 8, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    q[:, 1] = c.q.cuda()
    out = torch.full((T, 8 * 128 + 12), 7.0, device="cuda")
    tab = torch.full((3, 50), -7, dtype=torch.int32, device="cuda")
    tab[:, :c.table.shape[1]] = _i32(c.table)
    view = out[:, :8 * 128].unflatten(1, (8, 128))
    sf.attn_paged(q[:, 1], c.kv, _i32(c.cu), _i32(c.lens), tab[:, :c.table.shape[1]], view)
    assert torch.equal(view, want) and torch.all(out[:, 8 * 128:] == 7.0)


def test_attention_rows_behind_the_buffer(sf):
    """cu_rows past T, and lengths outside the table: clamped, never read or written out of bounds."""
    c = _Case(sf, 41, [1, 3], [60, 90], 4, 2, 128, 16, extra_rows=0)
    out = torch.full((2, 4, 128), 7.0, device="cuda")
    sf.attn_paged(c.q[:2].cuda(), c.kv, _i32(c.cu), _i32(c.lens), _i32(c.table), out)
    c.check(sf, out=out)      # to rounding: fewer columns are other runs of stages, whose sums come in another order
    out = c.run(sf)
    c.lens = [-5, 10 ** 9]
    got = c.run(sf)                                       # request 0 has no token, request 1 all that its table holds
    assert torch.all(got[0] == 0.0) and torch.isfinite(out).all()


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 3])
def test_attention_window_longer_than_any_request(sf, window):
    """The largest windows beside requests of more rows than tokens."""
    c = _Case(sf, 53, [5, 3, 1], [1, 90, 0], 8, 2, 128, 16)
    c.check(sf, window=window)
    assert torch.equal(c.run(sf, window=window), c.run(sf))


def test_attention_longest_table(sf):
    """A table of 2^31 - 16 tokens, the most there can be: one page in its first half, another in its second, a third
    one for the last 11 tokens, which change nothing that counts here (2^-24)."""
    d, P, n = 64, 16, 2 ** 27 - 1
    c = _Case(sf, 59, [1, 1, 1], [16, 16, 16], 1, 1, d, P, extra_rows=0)
    a, b, last = (int(c.table[i, 0]) for i in range(3))
    table = torch.full((1, n), a, dtype=torch.int32, device="cuda")
    table[0, n // 2:] = b
    table[0, -1] = last
    got = _f64(sf.attn_paged(c.q[:1].cuda(), c.kv, _i32([0, 1]), _i32([n * P - 5]), table))[0]
    k, v = (np.concatenate([c.val[w, a, 0], c.val[w, b, 0]]) for w in (0, 1))
    s = _f64(c.q)[0] @ k.T / np.sqrt(d)
    w = np.exp(s - s.max(-1, keepdims=True))
    want = (w / w.sum(-1, keepdims=True)) @ v
    # a lane sums the weights of up to 2^31 / (148 * 8 * 8) = 226722 tokens one by one: 2^-24 of the sum each
    assert np.abs(got - want).max() <= np.abs(v).max() * 226722 * 2.0 ** -23


def test_attention_repeats_bit_for_bit(sf):
    c = _Case(sf, 43, [1, 2, 1], [9000, 64, 1200], 8, 2, 128, 64)
    first = c.run(sf)
    ws = torch.full((sf.attn_paged_workspace_size(c.T, 3, 8, 2, 128),), 0xFF, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        assert torch.equal(c.run(sf, workspace=ws), first)


def test_attention_in_graphs_and_on_other_streams(sf):
    """Two captured graphs with a workspace each, replayed on two streams at once, with lengths that change between replays."""
    cs = [_Case(sf, 47 + i, [1, 1], [3000 + i, 200], 8, 2, 128, 64) for i in range(2)]
    jobs = []
    for c in cs:
        out = torch.zeros(c.q.shape, device="cuda")
        lens = _i32(c.lens)
        job = sf.PagedAttention(c.q.cuda(), c.kv, _i32(c.cu), lens, _i32(c.table), out)
        g = torch.cuda.CUDAGraph()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=s):
            job.run()
        jobs.append((job, g, lens, out))
    torch.cuda.synchronize()
    for lens in ([3000, 200], [1, 64], [2500, 0]):
        streams = [torch.cuda.Stream() for _ in cs]
        for (job, g, d_lens, out), s in zip(jobs, streams):
            d_lens.copy_(_i32(lens))
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                for _ in range(4):
                    g.replay()
        torch.cuda.synchronize()
        for c, (job, g, d_lens, out) in zip(cs, jobs):
            c.lens = lens
            rows = int(c.cu[-1])
            assert torch.equal(out[:rows], c.run(sf)[:rows])


def test_functions_on_another_stream(sf):
    """A function allocates on the stream it is given: nothing that the current stream does with its memory meantime
    gets in the way, and the zeros of an output come before the call."""
    c = _Case(sf, 61, [1, 2], [4000, 300], 8, 2, 128, 64)
    q, cu, lens, table = c.q.cuda(), _i32(c.cu), _i32(c.lens), _i32(c.table)
    want = sf.attn_paged(q, c.kv, cu, lens, table)
    x, A, B, scale, _ = _lora_case(5, 128, 96, 8, 2, 62)
    args = [t.cuda() for t in (x, A, B, scale)] + [_i32([0, 1, 0, -1, 1])]
    add = sf.lora_add(*args)
    torch.cuda.synchronize()
    need = sf.attn_paged_workspace_size(c.T, 2, 8, 2, 128)
    s = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s):
            torch.cuda._sleep(5_000_000)
        out, got = sf.attn_paged(q, c.kv, cu, lens, table, stream=s), sf.lora_add(*args, stream=s)
        for _ in range(20):
            torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
            torch.full(want.shape, 9.0, device="cuda")
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(got, add)


# ---- adapters --------------------------------------------------------------------


def _lora_case(T, K, N, rank, n, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, K), generator=g).to(torch.bfloat16)
    A = (torch.randn((n, rank, K), generator=g) / K ** 0.5).to(torch.bfloat16)
    B = torch.randn((n, N, rank), generator=g).to(torch.bfloat16)
    scale = torch.rand(n, generator=g) + 0.5
    return x, A, B, scale, torch.randn((T, N), generator=g)


def _lora_tol(x, A, B, scale, ids, want, K, rank):
    M = osv.lora(np.abs(x), np.abs(A), np.abs(B), np.abs(scale), ids, None)
    return 2.0 ** -24 * (np.abs(want) + (K / 8 + rank / 8 + 40) * M)


@pytest.mark.parametrize("T,K,N,rank,n", [
    (1, 4096, 4096, 16, 3), (16, 4096, 1024, 16, 16), (5, 8, 1, 8, 2), (17, 520, 777, 24, 4), (3, 1000, 130, 128, 3),
    (64, 512, 1024, 64, 5), (300, 264, 200, 32, 7), (33, 4096, 96, 40, 2), (130, 1032, 4100, 128, 1),
    (700, 72, 520, 16, 5), (128, 64, 3000, 8, 30), (1300, 128, 36, 48, 2)])
def test_lora(sf, T, K, N, rank, n):
    x, A, B, scale, y = _lora_case(T, K, N, rank, n, T + K)
    rng = np.random.default_rng(T)
    ids = rng.integers(-1, n + 1, T)                      # -1 and n: no adapter
    want = osv.lora(_f64(x), _f64(A), _f64(B), scale.numpy(), ids, _f64(y))
    tol = _lora_tol(_f64(x), _f64(A), _f64(B), scale.numpy(), ids, want, K, rank)
    yd = y.cuda()
    out = sf.lora_add(x.cuda(), A.cuda(), B.cuda(), scale.cuda(), _i32(ids), torch.full((T, N), 7.0, device="cuda"), yd)
    assert np.all(np.abs(_f64(out) - want) <= tol)
    bare = [t for t in range(T) if not 0 <= ids[t] < n]
    assert torch.equal(out[bare].cpu(), y[bare])          # no adapter: the row itself
    # in place, and without y
    got = sf.lora_add(x.cuda(), A.cuda(), B.cuda(), scale.cuda(), _i32(ids), y=yd)
    assert got is yd and torch.equal(got, out)
    none = sf.lora_add(x.cuda(), A.cuda(), B.cuda(), scale.cuda(), _i32(ids))
    assert np.all(np.abs(_f64(none) - (want - _f64(y))) <= tol)


def test_lora_runs_row_of_and_strides(sf):
    """Runs of rows of one request (prompts), ids per request, strided rows; the gaps stay as they are."""
    T, K, N, rank, n = 100, 256, 300, 16, 3
    x, A, B, scale, y = _lora_case(T, K, N, rank, n, 3)
    of = np.repeat([0, 1, 2, 3, -1, 4], [40, 1, 17, 30, 5, 7])
    per = [2, 0, -1, 1]                                   # request 4 lies behind n_ids
    ids = np.array([per[o] if 0 <= o < 4 else -1 for o in of])
    want = osv.lora(_f64(x), _f64(A), _f64(B), scale.numpy(), ids, _f64(y))
    xs = torch.full((T, K + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    xs[:, :K] = x.cuda()
    ys, outs = (torch.full((T, N + 5), 7.0, device="cuda") for _ in range(2))
    ys[:, :N] = y.cuda()
    sf.lora_add(xs[:, :K], A.cuda(), B.cuda(), scale.cuda(), _i32(per), outs[:, :N], ys[:, :N], row_of=_i32(of))
    tol = _lora_tol(_f64(x), _f64(A), _f64(B), scale.numpy(), ids, want, K, rank)
    assert np.all(np.abs(_f64(outs[:, :N]) - want) <= tol) and torch.all(outs[:, N:] == 7.0)


def test_lora_prompts_of_one_adapter(sf):
    """Whole windows of one adapter, and of none."""
    T, K, N, rank, n = 900, 320, 260, 32, 4
    x, A, B, scale, y = _lora_case(T, K, N, rank, n, 4)
    ids = np.repeat([2, -1, 0, 3, 2], [301, 150, 17, 400, 32])
    want = osv.lora(_f64(x), _f64(A), _f64(B), scale.numpy(), ids, _f64(y))
    out = sf.lora_add(x.cuda(), A.cuda(), B.cuda(), scale.cuda(), _i32(ids), torch.full((T, N), 7.0, device="cuda"),
                      y.cuda())
    tol = _lora_tol(_f64(x), _f64(A), _f64(B), scale.numpy(), ids, want, K, rank)
    assert np.all(np.abs(_f64(out) - want) <= tol)


def test_lora_nonfinite_stays_in_its_row_and_adapter(sf):
    T, K, N, rank, n = 20, 128, 64, 8, 3
    x, A, B, scale, y = _lora_case(T, K, N, rank, n, 5)
    ids = np.arange(T) % n
    clean = sf.lora_add(x.cuda(), A.cuda(), B.cuda(), scale.cuda(), _i32(ids), torch.empty((T, N), device="cuda"),
                        y.cuda())
    x[4, 7] = float("nan")
    A[2, 3, 5] = float("inf")
    B[2, 9, 1] = float("nan")
    out = sf.lora_add(x.cuda(), A.cuda(), B.cuda(), scale.cuda(), _i32(ids), torch.empty((T, N), device="cuda"),
                      y.cuda())
    ok = [t for t in range(T) if t != 4 and ids[t] != 2]
    assert torch.equal(out[ok], clean[ok]) and torch.isnan(out[4]).all()


@pytest.mark.parametrize("rank", [8, 24, 72])
def test_lora_infinite_inputs(sf, rank):
    """An infinite A x gives what the formula gives: infinities of B's signs, NaN where they cancel."""
    x, A, B, scale, y = _lora_case(3, 64, 40, rank, 1, 9)
    A, B = A.abs() + 1.0, B.abs() + 1.0
    B[0, 7], B[0, 9, 2] = -B[0, 7], -1.0
    x[1, 9], x[2, 3], x[2, 50] = float("-inf"), float("inf"), float("-inf")
    out = _f64(sf.lora_add(x.cuda(), A.cuda(), B.cuda(), scale.cuda(), _i32([0, 0, 0]), y=y.cuda()))
    want = np.full(40, -np.inf)
    want[7], want[9] = np.inf, np.nan
    assert np.isfinite(out[0]).all() and np.isnan(out[2]).all()
    np.testing.assert_array_equal(out[1], want)


def test_lora_repeats_bit_for_bit_in_a_graph(sf):
    T, K, N, rank, n = 24, 2048, 1000, 16, 6
    x, A, B, scale, y = _lora_case(T, K, N, rank, n, 6)
    ids = _i32(np.arange(T) % n)
    args = [t.cuda() for t in (x, A, B, scale)]
    out = torch.empty((T, N), device="cuda")
    job = sf.LoraAdd(*args, ids, out, y.cuda())
    job.run()
    first = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        job.run()
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)


def test_lora_forks_and_joins_in_a_graph(sf):
    """Calls of two streams that wait for one another, eager and captured: each sees what both streams wrote before it."""
    T, K, N, rank, n = 16, 512, 512, 16, 4
    x, A, B, scale, y = _lora_case(T, K, N, rank, n, 8)
    ids = _i32(np.arange(T) % n)
    A, B, scale = A.cuda(), B.cuda(), scale.cuda()
    x, y0, y1, y2 = x.cuda(), y.cuda(), torch.empty((T, N), device="cuda"), torch.empty((T, N), device="cuda")
    x1, x2 = torch.empty_like(x), torch.empty_like(x)
    first, left, right, last = (sf.LoraAdd(a, A, B, scale, ids, out, src) for a, out, src in
                                ((x, y1, y0), (x1, y1, y1), (x1, y2, y0), (x2, y1, y2)))
    side = torch.cuda.Stream()

    def step():
        main = torch.cuda.current_stream()
        first.run()
        x1.copy_(y1)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            right.run()
        left.run()
        x2.copy_(y1)
        main.wait_stream(side)
        last.run()

    side.wait_stream(torch.cuda.current_stream())
    one = sf.lora_add(x, A, B, scale, ids, torch.empty_like(y1), y0)
    b1 = one.to(torch.bfloat16)
    two = sf.lora_add(b1, A, B, scale, ids, torch.empty_like(y1), one)
    three = sf.lora_add(b1, A, B, scale, ids, torch.empty_like(y1), y0)
    want = sf.lora_add(two.to(torch.bfloat16), A, B, scale, ids, torch.empty_like(y1), three)
    for _ in range(3):
        step()
        torch.cuda.synchronize()
        assert torch.equal(y1, want) and torch.equal(y2, three)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        step()
    for _ in range(3):
        y1.zero_(), y2.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y1, want) and torch.equal(y2, three)


# ---- a step of all of them -----------------------------------------------------------


def test_steps_together(sf):
    """Three steps of a small batch: plan, the q/k/v projection through 2+2-bit weights with per-request adapters, append
    with RoPE, attention; against the oracle on the same projections."""
    rng = np.random.default_rng(71)
    Hq, Hkv, d, H, P, R, MP, pages, rows = 4, 2, 64, 256, 16, 3, 6, 14, 16
    N = (Hq + 2 * Hkv) * d
    qw = sf.quantize_nested(_dev((rng.standard_normal((N, H)) * 0.05).astype(np.float32)), 64, 2, 2)
    _, A, B, scale, _ = _lora_case(1, H, N, 8, 2, 72)
    B = (B.float() * 0.1).to(torch.bfloat16)
    d_lens, d_n = _i32([0] * R), _i32([pages])
    table, free = torch.full((R, MP), -1, dtype=torch.int32, device="cuda"), _i32(np.arange(pages))
    keep, add, adapters = _i32([0] * R), _i32([0] * R), _i32([1, -1, 0])
    plan = sf.PagedPlan(d_lens, add, table, free, d_n, P, rows, keep=keep)
    kv = sf.PagedKV.empty(pages, Hkv, P, d)
    qkv = torch.zeros((rows, N), device="cuda")
    x = torch.zeros((rows, H), dtype=torch.bfloat16, device="cuda")
    q, k, v = (qkv[:, a * d:b * d].unflatten(1, (b - a, d)) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, N // d)))
    lora = sf.LoraAdd(x, A.cuda(), B.cuda(), scale.cuda(), adapters, y=qkv, row_of=plan.row_request)
    append = sf.PagedAppend(kv, k, v, plan.slots, plan.positions, 10000.0, q)
    attn = sf.PagedAttention(append.q_out, kv, plan.cu_rows, d_lens, table)
    pool = np.zeros((2, pages, Hkv, P, d))
    st = dict(lens=[0] * R, table=[[-1] * MP] * R, free=list(range(pages)))
    for keeps, adds in (([0, 0, 0], [9, 5, 0]), ([9, 5, 0], [1, 1, 12]), ([8, 0, 12], [3, 7, 1])):
        keep.copy_(_i32(keeps))
        add.copy_(_i32(adds))
        x.copy_(torch.from_numpy(rng.standard_normal((rows, H)).astype(np.float32)))
        before = attn.out.clone()
        plan.run()
        sf.gemv_refine(qw, x, y=qkv)
        lora.run()
        append.run()
        attn.run()
        torch.cuda.synchronize()
        st = osv.plan(st["lens"], keeps, adds, st["table"], st["free"], pages, P, rows)
        T = st["cu"][-1]
        assert plan.slots.tolist() == st["slots"] and d_lens.tolist() == st["lens"]
        base = sf.gemv_refine(qw, x)
        ids = [[1, -1, 0][i] for i in st["request"][:T]]
        want = osv.lora(_f64(x)[:T], _f64(A), _f64(B), scale.numpy(), ids, _f64(base)[:T])
        np.testing.assert_allclose(_f64(qkv)[:T], want, atol=2.0 ** -17 * np.abs(want).max())
        rot = osv.rope_rows(_f64(k)[:T], st["positions"][:T], 10000.0).astype(np.float32)
        for w, vals in ((0, rot), (1, _f64(v)[:T].astype(np.float32))):
            got = osv.values(*osv.quantize_rows(vals))
            for t in range(T):
                pool[w, st["slots"][t] // P, :, st["slots"][t] % P] = got[t]
        qr = oattn.bf16_to_f64(odec.f64_to_bf16_bits(osv.rope_rows(_f64(q)[:T], st["positions"][:T], 10000.0)))
        ref = osv.attention(qr, pool[0], pool[1], st["cu"], st["lens"], st["table"])
        # q differs from the oracle's by a bf16 rounding where fp64 values straddle one: rarely, and by 2^-7 of an entry
        assert np.abs(_f64(attn.out)[:T] - ref).max() <= 2e-4 * np.abs(pool[1]).max()
        assert torch.equal(attn.out[T:], before[T:])      # rows behind the step's last stay as they were
