"""The serving operators at the ends of their ranges: page numbers that no pool
has, plans made by several host threads, rotations bit by bit, token-heads of
every size, long inner loops of the adapters, values near the largest float,
captured steps."""

import threading

import numpy as np
import pytest
import torch

from oracle import serving as osv

pytestmark = pytest.mark.gpu


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


def _to_bf16(a):
    """fp64 rounded once to bf16 (ties to even, subnormals of steps 2^-133), as fp64."""
    step = np.maximum(np.frexp(a)[1] - 8, -133)
    return np.ldexp(np.rint(np.ldexp(a, -step)), step)


# ---- plan ------------------------------------------------------------------------


@pytest.mark.parametrize("P", [16, 64, 256])
def test_plan_page_numbers_that_no_pool_has(sf, P):
    """A table or free-list entry whose tokens' slots would not fit 32 bits gives slots of -1, never another page's."""
    first = 2 ** 31 // P                                  # (2^31 / P) P + 16 would come out as slot 16
    bad = [first, first + 1, 2 ** 31 - 1, -(2 ** 31), -1, -first]
    table = np.array([[b, first - 1] for b in bad])
    lens, add = [P // 2] * len(bad), [P // 2 + 2] * len(bad)    # rows on the first page and, from the list, the second
    free = bad[::-1]
    want = osv.plan(lens, lens, add, table.tolist(), free, 8, P, 2048)
    job = sf.paged_plan(_i32(lens), _i32(add), _i32(table), _i32(free + [0, 0]), _i32([len(free)]), P, 2048)
    assert int(job.status.item()) == osv.PLAN_OK
    assert job.slots.tolist() == want["slots"] == [-1] * 2048
    assert job.positions.tolist() == want["positions"] and job.row_request.tolist() == want["request"]
    # the last page that there can be
    last = sf.paged_plan(_i32([P - 1]), _i32([1]), _i32([[first - 1]]), _i32([0]), _i32([0]), P, 1)
    assert last.slots.tolist() == [2 ** 31 - 1]


@pytest.mark.parametrize("in_place", [False, True])
def test_plan_negative_free_count(sf, in_place):
    """Refused on the device like any other plan: every output as it has to be, inputs as they were."""
    lens, add, table, free, rows = [40, 20, 0], [1, 1, 1], [[3, 5, 1, -1], [0, 2, -1, -1], [-1] * 4], [4, 6, 7], 8
    d_lens, d_n, tab, lst = _i32(lens), _i32([-1]), _i32(table), _i32(free)
    kw = {} if in_place else dict(lens_out=torch.full_like(d_lens, -9), n_free_out=torch.full_like(d_n, -9))
    job = sf.paged_plan(d_lens, _i32(add), tab, lst, d_n, 16, rows, **kw)
    assert int(job.status.item()) == osv.PLAN_PAGES
    assert job.lens_out.tolist() == lens and d_lens.tolist() == lens
    assert job.n_free_out.tolist() == [-1] and d_n.tolist() == [-1]
    assert tab.tolist() == table and lst.tolist() == free and job.cu_rows.tolist() == [0] * 4
    assert job.slots.tolist() == [-1] * rows and job.positions.tolist() == [0] * rows
    assert job.row_request.tolist() == [-1] * rows


def test_plans_of_several_host_threads(sf):
    """Plans of different sizes made at once: each call's shared memory is its own."""
    P, errors = 16, []

    def loop(R):
        try:
            lens = _i32([0] * R)
            with torch.cuda.stream(torch.cuda.Stream()):
                job = sf.PagedPlan(lens, _i32([1] * R), _i32(np.full((R, 2), -1)), _i32(np.arange(R)), _i32([R]), P, R,
                                   lens_out=torch.empty_like(lens), n_free_out=_i32([0]))
                for _ in range(3000):
                    job.run()
        except Exception as e:  # noqa: BLE001 - handed to the test
            errors.append(e)

    threads = [threading.Thread(target=loop, args=(R,)) for R in (2600, 8192, 4000, 6000)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors[0]


# ---- append ----------------------------------------------------------------------


def test_calls_without_rows(sf):
    """T = 0, an append with queries and without, attention, adapters: nothing to do."""
    kv = sf.PagedKV.empty(2, 2, 16, 64)
    k = torch.zeros((0, 2, 64), device="cuda")
    q = torch.zeros((0, 4, 64), device="cuda")
    none = _i32(np.zeros(0))
    assert sf.paged_append(kv, k, k, none) is None
    out = sf.paged_append(kv, k, k, none, none, 10000.0, q)
    assert out.shape == (0, 4, 64) and torch.all(kv.k_param == 0)
    got = sf.attn_paged(out, kv, _i32([0, 0]), _i32([0]), _i32([[0]]))
    assert got.shape == (0, 4, 64)
    x, A, B = (torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((0, 16), (1, 8, 16), (1, 5, 8)))
    assert sf.lora_add(x, A, B, torch.ones(1, device="cuda"), none).shape == (0, 5)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("src", ["fp32", "bf16"])
@pytest.mark.parametrize("gain", [1.0, 1e-36, 1e30])
def test_append_rotates_queries_to_the_bit(sf, d, src, gain):
    """q_out is the fp64 rotation rounded once to bf16.  An angle is off by its own rounding (positions below 2^20: 2^-33,
    twice for two implementations), an entry by 2^-31 of its pair's size at most: between the two ends' roundings."""
    T, Hq, theta = 700, 8, 500000.0
    g = torch.Generator().manual_seed(d)
    q = (torch.randn((T, Hq, d), generator=g) * gain).to(torch.float32 if src == "fp32" else torch.bfloat16)
    pos = np.random.default_rng(d).integers(0, 1 << 20, T).astype(np.int32)
    pos[:3] = 0, 1, 2 ** 20 - 1
    kv = sf.PagedKV.empty(-(-T // 16), 1, 16, d)
    k = torch.zeros((T, 1, d), dtype=q.dtype, device="cuda")
    got = sf.paged_append(kv, k, k, _i32(np.arange(T)), _i32(pos), theta, q.cuda())
    x, got = _f64(q), _f64(got)
    want = osv.rope_rows(x, pos, theta)
    size = np.abs(x[..., :d // 2]) + np.abs(x[..., d // 2:])
    e = 2.0 ** -31 * np.concatenate([size, size], -1)
    lo, hi = _to_bf16(want - e), _to_bf16(want + e)
    assert np.mean(lo != hi) < 1e-5
    assert np.all((got >= lo) & (got <= hi))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_append_quantizes_every_size(sf, d):
    """Token-heads from 2^-40 to 2^40, offset to either side, constant ones, one entry apart, spans that overflow: codes,
    scales and zero points are the quantizer's."""
    rng = np.random.default_rng(d)
    rows = []
    for e in range(-40, 41, 2):
        z = rng.standard_normal((5, d))
        z[1] += 30.0
        z[2] -= 30.0
        z[3] = 1.0
        z[4] = 0.0
        z[4, 5] = 1.0
        rows.append(z * 2.0 ** e)
    rows.append(np.where(np.arange(d) % 2, 3e38, -3e38)[None])
    rows.append(np.full((1, d), -1e-42))
    x = np.concatenate(rows).astype(np.float32)
    T = len(x)
    kv = sf.PagedKV.empty(-(-T // 16), 1, 16, d)
    xd = _dev(x[:, None])
    sf.paged_append(kv, xd, xd, _i32(np.arange(T)))
    with np.errstate(over="ignore"):
        c, s, z = osv.quantize_rows(x)
    for codes, param in ((kv.k_codes, kv.k_param), (kv.v_codes, kv.v_param)):
        w = codes.reshape(-1, d // 8)[:T].cpu().numpy().view(np.uint32)
        got = ((w[..., None] >> (4 * np.arange(8, dtype=np.uint32))) & 15).reshape(T, d)
        p = param.reshape(-1, 2)[:T].cpu().numpy()
        np.testing.assert_array_equal(p[:, 0], s)
        np.testing.assert_array_equal(p[:, 1], z)
        np.testing.assert_array_equal(got, c)


# ---- adapters --------------------------------------------------------------------


def _lora(T, K, N, rank, n, seed, positive=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, A, B = (torch.randn(s, generator=g, device="cuda") for s in ((T, K), (n, rank, K), (n, N, rank)))
    if positive:
        x, A = x.abs(), A.abs()
    return (x.to(torch.bfloat16), (A / K ** 0.5).to(torch.bfloat16), B.to(torch.bfloat16),
            torch.rand(n, generator=g, device="cuda") + 0.5, torch.randn((T, N), generator=g, device="cuda"))


def _lora_exact(x, A, B, scale, ids, y):
    """The formula in 64 bits, and the same of absolute values."""
    out, size = y.double(), torch.zeros(y.shape, dtype=torch.float64, device="cuda")
    for a in range(len(A)):
        rows = (ids == a).nonzero()[:, 0]
        for at, f in ((out, lambda t: t.double()), (size, lambda t: t.double().abs())):
            at[rows] += f(scale[a]) * ((f(x[rows]) @ f(A[a]).t()) @ f(B[a]).t())
    return out, size


@pytest.mark.parametrize("positive", [False, True])
@pytest.mark.parametrize("T,K,N,rank,n,runs", [
    # several steps of a warp's part of K
    (3, 12288, 200, 16, 2, 1), (9, 12296, 96, 32, 3, 1), (20, 16384, 40, 64, 4, 1), (2, 14336, 64, 128, 1, 1),
    # so many rows that a cluster has two blocks, and one
    (2400, 2048, 96, 32, 4, 100), (2401, 2056, 36, 72, 3, 7), (4801, 12288, 40, 16, 5, 300), (4777, 2048, 64, 64, 3, 1),
    (4900, 2048, 40, 128, 4, 50)])
def test_lora_long_loops_and_small_clusters(sf, T, K, N, rank, n, runs, positive):
    """A sum over K runs through at most K/16 tensor-core products (truncated: 2^-23 of the sum each) and 72 partial sums,
    the second product through 3 rank/16 and the output's own: 2^-24 (|out| + (K/8 + rank/2 + 80) M), M the formula of
    absolute values."""
    x, A, B, scale, y = _lora(T, K, N, rank, n, T + K, positive)
    ids = _i32(np.repeat(np.random.default_rng(T).integers(-1, n, T), runs)[:T])
    out = sf.lora_add(x, A, B, scale, ids, torch.full((T, N), 7.0, device="cuda"), y)
    want, size = _lora_exact(x, A, B, scale, ids, y)
    err = (out.double() - want).abs()
    print("error over the formula of absolute values", (err / (size + want.abs()).clamp(min=1e-30)).max().item())
    assert torch.all(err <= 2.0 ** -24 * (want.abs() + (K / 8 + rank / 2 + 80) * size))


@pytest.mark.parametrize("rank", [8, 24, 128])
def test_lora_near_the_largest_float(sf, rank):
    """scale A x between the largest bf16 and the largest fp32 value: finite outputs stay finite."""
    K, N = 64, 40
    x = torch.zeros((2, K), dtype=torch.bfloat16)
    A = torch.zeros((1, rank, K), dtype=torch.bfloat16)
    B = torch.zeros((1, N, rank), dtype=torch.bfloat16)
    x[:, 3] = torch.tensor([1.0, -1.0])
    A[0, 5, 3] = 2.0 ** 127
    B[0, :, 5] = torch.linspace(-0.5, 0.5, N).to(torch.bfloat16)
    scale = torch.tensor([1.9999])
    out = sf.lora_add(x.cuda(), A.cuda(), B.cuda(), scale.cuda(), _i32([0, 0]), y=torch.zeros((2, N), device="cuda"))
    want = x[:, 3:4].double() * scale.double() * 2.0 ** 127 * B[0, :, 5].double()
    assert torch.all((out.cpu().double() - want).abs() <= 2.0 ** -22 * want.abs())


# ---- a step of all of them, captured -------------------------------------------------


def test_captured_steps_equal_eager_ones(sf):
    """Plan, adapters, append with RoPE and attention of a decode loop, replayed from one graph as often as called one by
    one: the same lengths, pages, pool and outputs, bit for bit, in a batch padded to twice its rows."""
    Hq, Hkv, d, H, P, R, MP, rows, pages = 8, 2, 128, 256, 16, 5, 12, 40, 64
    N = (Hq + 2 * Hkv) * d
    x, A, B, scale, _ = _lora(rows, H, N, 16, 3, 90)
    base = torch.randn((rows, N), generator=torch.Generator(device="cuda").manual_seed(91), device="cuda")
    ids = _i32([2, -1, 0, 1, 2])

    class Loop:
        def __init__(self):
            self.lens, self.n_free = _i32([0] * R), _i32([pages])
            self.table, self.free = _i32(np.full((R, MP), -1)), _i32(np.arange(pages))
            self.keep, self.add = _i32([0] * R), _i32([0] * R)
            self.plan = sf.PagedPlan(self.lens, self.add, self.table, self.free, self.n_free, P, rows, keep=self.keep)
            self.kv = sf.PagedKV.empty(pages, Hkv, P, d)
            self.qkv = torch.zeros((rows, N), device="cuda")
            q, k, v = (self.qkv[:, a * d:b * d].unflatten(1, (b - a, d)) for a, b in
                       ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, N // d)))
            self.lora = sf.LoraAdd(x, A, B, scale, ids, self.qkv, base, row_of=self.plan.row_request)
            self.append = sf.PagedAppend(self.kv, k, v, self.plan.slots, self.plan.positions, 10000.0, q,
                                         torch.zeros((rows, Hq, d), dtype=torch.bfloat16, device="cuda"))
            self.attn = sf.PagedAttention(self.append.q_out, self.kv, self.plan.cu_rows, self.lens, self.table)

        def step(self):
            for job in (self.plan, self.lora, self.append, self.attn):
                job.run()

        def state(self):
            kv = self.kv
            return (self.lens, self.n_free, self.table, self.plan.slots, self.plan.status, self.qkv, self.append.q_out,
                    kv.k_codes, kv.k_param, kv.v_codes, kv.v_param, self.attn.out)

    eager, replayed = Loop(), Loop()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        replayed.step()
    lens = [0] * R
    rng = np.random.default_rng(92)
    for _ in range(12):
        keep = [int(n if rng.random() < 0.7 else rng.integers(0, n + 1)) for n in lens]
        add = [int(min(rng.integers(0, 5), MP * P - k)) for k in keep]
        for loop in (eager, replayed):
            loop.keep.copy_(_i32(keep))
            loop.add.copy_(_i32(add))
        eager.step()
        graph.replay()
        torch.cuda.synchronize()
        lens = [k + a for k, a in zip(keep, add)]
        assert eager.lens.tolist() == lens
        for a, b in zip(eager.state(), replayed.state()):
            assert torch.equal(a, b)
