"""The serving operators at the ends of their ranges: page numbers that no pool
has, plans made by several host threads, rotations bit by bit, token-heads of
every size, long inner loops of the adapters, values near the largest float."""

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


# ---- adapters --------------------------------------------------------------------


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
