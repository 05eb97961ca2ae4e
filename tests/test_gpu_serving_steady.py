"""Attention over the paged cache where every warp works through several stages,
for each kernel that the sizes choose, against a plain form in 64 bits.

A few real pages serve many table entries, so that the caches are long and the
reference stays cheap.  Keys' and values' sizes grow and fall from page to page,
so that the softmax references and the values' power of two change inside a
warp's run; short and long requests alternate, so that a run holds the end of
one segment, whole ones and the start of another.

Tolerance, per output, with s_t = scale (q . k_t), p_t the softmax weights, c_t,
z_t and k_s,t (v_s,t) a token's code, zero point and scale:
  score   q enters with 22 bits of its row's largest entry: 2^-22 max|q| |k_t|_1
          scale; the sum of X c is put together in fp32 by three operations,
          the zero point's part is a fourth, the two scales two more: 6 2^-24 of
          scale ks (|sum q c| + |z sum q|) + |s_t|; minus the reference 2^-24
          (|s_t| + |s_max| + 8);
  weight  relatively the score's error, 2^-21 (exponential) and 2^-21 (pairs of
          f16); an output moves by sum p_t e_t |v_t - out|, at most.  The smaller
          f16 ends at 2^-24, so a product p v_s is also off by up to 2^-25 (and
          at most by itself) where the largest v_s is scaled to 2^10 or more and
          the largest weight is 2^-2 or more: 2^-33 max v_s of the normalised
          one, times |c - 8| <= 8;
  sums    of w (c - 8) and w (z - 8), at most 256 fp32 additions in a row: 2^-24
          256 sum p_t v_s (|c - 8| + |z - 8|), and as much of the output for the
          sum of weights.
bf16: half a step more, 2^-8 of the value.
"""

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


def _i32(a):
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()


LEVELS = 6  # sizes of keys and values, a page kind each


class Cache:
    """Requests over a pool of 4 LEVELS pages (every kind four times); page j of a
    request is of the kind that a triangle wave says, so sizes grow and fall."""

    def __init__(self, sf, seed, n, lens, Hq, Hkv, d, P, extra_rows=1, k_step=1.5, v_step=2.5):
        rng = np.random.default_rng(seed)
        self.n, self.lens, self.P = n, lens, P
        pages = 4 * LEVELS
        kind = np.arange(pages) % LEVELS
        codes, param = [], []
        for step in (k_step, v_step):
            x = rng.standard_normal((pages, Hkv, P, d)) * (0.7 * step ** kind)[:, None, None, None]
            c, s, z = osv.quantize_rows(x.astype(np.float32))
            w = (c.reshape(*c.shape[:-1], -1, 8).astype(np.uint32) << (4 * np.arange(8, dtype=np.uint32))).sum(
                -1, dtype=np.uint32)
            codes.append((torch.from_numpy(c).cuda(), torch.from_numpy(w.view(np.int32)).cuda()))
            param.append(torch.from_numpy(np.stack([s, z], -1)).cuda())
        self.c, self.p = [c for c, _ in codes], param
        self.kv = sf.PagedKV(codes[0][1], param[0], codes[1][1], param[1])
        most = max(-(-x // P) for x in lens) + 1
        table = np.full((len(lens), most), pages + 3, np.int64)
        for i, x in enumerate(lens):
            j = np.arange(-(-x // P)) + 3 * i
            wave = np.abs((j + LEVELS - 1) % (2 * LEVELS - 2) - (LEVELS - 1))
            table[i, :len(j)] = wave + LEVELS * rng.integers(0, 4, len(j))
        self.table = table
        self.cu = np.concatenate([[0], np.cumsum(n)])
        self.T = int(self.cu[-1]) + extra_rows
        self.q = torch.from_numpy(rng.standard_normal((self.T, Hq, d)).astype(np.float32)).to(torch.bfloat16).cuda()

    def run(self, sf, dtype, window=0):
        out = torch.full(self.q.shape, 7.0, dtype=dtype, device="cuda")
        return sf.attn_paged(self.q, self.kv, _i32(self.cu), _i32(self.lens), _i32(self.table), out, window=window)

    def exact(self, window=0):
        """The outputs in 64 bits and how far an fp32 result may be off."""
        T, Hq, d = self.q.shape
        Hkv = self.c[0].shape[1]
        g, scale = Hq // Hkv, 1.0 / np.sqrt(d)
        want = torch.full((T, Hq, d), 7.0, dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(want)
        for i, L in enumerate(self.lens):
            n = self.n[i]
            if n == 0:
                continue
            tok = np.arange(L)
            pg, off = torch.from_numpy(self.table[i, tok // self.P]).cuda(), torch.from_numpy(tok % self.P).cuda()
            for h in range(Hkv):
                (kc, ks, kz), (vc, vs, vz) = (
                    (self.c[w][pg, h, off].double(), *(self.p[w][pg, h, off].double()[:, z] for z in (0, 1)))
                    for w in (0, 1))
                q = self.q[self.cu[i]:self.cu[i + 1], h * g:(h + 1) * g].double()        # [n][g][d]
                qc, qs = q @ kc.t(), q.sum(-1, keepdim=True)
                s = scale * ks * (qc - kz * qs)
                e = scale * 2.0 ** -22 * q.abs().amax(-1, keepdim=True) * (ks * (kc - kz[:, None]).abs().sum(-1)) \
                    + 6 * 2.0 ** -24 * (scale * ks * (qc.abs() + (kz * qs).abs()) + s.abs())
                at = torch.arange(L - n, L, device="cuda")[:, None, None]
                t = torch.arange(L, device="cuda")
                see = t <= at
                if window:
                    see &= t > at - window
                s = torch.where(see, s, -torch.inf)
                top = s.amax(-1, keepdim=True)
                p = torch.where(see, torch.exp(s - top.clamp(min=-1e300)), 0.0)
                p /= p.sum(-1, keepdim=True).clamp(min=1e-300)
                v = vs[:, None] * (vc - vz[:, None])
                o = p @ v
                e = torch.where(see, e + 2.0 ** -24 * (s.abs() + top.abs() + 8) + 2.0 ** -20, 0.0)
                # sum p e |v - o| <= sum p e |v| + sum p e |o|
                pe = p * e
                size = vs[:, None] * ((vc - 8).abs() + (vz[:, None] - 8).abs())
                x = pe @ v.abs() + pe.sum(-1, keepdim=True) * o.abs() + 256 * 2.0 ** -24 * (p @ size + o.abs())
                x += 8 * torch.minimum(p * vs, 2.0 ** -33 * vs.max()).sum(-1, keepdim=True)
                want[self.cu[i]:self.cu[i + 1], h * g:(h + 1) * g] = o
                tol[self.cu[i]:self.cu[i + 1], h * g:(h + 1) * g] = x
        return want, tol


def _mixed(rng, longs, shorts):
    """Long requests with runs of short ones before and after each."""
    lens = []
    for x in longs:
        lens += rng.integers(1, 400, shorts).tolist() + [x]
    return lens + rng.integers(1, 400, shorts).tolist()


# d, query heads, KV heads, page size, rows of a request: 4 (packed), 8 and 16 columns
KERNELS = [(64, 16, 4, 64, 1), (64, 24, 4, 16, 1), (64, 40, 4, 256, 1), (64, 12, 4, 64, 4),
           (128, 16, 4, 64, 1), (128, 10, 5, 16, 1), (128, 32, 4, 128, 1), (128, 16, 4, 16, 4), (128, 48, 4, 64, 1),
           (256, 8, 2, 64, 1), (256, 12, 2, 16, 1), (256, 16, 2, 32, 2)]


@pytest.mark.parametrize("d,Hq,Hkv,P,rows", KERNELS)
def test_several_stages_a_warp(sf, d, Hq, Hkv, P, rows):
    rng = np.random.default_rng(d + Hq + rows)
    lens = _mixed(rng, [30011, 60000, 8200, 14021], 9)
    n = [int(min(x, rng.integers(1, rows + 1))) for x in lens]
    c = Cache(sf, 3, n, lens, Hq, Hkv, d, P)
    cols = 16 if Hq // Hkv * rows > 8 and d < 256 else 8 if Hq // Hkv * rows > 4 else 4
    tok, warps = (32, 8) if d == 256 else (64, 12 if d == 64 and cols < 16 else 8)
    units = sum(-(-k * (Hq // Hkv) // cols) * Hkv * -(-x // tok) for k, x in zip(n, lens))
    assert units >= 3 * warps * torch.cuda.get_device_properties(0).multi_processor_count
    want, tol = c.exact()
    out = c.run(sf, torch.float32)
    live = int(c.cu[-1])
    err = (out.double() - want).abs()
    print("largest error", err[:live].max().item(), "of its tolerance", (err / tol)[:live].nan_to_num().max().item(),
          "tolerance over the largest value", (tol[:live].max() / want[:live].abs().max()).item())
    assert torch.all(err <= tol)
    assert torch.all(out[live:] == 7.0)


@pytest.mark.parametrize("d,Hq,Hkv,P,rows", [KERNELS[0], KERNELS[6], KERNELS[7], KERNELS[9]])
def test_several_stages_a_warp_with_a_window(sf, d, Hq, Hkv, P, rows):
    rng = np.random.default_rng(d + Hq + rows + 1)
    lens = _mixed(rng, [30011, 9000, 40000], 7)
    c = Cache(sf, 4, [int(min(x, rng.integers(1, rows + 1))) for x in lens], lens, Hq, Hkv, d, P)
    want, tol = c.exact(window=5003)
    out = c.run(sf, torch.float32, window=5003)
    assert torch.all((out.double() - want).abs() <= tol)


@pytest.mark.parametrize("d,Hq,Hkv,P,rows", KERNELS)
def test_bf16_outputs_are_the_fp32_ones_rounded(sf, d, Hq, Hkv, P, rows):
    """Nothing but the last rounding depends on the output's type: long caches, and queries and keys whose largest
    channels are some hundred times the others."""
    rng = np.random.default_rng(d + Hq + rows + 2)
    lens = _mixed(rng, [20011, 30000], 5)
    c = Cache(sf, 5, [int(min(x, rng.integers(1, rows + 1))) for x in lens], lens, Hq, Hkv, d, P, k_step=1.2)
    for outliers in (False, True):
        if outliers:
            c.q[:, :, 3] *= 300.0
            c.p[0][..., 0] *= 0.01                        # (scores of the same size as before)
        want = c.run(sf, torch.float32)
        assert torch.equal(c.run(sf, torch.bfloat16), want.to(torch.bfloat16))
        exact, tol = c.exact()
        assert torch.all((want.double() - exact).abs() <= tol)
