"""The paged 4-bit serving operators: what is measured, and their plain forms.

Four operators that a decode or prompt step of several requests runs:

  plan    block tables and slot maps from the requests' lengths
  append  RoPE of a step's queries and keys, K and V quantized to 4 bits and written to their slots
  attn    attention of every request's rows over its 4-bit pages
  lora    per-request low-rank adapters added to a shared projection's output

``run`` computes them with elementary torch operations where ``own`` is false, and calls the library where it is true.
Shapes are those of the Llama-3.1-8B and Qwen3-8B layers that the repository's workloads use (32 query and 8 KV heads
of 128, hidden 4096, MLP 14336 and 12288), and generic ones beside them.
"""

import math

import numpy as np
import torch

own = False

_DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
_THETA = 500000.0


def listed():
    return [
        # one more token for each of 16 requests: the step of a small decode batch, where latency is all
        dict(name="plan_decode_16", op="plan", R=16, P=64, max_pages=256, max_rows=16, mix="decode"),
        # a large server's step: finished requests leave, prompts arrive, speculated tokens are taken back
        dict(name="plan_mixed_1000", op="plan", R=1000, P=16, max_pages=512, max_rows=65536, mix="mixed"),
        # the rows of a 16-request decode step, straight from the fp32 q/k/v projections
        dict(name="append_decode_16", op="append", T=16, Hq=32, Hkv=8, d=128, P=64, pages=512, src="fp32", rope=True),
        # a long prompt's chunk (an odd number of rows), rotated and appended; as in the other two, the values that the
        # pages then hold come back in bf16 (what dense attention over the chunk reads)
        dict(name="append_prompt_4099", op="append", T=4099, Hq=32, Hkv=8, d=128, P=64, pages=96, src="fp32",
             rope=True),
        # bf16 rows that are rotated already (a cache rebuilt from another engine's values), heads of 64
        dict(name="append_bf16_d64_1500", op="append", T=1500, Hq=0, Hkv=8, d=64, P=16, pages=128, src="bf16",
             rope=False),
        # one short conversation: the smallest attention call
        dict(name="attn_1x500", op="attn", R=1, rows=1, lo=500, hi=500, Hq=32, Hkv=8, d=128, P=64, window=0,
             out="bf16"),
        # an ordinary decode batch: 16 requests of ragged lengths
        dict(name="attn_16x8k", op="attn", R=16, rows=1, lo=200, hi=8191, Hq=32, Hkv=8, d=128, P=64, window=0,
             out="fp32"),
        # one request at 128K tokens: the work has to be split along the cache
        dict(name="attn_1x128k", op="attn", R=1, rows=1, lo=131072, hi=131072, Hq=32, Hkv=8, d=128, P=128, window=0,
             out="fp32"),
        # 64 requests, each checking up to 4 speculated tokens, small pages: the largest call
        dict(name="attn_verify_64x8k", op="attn", R=64, rows=4, lo=1000, hi=12001, Hq=32, Hkv=8, d=128, P=16,
             window=0, out="bf16"),
        # a decode batch of 16 rows, each with an adapter of its own, beside the o or q projection
        dict(name="lora_decode_16", op="lora", T=16, K=4096, N=4096, rank=16, adapters=32, runs=1),
        # 64 rows beside the gate projection, larger adapters, a few rows without one
        dict(name="lora_gate_64", op="lora", T=64, K=4096, N=14336, rank=64, adapters=16, runs=1),
        # prompts of several requests packed in one batch beside the q projection
        dict(name="lora_prompt_2050", op="lora", T=2050, K=4096, N=4096, rank=32, adapters=8, runs=300),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "attn", "attn", "lora"])
    if op == "plan":
        mix = rng.choice(["decode", "mixed"])
        R = _log(rng, 1, 1000)
        return dict(op=op, R=R, P=rng.choice([16, 32, 64, 128]), max_pages=rng.randint(64, 512),
                    max_rows=R + rng.randint(0, 9) if mix == "decode" else 65536, mix=mix)
    if op == "append":
        T = _log(rng, 1, 4000)
        d, Hkv = rng.choice([64, 128, 128, 256]), rng.choice([1, 2, 4, 8])
        if d == 256:
            Hkv = min(Hkv, 4)
        P = rng.choice([16, 32, 64, 128])
        rope = rng.random() < 0.6
        return dict(op=op, T=T, Hq=Hkv * rng.choice([1, 2, 4]) if rope else 0, Hkv=Hkv, d=d, P=P,
                    pages=-(-T // P) + rng.randint(1, 40), src=rng.choice(["fp32", "bf16"]), rope=rope)
    if op == "attn":
        d = rng.choice([64, 128, 128, 128, 256])
        Hkv = rng.choice([1, 2, 4, 8, 8])
        group = rng.choice([1, 2, 4, 4, 5, 8])
        R = _log(rng, 1, 64)
        most = min(131072, 8192 * 64 * 8 * 128 // (2 * R * Hkv * d))
        hi = _log(rng, 16, most)
        rows = rng.choice([1, 1, 1, 2, 4, 7])
        if group * rows > 16 and hi * R * Hkv > 1 << 20:
            rows = 1
        return dict(op=op, R=R, rows=rows, lo=max(rows, hi // rng.randint(1, 20)), hi=max(hi, rows), Hq=Hkv * group,
                    Hkv=Hkv, d=d, P=rng.choice([16, 32, 64, 128]), window=rng.choice([0, 0, 0, _log(rng, 8, 4096)]),
                    out=rng.choice(["fp32", "bf16"]))
    T = _log(rng, 1, 1500)
    K, N = rng.choice([(4096, 4096), (4096, 1024), (4096, 12288), (2048, 1000), (520, 777), (12288, 4096)])
    if T > 128 and max(K, N) > 4096:
        T = 128
    return dict(op=op, T=T, K=K, N=N, rank=rng.choice([8, 16, 32, 64]), adapters=rng.randint(1, 16),
                runs=rng.choice([1, 1, 7, 100]))


# ---- inputs ------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 13)
    return g


def _quant4(x):
    """4-bit min-max quantization, one group per last axis: codes (int64), fp16 scale and zero."""
    lo, hi = x.amin(-1), x.amax(-1)
    fifteen = torch.full_like(lo, 15.0)
    s16 = torch.clamp((hi - lo) / fifteen, max=65504.0).to(torch.float16)
    s16 = torch.where(s16 == 0, torch.ones_like(s16), s16)
    s = s16.float()
    z = torch.clamp(torch.round(-lo / s), 0, 15) + 0.0
    c = torch.clamp(torch.round(x / s.unsqueeze(-1)) + z.unsqueeze(-1), 0, 15)
    return c.to(torch.int64), s16, z.to(torch.float16)


def _pack(c):
    """Codes [..., d] -> int32 words [..., d/8], code j at bits 4j of the row's little-endian stream."""
    c = c.reshape(*c.shape[:-1], -1, 8)
    w = (c << (4 * torch.arange(8, device=c.device))).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def _kv_pool(g, pages, Hkv, P, d):
    """Pages filled with quantized N(0, 1) keys (4 outlier channels per head x10) and values."""
    k_codes = torch.empty((pages, Hkv, P, d // 8), dtype=torch.int32, device="cuda")
    v_codes = torch.empty_like(k_codes)
    k_param = torch.empty((pages, Hkv, P, 2), dtype=torch.float16, device="cuda")
    v_param = torch.empty_like(k_param)
    gain = torch.ones((Hkv, d), device="cuda")
    gain.scatter_(1, torch.rand((Hkv, d), generator=g, device="cuda").argsort(1)[:, :4], 10.0)
    step = max(1, (1 << 26) // (Hkv * P * d))
    for at in range(0, pages, step):
        n = min(step, pages - at)
        for codes, param, by in ((k_codes, k_param, gain[:, None]), (v_codes, v_param, 1.0)):
            c, s, z = _quant4(torch.randn((n, Hkv, P, d), generator=g, device="cuda") * by)
            codes[at:at + n] = _pack(c)
            param[at:at + n, ..., 0] = s
            param[at:at + n, ..., 1] = z
    return k_codes, k_param, v_codes, v_param


def _plan_inputs(case, seed):
    rng = np.random.default_rng(seed)
    R, P, MP, rows = case["R"], case["P"], case["max_pages"], case["max_rows"]
    most = MP * P
    lens = rng.integers(0, most // 2 + 1, R)
    keep, add = lens.copy(), np.ones(R, np.int64)
    if case["mix"] == "mixed":
        kind = rng.random(R)
        gone = kind < 0.1                       # finished: its pages go back
        keep[gone], add[gone] = 0, 0
        new = (kind >= 0.1) & (kind < 0.2)      # the row now holds a new prompt
        keep[new] = 0
        add[new] = rng.integers(1, max(2, min(most, rows // max(1, R // 5)) // 2), int(new.sum()))
        spec = (kind >= 0.2) & (kind < 0.4)     # speculated tokens taken back, more proposed
        keep[spec] = np.maximum(0, lens[spec] - rng.integers(0, 8, int(spec.sum())))
        add[spec] = rng.integers(0, 6, int(spec.sum()))
    have = -(-lens // P)
    pages = R * MP
    perm = rng.permutation(pages).astype(np.int32)
    table = np.full((R, MP), -1, np.int32)
    used = 0
    for i in range(R):
        table[i, :have[i]] = perm[used:used + have[i]]
        used += have[i]
    free = np.full(pages, -1, np.int32)
    free[:pages - used] = perm[used:]
    dev = {k: torch.from_numpy(np.ascontiguousarray(v, np.int32)).cuda() for k, v in
           dict(lens=lens, keep=keep, add=add, table=table, free=free, n_free=np.array([pages - used])).items()}
    return dev


def _append_inputs(case, seed):
    g = _gen(seed)
    T, Hq, Hkv, d, P, pages = (case[k] for k in ("T", "Hq", "Hkv", "d", "P", "pages"))
    dt = _DT[case["src"]]
    # one fused projection output [T][(Hq + 2 Hkv) d], read as strided q, k and v
    qkv = torch.randn((T, (Hq + 2 * Hkv) * d), generator=g, device="cuda").to(dt)
    s = dict(q=qkv[:, :Hq * d].unflatten(1, (Hq, d)) if Hq else None,
             k=qkv[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d)),
             v=qkv[:, (Hq + Hkv) * d:].unflatten(1, (Hkv, d)))
    slots = torch.rand(pages * P, generator=g, device="cuda").argsort()[:T].to(torch.int32)
    if T >= 3:
        slots[T // 2] = -1                      # a padded row of the batch
    s["slots"] = slots
    s["positions"] = torch.randint(0, 131072, (T,), generator=g, device="cuda", dtype=torch.int32)
    for n in ("k", "v"):
        s[n + "_codes"] = torch.zeros((pages, Hkv, P, d // 8), dtype=torch.int32, device="cuda")
        s[n + "_param"] = torch.zeros((pages, Hkv, P, 2), dtype=torch.float16, device="cuda")
        s[n + "_val"] = torch.zeros((T, Hkv, d), dtype=torch.bfloat16, device="cuda")
    s["q_out"] = torch.zeros((T, Hq, d), dtype=torch.bfloat16, device="cuda") if case["rope"] else None
    return s


def _attn_inputs(case, seed):
    g = _gen(seed)
    rng = np.random.default_rng(seed)
    R, rows, Hq, Hkv, d, P = (case[k] for k in ("R", "rows", "Hq", "Hkv", "d", "P"))
    n = rng.integers(1, rows + 1, R)
    lens = np.maximum(rng.integers(case["lo"], case["hi"] + 1, R), n)
    if R >= 4:
        n[1] = lens[1] = 0                      # a row of the batch that holds no request
    lens[0] = max(case["hi"], n[0])
    used = -(-lens // P)
    pages = int(used.sum()) + 3
    perm = rng.permutation(pages).astype(np.int32)
    table = np.full((R, int(used.max()) + 1), -1, np.int32)
    at = 0
    for i in range(R):
        table[i, :used[i]] = perm[at:at + used[i]]
        at += used[i]
    cu = np.zeros(R + 1, np.int32)
    cu[1:] = np.cumsum(n)
    T = R * rows + (2 if R >= 4 else 0)         # the batch's room: there may be rows behind the last request
    k_codes, k_param, v_codes, v_param = _kv_pool(g, pages, Hkv, P, d)
    return dict(q=torch.randn((T, Hq, d), generator=g, device="cuda").to(torch.bfloat16),
                cu=torch.from_numpy(cu).cuda(), lens=torch.from_numpy(lens.astype(np.int32)).cuda(),
                table=torch.from_numpy(table).cuda(), max_len=int(lens.max()), max_n=int(n.max()),
                k_codes=k_codes, k_param=k_param, v_codes=v_codes, v_param=v_param,
                out=torch.zeros((T, Hq, d), dtype=_DT[case["out"]], device="cuda"))


def _lora_inputs(case, seed):
    g = _gen(seed)
    rng = np.random.default_rng(seed)
    T, K, N, r, n = (case[k] for k in ("T", "K", "N", "rank", "adapters"))
    x = torch.randn((T, K), generator=g, device="cuda")
    A = torch.randn((n, r, K), generator=g, device="cuda") / math.sqrt(K)
    B = torch.randn((n, N, r), generator=g, device="cuda") / math.sqrt(r)
    ids = np.repeat(rng.integers(-1 if T >= 8 else 0, n, T), case["runs"])[:T]   # -1: a row without an adapter
    if case["runs"] == 1 and T <= n:
        ids = rng.permutation(n)[:T]
    return dict(x=x.to(torch.bfloat16), A=A.to(torch.bfloat16), B=B.to(torch.bfloat16),
                scale=torch.rand(n, generator=g, device="cuda") + 0.5,
                ids=torch.from_numpy(np.ascontiguousarray(ids, np.int32)).cuda(),
                y=torch.randn((T, N), generator=g, device="cuda"),
                out=torch.zeros((T, N), dtype=torch.float32, device="cuda"))


def prepare(case, seed):
    s = dict(plan=_plan_inputs, append=_append_inputs, attn=_attn_inputs, lora=_lora_inputs)[case["op"]](case, seed)
    s["case"] = case
    if own:
        import quantized_gemv_kv_b200 as sf
        if case["op"] == "plan":
            s["job"] = sf.PagedPlan(s["lens"], s["add"], s["table"], s["free"], s["n_free"], case["P"],
                                    case["max_rows"], keep=s["keep"], lens_out=torch.empty_like(s["lens"]),
                                    n_free_out=torch.empty_like(s["n_free"]))
        elif case["op"] == "append":
            kv = sf.PagedKV(s["k_codes"], s["k_param"], s["v_codes"], s["v_param"])
            s["job"] = sf.PagedAppend(kv, s["k"], s["v"], s["slots"], positions=s["positions"] if case["rope"] else None,
                                      theta=_THETA if case["rope"] else 0.0, q=s["q"], q_out=s["q_out"],
                                      k_val=s["k_val"], v_val=s["v_val"])
        elif case["op"] == "attn":
            kv = sf.PagedKV(s["k_codes"], s["k_param"], s["v_codes"], s["v_param"])
            s["job"] = sf.PagedAttention(s["q"], kv, s["cu"], s["lens"], s["table"], s["out"],
                                         window=case["window"])
        else:
            s["job"] = sf.LoraAdd(s["x"], s["A"], s["B"], s["scale"], s["ids"], s["out"], y=s["y"])
    return s


# ---- one pass ----------------------------------------------------------------


def run(state):
    op = state["case"]["op"]
    if own:
        state["job"].run()
        if op == "plan":
            j = state["job"]
            return dict(lens=j.lens_out, n_free=j.n_free_out, table=state["table"], free=state["free"],
                        cu=j.cu_rows, slots=j.slots, positions=j.positions, request=j.row_request, status=j.status)
        if op == "append":
            return {k: state[k] for k in ("q_out", "k_codes", "k_param", "v_codes", "v_param", "k_val", "v_val")}
        return dict(out=state["out"])
    return dict(plan=_plain_plan, append=_plain_append, attn=_plain_attn, lora=_plain_lora)[op](state)


def _plain_plan(s):
    P, rows = s["case"]["P"], s["case"]["max_rows"]
    lens, keep, add, table, free, n_free = (s[k].long() for k in ("lens", "keep", "add", "table", "free", "n_free"))
    dev, MP = lens.device, table.shape[1]
    new = keep + add
    have, want = (lens + P - 1) // P, (new + P - 1) // P
    grow, back = (want - have).clamp(min=0), (have - want).clamp(min=0)
    cu = torch.cat([add.new_zeros(1), add.cumsum(0)])
    cg, cb = grow.cumsum(0), back.cumsum(0)
    status = torch.zeros_like(n_free)
    status = torch.where((cg[-1:] > n_free + cb[-1:]) | (n_free + cb[-1:] > free.numel()) | (n_free < 0), 3, status)
    status = torch.where(cu[-1:] > rows, 2, status)
    bad = (lens < 0) | (lens > MP * P) | (keep < 0) | (keep > lens) | (add < 0) | (new > MP * P)
    status = torch.where(bad.any(), 1, status)
    ok = status == 0
    # pages given back, in request order, on top of the free list
    i = torch.arange(free.numel(), device=dev)
    f = i - n_free
    owner = torch.searchsorted(cb, f.clamp(min=0), right=True).clamp(max=lens.numel() - 1)
    page = table[owner, (want[owner] + f - (cb - back)[owner]).clamp(0, MP - 1)]
    free2 = torch.where(ok & (f >= 0) & (f < cb[-1:]), page, free)
    # pages taken from its top
    j = torch.arange(MP, device=dev)
    taken = (j >= have[:, None]) & (j < want[:, None])
    a = (cg - grow)[:, None] + j - have[:, None]
    page = free2[(n_free + cb[-1:] - 1 - a).clamp(0, free.numel() - 1)]
    table2 = torch.where(ok & taken, page, table)
    # the step's rows
    r = torch.arange(rows, device=dev)
    req = torch.searchsorted(cu[1:], r, right=True).clamp(max=lens.numel() - 1)
    live = ok & (r < cu[-1:])
    pos = keep[req] + r - cu[req]
    slot = table2[req, (pos // P).clamp(0, MP - 1)] * P + pos % P
    out = dict(lens=torch.where(ok, new, lens), n_free=torch.where(ok, n_free + cb[-1:] - cg[-1:], n_free),
               table=table2, free=free2, cu=torch.where(ok, cu, 0), slots=torch.where(live, slot, -1),
               positions=torch.where(live, pos, 0), request=torch.where(live, req, -1), status=status)
    return {k: v.to(torch.int32) for k, v in out.items()}


def _plain_rope(x, pos):
    """RoPE in 64 bits (far positions), pairs (i, i + d/2); x [T][H][d]."""
    d = x.shape[-1]
    ang = pos.double()[:, None] * torch.pow(_THETA, -2.0 * torch.arange(d // 2, device=x.device,
                                                                       dtype=torch.float64) / d)
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    lo, hi = x[..., :d // 2].double(), x[..., d // 2:].double()
    return torch.cat([lo * c - hi * s, hi * c + lo * s], -1)


def _plain_append(s):
    P, slots = s["case"]["P"], s["slots"].long()
    pages = s["k_codes"].shape[0]
    live = (slots >= 0) & (slots < pages * P)
    out = {}
    k = s["k"].float()
    if s["q_out"] is not None:
        q = _plain_rope(s["q"].float(), s["positions"]).to(torch.bfloat16)
        out["q_out"] = torch.where(live[:, None, None], q, s["q_out"])
        k = _plain_rope(k, s["positions"]).float()
    # rows that are not live write to a spare page behind the pool
    page, off = torch.where(live, slots // P, pages), torch.where(live, slots % P, 0)
    for n, x in (("k", k), ("v", s["v"].float())):
        c, scale, zero = _quant4(x)
        for name, new in (("codes", _pack(c)), ("param", torch.stack([scale, zero], -1))):
            pool = s["%s_%s" % (n, name)]
            pool = torch.cat([pool, pool[:1]])
            pool[page, :, off] = new
            out["%s_%s" % (n, name)] = pool[:-1]
        val = scale.float().unsqueeze(-1) * (c.float() - zero.float().unsqueeze(-1))
        out[n + "_val"] = torch.where(live[:, None, None], val.to(torch.bfloat16), s[n + "_val"])
    return out


def _values(codes, param, page, off):
    """Tokens (page, off) [R][L] of a pool as fp32 [R][L][Hkv][d]."""
    w = codes[page, :, off]
    p = param[page, :, off].float()
    c = (w.unsqueeze(-1) >> (4 * torch.arange(8, device=w.device, dtype=torch.int32))) & 15
    return p[..., :1] * (c.flatten(-2).float() - p[..., 1:])


def _plain_attn(s):
    case = s["case"]
    P, Hkv, d, R = case["P"], case["Hkv"], case["d"], case["R"]
    g = case["Hq"] // Hkv
    L, nmax, cu, lens, q = s["max_len"], s["max_n"], s["cu"].long(), s["lens"].long(), s["q"]
    dev, T = q.device, q.shape[0]
    tok = torch.arange(L, device=dev)
    page = s["table"].long()[:, tok // P]
    page = torch.where(tok < lens[:, None], page, 0)
    off = (tok % P).expand(R, L)
    n = cu[1:] - cu[:-1]
    j = torch.arange(nmax, device=dev)
    qs = q[(cu[:-1, None] + j).clamp(max=T - 1)].float()                            # [R][nmax][Hq][d]
    qs = qs.reshape(R, nmax, Hkv, g, d).permute(0, 2, 1, 3, 4).reshape(R, Hkv, nmax * g, d)
    k = _values(s["k_codes"], s["k_param"], page, off).permute(0, 2, 3, 1)          # [R][Hkv][d][L]
    sc = torch.matmul(qs, k) / math.sqrt(d)
    del k
    at = (lens - n)[:, None] + j                                                    # position of row j
    see = (tok <= at[..., None]) & (tok < lens[:, None, None])
    if case["window"] > 0:
        see &= tok > at[..., None] - case["window"]
    see = see[:, None, :, None].expand(R, 1, nmax, g, L).reshape(R, 1, nmax * g, L)
    sc = torch.where(see, sc, -torch.inf)
    m = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - torch.where(torch.isfinite(m), m, torch.zeros_like(m)))
    del sc
    v = _values(s["v_codes"], s["v_param"], page, off).permute(0, 2, 1, 3)          # [R][Hkv][L][d]
    l = p.sum(-1, keepdim=True)
    o = torch.where(l > 0, torch.matmul(p, v) / l, torch.zeros_like(l))
    o = o.reshape(R, Hkv, nmax, g, d).permute(0, 2, 1, 3, 4).reshape(R, nmax, Hkv * g, d)
    t = torch.arange(T, device=dev)
    req = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=R - 1)
    rows = o[req, (t - cu[req]).clamp(0, nmax - 1)].to(s["out"].dtype)
    return dict(out=torch.where((t < cu[-1])[:, None, None], rows, s["out"]))


def _plain_lora(s):
    n, r, K = s["A"].shape
    x, ids = s["x"].float(), s["ids"].long()
    h = torch.matmul(x, s["A"].float().reshape(n * r, K).t()).reshape(-1, n, r)
    mine = (ids[:, None] == torch.arange(n, device=ids.device)) * s["scale"]
    h = (h * mine.unsqueeze(-1)).reshape(-1, n * r)
    return dict(out=s["y"] + torch.matmul(h, s["B"].float().permute(0, 2, 1).reshape(n * r, -1)))


# ---- what a pass cannot do without --------------------------------------------


def work(case):
    op = case["op"]
    if op == "plan":
        R, rows = case["R"], case["max_rows"]
        return {"bytes": 4 * (3 * R + R + R + 1) + 12 * rows + 8 * R, "flops": 0}
    if op == "append":
        T, Hq, Hkv, d = (case[k] for k in ("T", "Hq", "Hkv", "d"))
        e = 4 if case["src"] == "fp32" else 2
        b = T * ((Hq + 2 * Hkv) * d * e + Hkv * (d + 8) + 4)
        if case["rope"]:
            b += T * (Hq * d * 2 + 4)
        b += T * Hkv * d * 4
        return {"bytes": b, "flops": T * (Hq + 2 * Hkv) * d * 6}
    if op == "attn":
        R, Hq, Hkv, d, w = (case[k] for k in ("R", "Hq", "Hkv", "d", "window"))
        mean = (case["lo"] + case["hi"]) / 2
        if R > 1:
            mean = ((R - 1 - (R >= 4)) * mean + case["hi"]) / R
        n = (case["rows"] + 1) / 2
        if w:
            mean = min(mean, w + n)
        rows = R * n
        return {"bytes": R * mean * Hkv * (d + 8) + rows * Hq * d * (2 + (4 if case["out"] == "fp32" else 2)),
                "flops": 4 * rows * Hq * d * mean}
    T, K, N, r, n = (case[k] for k in ("T", "K", "N", "rank", "adapters"))
    used = min(n, -(-T // case["runs"]))
    return {"bytes": T * K * 2 + T * N * 8 + used * r * (K + N) * 2, "flops": 2 * T * r * (K + N)}


# ---- the definitions in 64 bits ------------------------------------------------


def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = dict(append=_append_inputs, attn=_attn_inputs, lora=_lora_inputs)[case["op"]](case, seed)
    return dict(append=_exact_append, attn=_exact_attn, lora=_exact_lora)[case["op"]](case, s)


def _exact_append(case, s):
    live = [t for t, slot in enumerate(s["slots"].tolist()) if slot >= 0]
    out = dict.fromkeys(("q_out", "k_codes", "k_param", "v_codes", "v_param", "k_val", "v_val"))
    pos = s["positions"].cpu().numpy().astype(np.float64)
    d = case["d"]

    def turned(x):
        """Each pair (i, i + d/2) as a complex number, times e^(i angle)."""
        z = (x[..., :d // 2] + 1j * x[..., d // 2:]) * np.exp(
            1j * pos[:, None, None] * _THETA ** (-np.arange(0, d, 2) / d))
        return np.concatenate([z.real, z.imag], -1)

    if case["rope"]:
        q = np.zeros((case["T"], case["Hq"], d))
        q[live] = turned(s["q"].double().cpu().numpy())[live]
        out["q_out"] = q
    for name in ("k", "v"):
        x = s[name].double().cpu().numpy()
        if name == "k" and case["rope"]:
            x = turned(x)
        lo, hi = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
        step = np.minimum((hi - lo) / 15, 65504.0).astype(np.float16).astype(np.float64)
        step[step == 0] = 1.0
        zero = np.clip(np.rint(-lo / step), 0, 15)
        val = np.zeros_like(x)
        val[live] = (step * (np.clip(np.rint(x / step) + zero, 0, 15) - zero))[live]
        out[name + "_val"] = val
        param = np.zeros(s[name + "_param"].shape)
        at = s["slots"].cpu().numpy()[live]
        param[at // case["P"], :, at % case["P"]] = np.concatenate([step, zero], -1)[live]
        out[name + "_param"] = param
    return {k: v for k, v in out.items() if v is not None}


def _exact_attn(case, s):
    P, d, g = case["P"], case["d"], case["Hq"] // case["Hkv"]
    cu, lens, table = s["cu"].tolist(), s["lens"].tolist(), s["table"].long()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")

    def tokens(name, pages, L):
        w, p = s[name + "_codes"][pages].long(), s[name + "_param"][pages].double()
        c = torch.stack([(w >> (4 * b)) & 15 for b in range(8)], -1).flatten(-2).double()
        x = p[..., :1] * (c - p[..., 1:])                      # [pages][Hkv][P][d]
        return x.transpose(0, 1).flatten(1, 2)[:, :L]          # [Hkv][L][d]

    for i in range(case["R"]):
        n, L = cu[i + 1] - cu[i], lens[i]
        if not n or not L:
            continue
        pages = table[i, :-(-L // P)]
        k, v = tokens("k", pages, L), tokens("v", pages, L)
        for j in range(n):
            last = L - n + j
            first = max(0, last - case["window"] + 1) if case["window"] else 0
            q = s["q"][cu[i] + j].double().reshape(case["Hkv"], g, d)
            a = torch.softmax(q @ k[:, first:last + 1].transpose(1, 2) / math.sqrt(d), -1)
            out[cu[i] + j] = (a @ v[:, first:last + 1]).reshape(-1, d)
    return dict(out=out)


def _exact_lora(case, s):
    out = s["y"].double()
    for a in sorted(set(s["ids"].tolist()) - {-1}):
        rows = (s["ids"] == a).nonzero()[:, 0]
        h = s["x"][rows].double() @ s["A"][a].double().t()
        out[rows] += s["scale"][a].double() * (h @ s["B"][a].double().t())
    return dict(out=out)
