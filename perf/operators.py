"""The paged-cache operators that the performance record covers: appending keys and values to a paged cache with the
rotary rotation applied on the way (`masw_paged_append`), and attention over such a cache (`masw_paged_attn`), both for
bf16 pages and for e4m3 pages with one scale per page and kv head.

`own = False` computes them with elementary torch operations in fp32; `own = True` makes the library's calls.
`exact` restates both definitions in fp64, written apart from the plain form.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn


def _case(name, op, dtype, B, hq, hkv, d, page, rows, kv, ragged=False, window=0, inter=False, strided=False):
    return dict(name=name, op=op, dtype=dtype, B=B, hq=hq, hkv=hkv, d=d, page=page, rows=rows, kv=kv, ragged=ragged,
                window=window, inter=inter, strided=strided)


def listed():
    return [
        # one new token for each of 8 sequences: the append of a decode step, where latency counts
        _case("append_step_b8_e4m3", "append", "e4m3", 8, 24, 8, 128, 64, 1, 2048, ragged=True, strided=True),
        # a verify block of 5 drafts + 1 for 32 sequences, ragged, from a fused QKV projection
        _case("append_verify_b32_bf16", "append", "bf16", 32, 32, 8, 128, 16, 6, 4096, ragged=True, strided=True),
        # 61 new tokens a sequence at most, small heads, adjacent-pair rotation, pages that end inside the rows
        _case("append_mixed_d64_e4m3", "append", "e4m3", 13, 8, 2, 64, 32, 61, 777, ragged=True, inter=True),
        # a whole 32K prompt of one sequence (the draft shape's 24 query and 8 kv heads)
        _case("append_prompt_32k_e4m3", "append", "e4m3", 1, 24, 8, 128, 64, 32768, 32768, strided=True),
        # one decode step of one sequence at 4K: the smallest attention call
        _case("decode_b1_4k_e4m3", "attn", "e4m3", 1, 24, 8, 128, 64, 1, 4096),
        # one decode step of 8 sequences at 32K
        _case("decode_b8_32k_e4m3", "attn", "e4m3", 8, 24, 8, 128, 64, 1, 32768),
        # a verify block (5 drafts + 1) of 4 sequences at 32K, 32 query heads over 8 kv heads
        _case("verify_b4_32k_e4m3", "attn", "e4m3", 4, 32, 8, 128, 64, 6, 32768),
        # 32 sequences of 4K..16K in bf16 pages of 16 tokens: a serving batch
        _case("decode_b32_ragged_bf16", "attn", "bf16", 32, 32, 8, 128, 16, 1, 16384, ragged=True),
        # one query token a sequence through a sliding window of 1024, one kv head for all query heads, small heads
        _case("decode_b64_window_mqa_e4m3", "attn", "e4m3", 64, 16, 1, 64, 32, 1, 9001, ragged=True, window=1024),
        # a 2K chunk of a prompt on top of a 30K prefix
        _case("chunk_2k_at_32k_e4m3", "attn", "e4m3", 1, 32, 8, 128, 64, 2048, 32768),
        # whole prompts of up to 4K, ragged, bf16 pages
        _case("prompt_b4_4k_bf16", "attn", "bf16", 4, 24, 8, 128, 64, 4096, 4096, ragged=True),
        # short query blocks (too many rows for one tile of few rows) on long caches
        _case("extend_b3_20k_e4m3", "attn", "e4m3", 3, 32, 8, 128, 64, 40, 20011, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn"])
    dtype = rng.choice(["e4m3", "e4m3", "bf16"])
    d = rng.choice([128, 128, 128, 64])
    hkv, g = rng.choice([(8, 3), (8, 4), (8, 4), (4, 1), (2, 8), (1, 16), (4, 6), (8, 2), (2, 5)])
    page = rng.choice([16, 32, 64, 64, 128])
    kind = rng.choice(["step", "step", "verify", "rows"])
    inter, strided, ragged = rng.random() < 0.3, rng.random() < 0.5, rng.random() < 0.7
    if op == "append":
        if kind == "rows":
            B = _log_int(rng, 1, 8)
            rows = _log_int(rng, 20, 24000 // B)
            kv = rows + _log_int(rng, 1, 2000)
        else:
            B = _log_int(rng, 1, 64)
            rows = 1 if kind == "step" else rng.randint(2, 9)
            kv = _log_int(rng, 40, 4096)
        return _case("", "append", dtype, B, hkv * g, hkv, d, page, rows, kv, ragged, 0, inter, strided) | {"name": "x"}
    window = rng.choice([0, 0, 0, rng.randint(100, 4000)])
    if kind == "rows":
        B = _log_int(rng, 1, 4)
        rows = _log_int(rng, 20, 1500 // B)
        kv = rows + _log_int(rng, 1, 20000)
    else:
        B = _log_int(rng, 1, 48)
        rows = 1 if kind == "step" else rng.randint(2, 8)
        kv = _log_int(rng, 100, min(32768, 500000 // B))
    return _case("", "attn", dtype, B, hkv * g, hkv, d, page, rows, kv, ragged, window, False, strided) | {"name": "x"}


def _lengths(case):
    """Host lists: new (query) rows and cache lengths, the latter counting the rows; ragged ones spread over
    [1, rows] and [kv / 4, kv]."""
    B, rows, kv = case["B"], case["rows"], case["kv"]
    if not case["ragged"]:
        return [rows] * B, [max(kv, rows)] * B
    u, w = [(b * 0.6180339887) % 1.0 for b in range(B)], [(b * 0.7548776662) % 1.0 for b in range(B)]
    n = [rows - int(u[b] * rows) for b in range(B)]
    return n, [max(n[b], kv - int(w[b] * (kv - kv // 4))) for b in range(B)]


def prepare(case, seed):
    c = case
    cpu = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    n, kl = _lengths(c)
    B, hq, hkv, d, P = c["B"], c["hq"], c["hkv"], c["d"], c["page"]
    T = sum(n)
    per = [-(-x // P) for x in kl]
    n_pages = sum(per) + 3
    perm = torch.randperm(n_pages, generator=cpu)
    width = max(per) + 1
    table = torch.zeros(B, width, dtype=torch.int32)
    at = 0
    for b in range(B):
        table[b, :per[b]] = perm[at:at + per[b]].to(torch.int32)
        at += per[b]
    s = dict(case=c, n=n, kl=kl, T=T, table=table.to(DEV), kv_len=torch.tensor(kl, dtype=torch.int32, device=DEV))
    starts = torch.zeros(B + 1, dtype=torch.int32)
    starts[1:] = torch.cumsum(torch.tensor(n), 0)
    s["row_start"] = starts.to(DEV)
    s["max_rows"] = max(n)
    e4 = c["dtype"] == "e4m3"
    shape = (n_pages, hkv, P, d)
    for x in ("k", "v"):
        if e4:
            # about N(0, 1) in units of 2^-6, with a scale of its own for each page and head
            s[x + "c"] = torch.randn(shape, generator=gen, device=DEV).mul_(60.0).clamp_(-448, 448).to(E4M3)
            s[x + "s"] = torch.exp2(torch.randint(-8, -4, shape[:2], generator=gen, device=DEV).float())
        else:
            s[x + "c"] = torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16)
            s[x + "s"] = None
    # rows of a fused QKV projection, or separate arrays
    qkv = torch.randn(T, (hq + 2 * hkv) * d, generator=gen, device=DEV)
    # a few loud channels, as keys have them
    loud = torch.rand((hq + 2 * hkv) * d, generator=gen, device=DEV) < 0.02
    qkv = torch.where(loud, qkv * 6, qkv).to(torch.bfloat16)
    q, k, v = qkv[:, :hq * d], qkv[:, hq * d:(hq + hkv) * d], qkv[:, (hq + hkv) * d:]
    if not c["strided"]:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    s["q"], s["k"], s["v"] = q.unflatten(1, (hq, d)), k.unflatten(1, (hkv, d)), v.unflatten(1, (hkv, d))
    if c["op"] == "append":
        pos = torch.arange(max(kl) + 1, dtype=torch.float64, device=DEV)
        inv = 500000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64, device=DEV) / d)
        ang = pos[:, None] * inv[None, :]
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        s["q_out"] = torch.zeros(T, hq, d, dtype=torch.bfloat16, device=DEV)
    else:
        s["o"] = torch.zeros(T, hq, d, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.zeros(T, hq, device=DEV)
    if own:
        from compressed_draft_kv_gb300 import capi
        s["cache"] = capi.masw_paged_cache(s["kc"], s["vc"], s["table"], s["ks"], s["vs"])
        if c["op"] == "append":
            s["rope"] = capi.masw_rope(s["cos_sin"], interleaved=c["inter"])
        else:
            need = capi.masw_paged_workspace_bytes(s["cache"], T, s["max_rows"], hq)
            s["ws"] = torch.empty(need, dtype=torch.uint8, device=DEV)
    return s


def _rows_of(s):
    """Per new row: its sequence and its position in it."""
    st = s["row_start"].long()
    r = torch.arange(s["T"], device=DEV)
    b = torch.searchsorted(st, r, right=True) - 1
    return b, s["kv_len"].long()[b] - (st[b + 1] - st[b]) + (r - st[b])


def _rotate(x, cos_sin, pos, inter):
    """x [T, H, D] -> fp32, the pairs of each head rotated by their position's angles."""
    c, sn = cos_sin[pos][:, None, :].chunk(2, -1)
    x = x.float()
    if inter:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat([a * c - b * sn, b * c + a * sn], -1)


def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s (1 where amax is 0)."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(-64, 119)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.ones_like(amax))


def _append_plain(s):
    c = s["case"]
    P = c["page"]
    b, pos = _rows_of(s)
    pid, off = s["table"].long()[b, pos // P], pos % P
    s["q_out"].copy_(_rotate(s["q"], s["cos_sin"], pos, c["inter"]))
    _store_plain(s, "k", _rotate(s["k"], s["cos_sin"], pos, c["inter"]), pid, off)
    _store_plain(s, "v", s["v"].float(), pid, off)
    return _append_out(s)


def _store_plain(s, name, x, pid, off):
    cache, scale = s[name + "c"], s[name + "s"]
    if scale is None:
        cache[pid, :, off] = x.to(torch.bfloat16)
        return
    n_pages, hkv, P, _ = cache.shape
    raw = cache.view(torch.uint8)
    amax = torch.zeros(n_pages, hkv, device=DEV)
    amax.scatter_reduce_(0, pid[:, None].expand(-1, hkv), x.abs().amax(-1), "amax")
    first = torch.full((n_pages,), P, device=DEV, dtype=torch.long).scatter_reduce_(0, pid, off, "amin")
    new = _pow2_scale(amax)
    # a page that this call starts takes the new rows' scale; one that it goes on with never lowers its own
    new = torch.where((first == 0)[:, None], new, torch.where(amax > 0, torch.maximum(new, scale), scale))
    # rows already there are rounded again where their page's scale grew
    grew = ((new > scale) & (first > 0)[:, None] & (first < P)[:, None]).any(1).nonzero()[:, 0]
    old = raw[grew].view(E4M3).float() * (scale[grew] / new[grew])[:, :, None, None]
    keep = (torch.arange(P, device=DEV)[None] < first[grew][:, None])[:, None, :, None]
    raw[grew] = torch.where(keep, old.to(E4M3).view(torch.uint8), raw[grew])
    scale.copy_(torch.where((first < P)[:, None], new, scale))
    raw[pid, :, off] = (x / scale[pid][:, :, None]).to(E4M3).view(torch.uint8)


def _append_out(s):
    out = {"k": s["kc"], "v": s["vc"], "q": s["q_out"]}
    if s["ks"] is not None:
        out |= {"k_scale": s["ks"], "v_scale": s["vs"]}
    return out


def _pages(s, name, width):
    """The sequences' rows [B, hkv, width * P, d] in fp32."""
    pid = s["table"].long()[:, :width]
    cache, scale = s[name + "c"], s[name + "s"]
    if scale is None:
        x = cache[pid].float()
    else:
        x = cache.view(torch.uint8)[pid].view(E4M3).float() * scale[pid][..., None, None]
    return x.transpose(1, 2).flatten(2, 3)


def _attn_plain(s):
    c = s["case"]
    B, hq, hkv, d, P = c["B"], c["hq"], c["hkv"], c["d"], c["page"]
    G, R = hq // hkv, s["max_rows"]
    width = -(-max(s["kl"]) // P)
    b, pos = _rows_of(s)
    j = torch.arange(s["T"], device=DEV) - s["row_start"].long()[b]
    q = torch.zeros(B, R, hq, d, device=DEV)
    at = torch.full((B, R), -1, device=DEV, dtype=torch.long)
    q[b, j], at[b, j] = s["q"].float(), pos
    key = torch.arange(width * P, device=DEV)
    K, V = _pages(s, "k", width), _pages(s, "v", width)
    V = torch.where((key[None] < s["kv_len"][:, None])[:, None, :, None], V, 0.0)
    q = q.unflatten(2, (hkv, G)).permute(0, 2, 3, 1, 4).flatten(2, 3)          # [B, hkv, G * R, d]
    x = (q @ K.transpose(-1, -2)).unflatten(2, (G, R)).mul_(1.0 / math.sqrt(d))
    see = key <= at[..., None]
    if c["window"]:
        see &= key > at[..., None] - c["window"]
    x = x.masked_fill_(~see[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp_min(-1e30)
    p = (x - m).exp_()
    del x
    l = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ V).unflatten(2, (G, R)) / l.clamp_min(1e-30)
    lse = (m + l.log())[..., 0]
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[b, j]
    s["o"].copy_(o)
    s["lse"].copy_(lse.permute(0, 3, 1, 2).flatten(2, 3)[b, j])
    return {"o": s["o"], "lse": s["lse"]}


def run(state):
    s = state
    if s["case"]["op"] == "append":
        if own:
            from compressed_draft_kv_gb300 import capi
            capi.masw_paged_append(s["cache"], s["kv_len"], s["k"], s["v"], rope=s["rope"], q=s["q"], q_out=s["q_out"],
                                   row_start=s["row_start"])
            return _append_out(s)
        return _append_plain(s)
    if own:
        from compressed_draft_kv_gb300 import capi
        capi.masw_paged_attn(s["cache"], s["kv_len"], s["q"], s["o"], s["lse"], row_start=s["row_start"],
                             max_rows=s["max_rows"], window=s["case"]["window"], workspace=s["ws"])
        return {"o": s["o"], "lse": s["lse"]}
    return _attn_plain(s)


def work(case):
    c = case
    e = 1 if c["dtype"] == "e4m3" else 2
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    nbytes = flops = 0.0
    for n, kl in zip(*_lengths(c)):
        if c["op"] == "append":
            # the rows read (bf16), their angles, the rows written, q written
            nbytes += n * (hq + 2 * hkv) * d * 2 + n * d * 4 + n * 2 * hkv * d * e + n * hq * d * 2
            if e == 1:
                nbytes += 2 * hkv * 4 * (n / c["page"] + 1)
            flops += n * (hq + hkv) * d * 3
            continue
        seen = min(kl, c["window"] + n - 1) if c["window"] else kl
        nbytes += seen * 2 * hkv * d * e + n * hq * (d * 2 + d * 2 + 4)
        if e == 1:
            nbytes += seen / c["page"] * 2 * hkv * 4
        vis = sum(min(kl - n + j + 1, c["window"] or kl) for j in range(n))
        flops += 4.0 * vis * hq * d
    return {"bytes": nbytes, "flops": flops}


# ---- the definitions in fp64 ------------------------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attn(s)


def _exact_append(s):
    """Per row: its head vectors turned by pos * theta^(-2i/d), in units of the page's scale, which is the power of two
    that the rows' largest magnitude calls for; rows that were there keep their value in the new unit."""
    c = s["case"]
    P, d, hkv, e4 = c["page"], c["d"], c["hkv"], c["dtype"] == "e4m3"
    half = d // 2
    i = torch.arange(half, dtype=torch.float64, device=DEV)
    theta = torch.exp(-2.0 * i / d * math.log(500000.0))
    first = torch.arange(half, device=DEV) * 2 if c["inter"] else torch.arange(half, device=DEV)
    second = first + (1 if c["inter"] else half)
    out = {"k": s["kc"].double(), "v": s["vc"].double(), "q": torch.zeros(s["T"], c["hq"], d, dtype=torch.float64, device=DEV)}
    if e4:
        out |= {"k_scale": s["ks"].double().clone(), "v_scale": s["vs"].double().clone()}
    row = 0
    for b in range(c["B"]):
        n, kl = s["n"][b], s["kl"][b]
        where = torch.arange(kl - n, kl, dtype=torch.float64, device=DEV)
        turn = torch.polar(torch.ones(n, half, dtype=torch.float64, device=DEV), where[:, None] * theta[None])[:, None]
        new = {}
        for name in ("q", "k"):
            x = s[name][row:row + n].double()
            z = torch.complex(x[..., first], x[..., second]) * turn
            y = torch.empty_like(x)
            y[..., first], y[..., second] = z.real, z.imag
            new[name] = y
        new["v"] = s["v"][row:row + n].double()
        out["q"][row:row + n] = new["q"]
        p = kl - n
        while p < kl:
            page, end = int(s["table"][b, p // P]), min(kl, (p // P + 1) * P)
            for name in ("k", "v"):
                x = new[name][p - (kl - n):end - (kl - n)].transpose(0, 1)       # [hkv, rows, d]
                if e4:
                    big = x.abs().amax((1, 2))
                    sc = torch.exp2(torch.ceil(torch.log2(big / 448.0)))
                    if p % P:
                        was = out[name + "_scale"][page]
                        sc = torch.maximum(sc, was)
                        out[name][page, :, :p % P] *= (was / sc)[:, None, None]
                    out[name + "_scale"][page] = sc
                    x = x / sc[:, None, None]
                out[name][page, :, p % P:p % P + end - p] = x
            p = end
        row += n
        if row > 40000 or c["B"] * c["rows"] // P > 20000:
            return None
    return out


def _exact_attn(s):
    c = s["case"]
    P, d, hkv, G, w = c["page"], c["d"], c["hkv"], c["hq"] // c["hkv"], c["window"]
    o = torch.zeros(s["T"], c["hq"], d, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["T"], c["hq"], dtype=torch.float64, device=DEV)
    row = 0
    for b in range(c["B"]):
        n, kl = s["n"][b], s["kl"][b]
        ids = s["table"][b, :-(-kl // P)].long()
        for h in range(hkv):
            kk, vv = s["kc"][:, h].view(torch.uint8 if s["ks"] is not None else torch.bfloat16)[ids], \
                s["vc"][:, h].view(torch.uint8 if s["ks"] is not None else torch.bfloat16)[ids]
            if s["ks"] is not None:
                kk = kk.view(E4M3).double() * s["ks"][ids, h].double()[:, None, None]
                vv = vv.view(E4M3).double() * s["vs"][ids, h].double()[:, None, None]
            kk, vv = kk.double().reshape(-1, d)[:kl], vv.double().reshape(-1, d)[:kl]
            for r0 in range(0, n, 512):
                r1 = min(n, r0 + 512)
                at = torch.arange(kl - n + r0, kl - n + r1, device=DEV)
                lo = max(0, int(kl - n + r0 - w + 1)) if w else 0
                hi = kl - n + r1
                cols = torch.arange(lo, hi, device=DEV)
                x = torch.einsum("rgd,kd->rgk", s["q"][row + r0:row + r1, h * G:(h + 1) * G].double(), kk[lo:hi])
                x = x / math.sqrt(d)
                hide = cols[None] > at[:, None]
                if w:
                    hide = hide | (cols[None] <= at[:, None] - w)
                x = x.masked_fill(hide[:, None], -math.inf)
                z = torch.logsumexp(x, -1)
                lse[row + r0:row + r1, h * G:(h + 1) * G] = z
                o[row + r0:row + r1, h * G:(h + 1) * G] = torch.einsum("rgk,kd->rgd", torch.exp(x - z[..., None]), vv[lo:hi])
        row += n
    return {"o": o, "lse": lse}
