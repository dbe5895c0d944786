"""Measured cases of the 4-bit cache tier, the cache prologue and the page operators.

Three operators around the paged cache of 576-value rows (512 latent + 64 rope, 32 rows a page):

* attn      one decode step of attention over a cache held in 4 bits, dense or over selected pages;
* prologue  what precedes it: the new rows' RMS norm (latent) and position rotation (rope part), quantised and
            written into the paged cache (E4M3, BF16 or 4 bits), and the queries' rotation and quantisation;
* pages     pages copied within a pool (forks, compaction with the page table's rewrite) and between pools of
            8 and 4 bits (demotion, promotion).

A 4-bit page of 32 rows is 10,752 bytes: 32 x 256 B of E2M1 codes, 16 x 32 scale codes (one byte per block of 32
latent values and row), 32 x 64 E4M3 codes of the rope part.  Value = kv_scale * 2^(scale code - 8) * E2M1 code.
In a 32-bit word of 8 values, nibble j's low 3 bits are value j's magnitude code; the nibbles' top bits, taken in
the order 1 3 5 7 0 2 4 6, are the signs of values 0 to 7.  Scale code 15 marks a block that held a NaN.
"""
import math

import torch

own = False

LATENT, ROPE, DIM, PAGE, BLOCK = 512, 64, 576, 32, 32
NBLK = LATENT // BLOCK
FP4_CODES, FP4_SCALES, FP4_PAGE = PAGE * 256, NBLK * PAGE, 10752
ROW_BYTES = {"fp8": 576, "bf16": 1152, "fp4": 336}
KIND = {"fp8": 0, "bf16": 1, "fp4": 2}  # the framework's cache kinds
SIGN_ORDER = [1, 3, 5, 7, 0, 2, 4, 6]   # nibble whose top bit is the sign of value j
EPS = 1e-6


# ------------------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # One request with a short prompt, one token at a time: latency.
        dict(name="attn_short", op="attn", batch=1, heads=12, q=1, len=1000, ragged=False, causal=False, topk=0, kv_scale=1.0),
        # A serving batch at 128K context, single tokens.
        dict(name="attn_b16_128k", op="attn", batch=16, heads=12, q=1, len=131072, ragged=False, causal=False, topk=0, kv_scale=0.5),
        # Verification of 8 drafted tokens over requests of uneven lengths.
        dict(name="attn_verify_ragged", op="attn", batch=8, heads=12, q=8, len=32777, ragged=True, causal=True, topk=0, kv_scale=1.0),
        # One request with a million tokens: the whole card on one row group.
        dict(name="attn_b1_1m", op="attn", batch=1, heads=12, q=1, len=1048576, ragged=False, causal=False, topk=0, kv_scale=1.0),
        # The same batch behind a block selector that keeps 256 pages of each request.
        dict(name="attn_selected", op="attn", batch=16, heads=12, q=1, len=131072, ragged=False, causal=False, topk=256, kv_scale=1.0),
        # A decode step of 16 requests with 8 drafted tokens into the 4-bit cache, the touched pages expanded to E4M3.
        dict(name="pro_step_fp4", op="prologue", requests=16, tokens=8, heads=12, kind="fp4", halves=False, norm=True, kv_scale=1.0, start=4099),
        # A chunk of a prompt into the E4M3 cache.
        dict(name="pro_chunk_fp8", op="prologue", requests=1, tokens=8192, heads=12, kind="fp8", halves=False, norm=True, kv_scale=0.37, start=100000),
        # Several prompts at once into the BF16 cache.
        dict(name="pro_prompts_bf16", op="prologue", requests=7, tokens=4681, heads=12, kind="bf16", halves=True, norm=True, kv_scale=1.0, start=0),
        # A request forked into 32 samples: each gets its own copy of the last, partly filled page.
        dict(name="pages_fork_bf16", op="pages", src="bf16", dst="bf16", n=32, rows=13, remap=False),
        # A pool compacted: live pages moved down and the page table rewritten.
        dict(name="pages_compact_fp8", op="pages", src="fp8", dst="fp8", n=16384, rows=32, remap=True),
        # Idle requests' pages demoted to the 4-bit pool.
        dict(name="pages_demote", op="pages", src="fp8", dst="fp4", n=16384, rows=32, remap=False),
        # A resumed request's pages promoted back.
        dict(name="pages_promote", op="pages", src="fp4", dst="fp8", n=5003, rows=32, remap=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "prologue", "pages"])
    if op == "attn":
        q, heads = rng.choice([1, 1, 1, 2, 3, 4, 8]), rng.choice([4, 8, 12, 12, 16, 24, 32])
        batch = _log(rng, 1, 32)
        length = max(8, min(_log(rng, 64, 1 << 20), (1 << 20) // batch, 24_000_000 // (batch * heads * q)))
        topk = rng.choice([0, 0, 0, _log(rng, 1, 300)])
        return dict(op=op, batch=batch, heads=heads, q=q, len=length, ragged=rng.random() < 0.5,
                    causal=q > 1, topk=min(topk, (length + PAGE - 1) // PAGE), kv_scale=rng.choice([1.0, 0.5, 0.37]))
    if op == "prologue":
        requests, heads = _log(rng, 1, 64), rng.choice([4, 8, 12, 12, 16])
        return dict(op=op, requests=requests, tokens=max(1, min(_log(rng, 1, 8192), 400_000 // (requests * (heads + 1)))), heads=heads,
                    kind=rng.choice(["fp8", "bf16", "fp4"]), halves=rng.random() < 0.5, norm=rng.random() < 0.8,
                    kv_scale=rng.choice([1.0, 0.5, 0.37]), start=rng.choice([0, _log(rng, 1, 100000)]))
    src, dst = rng.choice([("fp8", "fp8"), ("bf16", "bf16"), ("fp4", "fp4"), ("fp8", "fp4"), ("fp4", "fp8")])
    return dict(op=op, src=src, dst=dst, n=_log(rng, 1, 13000), rows=rng.choice([32, 32, rng.randint(1, 31)]),
                remap=src == dst and rng.random() < 0.5)


def _lens(case):
    """The requests' lengths: all the same, or spread evenly down to a fraction of the longest."""
    b, n, q = case["batch"], case["len"], case["q"]
    return [max(q, n - (n * i) // (b + 1) - (i % 5 if i else 0)) if case["ragged"] else max(q, n) for i in range(b)]


def _pages_of(n):
    return (n + PAGE - 1) // PAGE


def _visible(case):
    """(query row, key) pairs and cache rows read."""
    pairs = rows = 0
    for n in _lens(case):
        seen = n if not case["topk"] else min(n, case["topk"] * PAGE)
        rows += seen
        pairs += case["heads"] * (case["q"] * seen - (case["q"] * (case["q"] - 1) // 2 if case["causal"] and not case["topk"] else 0))
    return pairs, rows


def work(case):
    if case["op"] == "attn":
        pairs, rows = _visible(case)
        r = case["batch"] * case["q"] * case["heads"]
        return {"bytes": rows * ROW_BYTES["fp4"] + r * (DIM + 2 * LATENT + 4), "flops": 2 * pairs * (DIM + LATENT)}
    if case["op"] == "prologue":
        n = case["requests"] * case["tokens"]
        q_out = 2 * DIM if case["kind"] == "bf16" else DIM
        b = n * (2 * DIM + ROW_BYTES[case["kind"]]) + n * case["heads"] * (2 * DIM + q_out)
        if case["kind"] == "fp4":  # the expansion of the pages that were touched
            b += sum(len(p) for p in _touched(case)) * PAGE * (ROW_BYTES["fp4"] + ROW_BYTES["fp8"])
        return {"bytes": b, "flops": n * (5 * LATENT + (3 * ROPE + DIM) * (1 + case["heads"]))}
    n = case["n"] * case["rows"]
    b = n * (ROW_BYTES[case["src"]] + ROW_BYTES[case["dst"]]) + 8 * case["n"]
    return {"bytes": b + (8 * 4 * case["n"] if case["remap"] else 0), "flops": 0 if case["src"] == case["dst"] else 4 * n * LATENT}


# ------------------------------------------------------------------------------------- the formats, plain form
_MAG = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _fp4_values(pages):
    """[..., 10752] bytes -> [..., 32, 576] 32-bit values, before kv_scale."""
    lead = pages.shape[:-1]
    codes = pages[..., :FP4_CODES].reshape(*lead, PAGE, 256)
    nib = torch.stack((codes & 15, codes >> 4), dim=-1).reshape(*lead, PAGE, LATENT // 8, 8)
    mag = torch.tensor(_MAG, device=pages.device)[(nib & 7).int()]
    neg = (nib >> 3)[..., SIGN_ORDER]
    val = torch.where(neg == 1, -mag, mag).reshape(*lead, PAGE, NBLK, BLOCK)
    sc = (pages[..., FP4_CODES:FP4_CODES + FP4_SCALES] & 15).reshape(*lead, NBLK, PAGE).transpose(-1, -2)
    step = torch.where(sc == 15, float("nan"), torch.exp2(sc.float() - 8.0))
    lat = (val * step[..., None]).reshape(*lead, PAGE, LATENT)
    rope = pages[..., FP4_CODES + FP4_SCALES:].reshape(*lead, PAGE, ROPE).view(torch.float8_e4m3fn).float()
    return torch.cat((lat, rope), dim=-1)


def _e4m3(x):
    """Nearest E4M3 (ties to even), saturating at 448; the sign of a NaN is dropped."""
    x = torch.where(torch.isnan(x), float("nan"), x.clamp(-448.0, 448.0))
    return x.to(torch.float8_e4m3fn)


def _fp4_rows(x):
    """[n, 576] 32-bit values over kv_scale -> the three parts of the rows: codes [n, 256], scales [n, 16], rope [n, 64]."""
    v = x[:, :LATENT].reshape(-1, NBLK, BLOCK)
    amax = v.abs().amax(-1)
    bad = torch.isnan(amax)
    limits = 7.0 * torch.exp2(torch.arange(14, device=x.device, dtype=torch.float32) - 8.0)
    sc = (amax[..., None] > limits).sum(-1)
    a = v.abs() * torch.exp2(8.0 - sc.float())[..., None]
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int() + (a >= 3.5).int() + (a > 5.0).int())
    code = torch.where(bad[..., None], 0, code)
    neg = torch.where(bad[..., None], 0, torch.signbit(v).int())
    sc = torch.where(bad, 15, sc)
    nib = code.reshape(-1, LATENT // 8, 8)
    back = [SIGN_ORDER.index(j) for j in range(8)]
    nib = nib | (neg.reshape(-1, LATENT // 8, 8)[..., back] << 3)
    nib = nib.reshape(-1, 256, 2)
    return (nib[..., 0] | (nib[..., 1] << 4)).to(torch.uint8), sc.to(torch.uint8), _e4m3(x[:, LATENT:]).view(torch.uint8)


def _fp4_put(pool, page, slot, parts):
    codes, sc, rope = parts
    pool[:, :FP4_CODES].view(-1, PAGE, 256)[page, slot] = codes
    pool[:, FP4_CODES:FP4_CODES + FP4_SCALES].view(-1, NBLK, PAGE)[page, :, slot] = sc
    pool[:, FP4_CODES + FP4_SCALES:].view(-1, PAGE, ROPE)[page, slot] = rope


# ------------------------------------------------------------------------------------------------ the inputs
def _latents(n, gen):
    """n cache rows as a model has them: unit variance after the norm, with the spread between channel blocks that trained models show."""
    x = torch.randn(n, DIM, device="cuda", generator=gen)
    spread = torch.exp2(torch.randn(DIM // BLOCK, device="cuda", generator=gen))
    return x * spread.repeat_interleave(BLOCK)


def _pool(kind, pages, gen, kv_scale=1.0):
    shape = (pages, FP4_PAGE) if kind == "fp4" else (pages, PAGE, DIM)
    pool = torch.empty(shape, device="cuda", dtype=torch.bfloat16 if kind == "bf16" else torch.uint8)
    for a in range(0, pages, 2048):
        m = min(2048, pages - a)
        x = _latents(m * PAGE, gen) / (1.0 if kind == "bf16" else kv_scale)
        if kind == "bf16":
            pool[a:a + m] = x.bfloat16().view(m, PAGE, DIM)
        elif kind == "fp8":
            pool[a:a + m] = _e4m3(x).view(torch.uint8).view(m, PAGE, DIM)
        else:
            at = torch.arange(m * PAGE, device="cuda")
            _fp4_put(pool[a:a + m], at // PAGE, at % PAGE, _fp4_rows(x))
    return pool


def _table(lens, extra, gen):
    """The requests' pages, dealt from a shuffled pool; -1 past a request's last page."""
    need = [_pages_of(n) for n in lens]
    order = torch.randperm(sum(need) + extra, device="cuda", generator=gen, dtype=torch.int32)
    table = torch.full((len(lens), max(need)), -1, device="cuda", dtype=torch.int32)
    at = 0
    for i, k in enumerate(need):
        table[i, :k] = order[at:at + k]
        at += k
    return table, order


def _spans(case):
    return [(case["start"] + 37 * i, case["start"] + 37 * i + case["tokens"]) for i in range(case["requests"])]


def _touched(case):
    return [range(a // PAGE, _pages_of(b)) for a, b in _spans(case)]


def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    s = dict(case)
    if case["op"] == "attn":
        lens = _lens(case)
        table, order = _table(lens, 3, gen)
        pool = _pool("fp4", order.numel(), gen, case["kv_scale"])
        for i, n in enumerate(lens):  # what lies behind a sequence in its last page is rubbish
            if n % PAGE:
                p = int(table[i, n // PAGE])
                pool[p, :FP4_CODES].view(PAGE, 256)[n % PAGE:] = 255
                pool[p, FP4_CODES:FP4_CODES + FP4_SCALES].view(NBLK, PAGE)[:, n % PAGE:] = 255
                pool[p, FP4_CODES + FP4_SCALES:].view(PAGE, ROPE)[n % PAGE:] = 255
        q = torch.randn(case["batch"], case["q"], case["heads"], DIM, device="cuda", generator=gen) * 0.7
        s.update(lens=lens, lens_d=torch.tensor(lens, device="cuda", dtype=torch.int32), table=table, pool=pool, q=_e4m3(q).view(torch.uint8),
                 block_idx=None, softmax_scale=0.0722, q_scale=1.0)
        if case["topk"]:  # the selector's pages: ascending, the last ones of each request among them, -1 behind them
            sel = torch.full((case["batch"], case["topk"]), -1, device="cuda", dtype=torch.int32)
            for i, n in enumerate(lens):
                k = min(case["topk"], _pages_of(n))
                pick = torch.randperm(_pages_of(n) - 1, device="cuda", generator=gen)[:k - 1] if k > 1 else torch.empty(0, device="cuda", dtype=torch.int64)
                sel[i, :k] = torch.cat((pick.sort().values, torch.tensor([_pages_of(n) - 1], device="cuda"))).int()
            s["block_idx"] = sel
        return s
    if case["op"] == "prologue":
        spans = _spans(case)
        n = case["requests"] * case["tokens"]
        table, order = _table([b for _, b in spans], 2, gen)
        # Only the pages that this call touches are held by this process; the others' ids are never read.
        held = torch.cat([table[i, list(t)] for i, t in enumerate(_touched(case))])
        table = table.clone()
        rank = torch.empty_like(order)
        rank.fill_(-1)
        rank[held.long()] = torch.randperm(held.numel(), device="cuda", generator=gen, dtype=torch.int32)
        table = torch.where(table >= 0, rank[table.clamp(min=0).long()], -1)
        pages = held.numel() + 2
        angle = (torch.arange(case["start"] + 37 * case["requests"] + case["tokens"], device="cuda", dtype=torch.float64)[:, None]
                 * 10000.0 ** (-torch.arange(ROPE // 2, device="cuda", dtype=torch.float64) * 2 / ROPE))
        s.update(pages=pages, table=table, pool=_pool(case["kind"], pages, gen, case["kv_scale"]),
                 cos_sin=torch.cat((angle.cos(), angle.sin()), dim=1).float(),
                 req=torch.arange(case["requests"], device="cuda", dtype=torch.int32).repeat_interleave(case["tokens"]),
                 pos=torch.cat([torch.arange(a, b, device="cuda", dtype=torch.int32) for a, b in spans]),
                 rows=(_latents(n, gen) * 3.0).bfloat16(),
                 weight=(1.0 + 0.2 * torch.randn(LATENT, device="cuda", generator=gen)) if case["norm"] else None,
                 q=torch.randn(n, case["heads"], DIM, device="cuda", dtype=torch.bfloat16, generator=gen), q_scale=0.25)
        if case["kind"] == "fp4":
            ids = torch.cat([table[i, list(t)] for i, t in enumerate(_touched(case))])
            s.update(src_ids=ids, dst_ids=torch.arange(ids.numel(), device="cuda", dtype=torch.int32),
                     wide=torch.zeros(ids.numel(), PAGE, DIM, device="cuda", dtype=torch.uint8))
        return s
    n, same = case["n"], case["src"] == case["dst"]
    if same:  # destinations are free pages of the same pool
        order = torch.randperm(2 * n + 1, device="cuda", generator=gen, dtype=torch.int32)
        s["pool"] = s["to"] = _pool(case["src"], 2 * n + 1, gen)
        s.update(src_ids=order[:n].clone(), dst_ids=order[n:2 * n].clone())
    else:
        s["pool"], s["to"] = _pool(case["src"], n + 1, gen), _pool(case["dst"], n + 1, gen)
        s.update(src_ids=torch.randperm(n + 1, device="cuda", generator=gen, dtype=torch.int32)[:n].clone(),
                 dst_ids=torch.randperm(n + 1, device="cuda", generator=gen, dtype=torch.int32)[:n].clone())
    s["row_counts"] = None if case["rows"] == PAGE else torch.full((n,), case["rows"], device="cuda", dtype=torch.int32)
    if case["remap"]:  # every moved page stands in the tables of four requests that share it
        s["table"] = s["src_ids"].repeat(4).view(4, n).contiguous()
        s["table"][:, -1] = -1
        m = torch.arange(2 * n + 1, device="cuda", dtype=torch.int32)
        m[s["src_ids"].long()] = s["dst_ids"]
        s["map"] = m
    return s


# ------------------------------------------------------------------------------------------------ the passes
def run(s):
    if own:
        return {"attn": _own_attn, "prologue": _own_prologue, "pages": _own_pages}[s["op"]](s)
    return {"attn": _attn, "prologue": _prologue, "pages": _pages}[s["op"]](s)


def _attn(s):
    b, q_len, h, _ = s["q"].shape
    dev = s["q"].device
    sel = s["block_idx"]
    if sel is None:
        logical = torch.arange(s["table"].shape[1], device=dev, dtype=torch.int32).expand(b, -1)
    else:
        logical = sel
    page = torch.where(logical >= 0, s["table"].gather(1, logical.clamp(min=0).long()), -1)
    pos = (logical[..., None] * PAGE + torch.arange(PAGE, device=dev, dtype=torch.int32)).reshape(b, -1)
    live = (page[..., None].expand(-1, -1, PAGE).reshape(b, -1) >= 0) & (pos >= 0) & (pos < s["lens_d"][:, None])
    k = _fp4_values(s["pool"][page.clamp(min=0).long()]).reshape(b, -1, DIM)
    k = torch.where(live[..., None], k, 0.0)
    q = s["q"].view(torch.float8_e4m3fn).float().reshape(b, q_len * h, DIM)
    t = torch.matmul(q, k.transpose(1, 2)) * (s["softmax_scale"] * s["q_scale"] * s["kv_scale"])
    see = live[:, None, :]
    if s["causal"]:
        limit = s["lens_d"][:, None] - q_len + torch.arange(1, q_len + 1, device=dev)
        see = see & (pos[:, None, :] < limit.repeat_interleave(h, dim=1)[..., None])
    t = torch.where(see, t, -math.inf)
    top = t.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    p = torch.exp(t - top)
    den = p.sum(-1, keepdim=True)
    o = torch.matmul(p, k[..., :LATENT]) * s["kv_scale"]
    o = torch.where(den > 0, o / den, 0.0)
    lse = (top + torch.log(den)).squeeze(-1)
    return {"out": o.reshape(b, q_len, h, LATENT).bfloat16(), "lse": lse.reshape(b, q_len, h)}


def _rotate(x, cos, sin, halves):
    if halves:
        a, b = x[..., :ROPE // 2], x[..., ROPE // 2:]
        return torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)


def _prologue(s):
    cs = s["cos_sin"][s["pos"].long()]
    cos, sin = cs[:, :ROPE // 2], cs[:, ROPE // 2:]
    x = s["rows"].float()
    lat = x[:, :LATENT]
    if s["weight"] is not None:
        lat = lat * torch.rsqrt(lat.square().mean(-1, keepdim=True) + EPS) * s["weight"]
    x = torch.cat((lat, _rotate(x[:, LATENT:], cos, sin, s["halves"])), dim=1)
    page = s["table"][s["req"].long(), (s["pos"] // PAGE).long()].long()
    slot = (s["pos"] % PAGE).long()
    q = s["q"].float()
    q = torch.cat((q[..., :LATENT], _rotate(q[..., LATENT:], cos[:, None], sin[:, None], s["halves"])), dim=-1)
    if s["kind"] == "bf16":
        s["pool"][page, slot] = x.bfloat16()
        return {"pool": s["pool"], "q": q.bfloat16()}
    q = _e4m3(q * (1.0 / s["q_scale"]))
    x = x * (1.0 / s["kv_scale"])
    if s["kind"] == "fp8":
        s["pool"][page, slot] = _e4m3(x).view(torch.uint8)
        return {"pool": s["pool"].view(torch.float8_e4m3fn), "q": q}
    _fp4_put(s["pool"], page, slot, _fp4_rows(x))
    s["wide"][s["dst_ids"].long()] = _e4m3(_fp4_values(s["pool"][s["src_ids"].long()])).view(torch.uint8)
    return {"pool": s["wide"].view(torch.float8_e4m3fn), "q": q}


def _pages(s):
    src, dst, r = s["src_ids"].long(), s["dst_ids"].long(), s["rows"]
    if s["src"] == s["dst"]:
        if s["src"] == "fp4":
            got, to = s["pool"][src], s["to"]
            to[:, :FP4_CODES].view(-1, PAGE, 256)[dst, :r] = got[:, :FP4_CODES].reshape(-1, PAGE, 256)[:, :r]
            a, b = FP4_CODES, FP4_CODES + FP4_SCALES
            to[:, a:b].view(-1, NBLK, PAGE)[dst, :, :r] = got[:, a:b].reshape(-1, NBLK, PAGE)[:, :, :r]
            to[:, b:].view(-1, PAGE, ROPE)[dst, :r] = got[:, b:].reshape(-1, PAGE, ROPE)[:, :r]
        elif r == PAGE:
            s["to"][dst] = s["pool"][src]
        else:
            s["to"][dst, :r] = s["pool"][src, :r]
    elif s["src"] == "fp8":
        x = s["pool"][src, :r].view(torch.float8_e4m3fn).float().reshape(-1, DIM)
        parts = _fp4_rows(x)
        _fp4_put(s["to"], dst.repeat_interleave(r), torch.arange(r, device=dst.device).repeat(len(dst)), parts)
    else:
        s["to"][dst, :r] = _e4m3(_fp4_values(s["pool"][src])[:, :r]).view(torch.uint8)
    if not s["remap"]:
        return {"pool": s["to"]}
    t = s["table"]
    t.copy_(torch.where(t >= 0, s["map"][t.clamp(min=0).long()], t))
    return {"pool": s["to"], "table": t}


# ------------------------------------------------------------------- the passes through the framework's operators
def _own_attn(s):
    import split_kv_mla_paged_gb300 as mla
    b, q_len, h, _ = s["q"].shape
    k = s.get("kept")
    if k is None:  # the plan, workspace and outputs that a serving loop keeps for a batch
        lens = s["lens"] if s["block_idx"] is None else [PAGE * s["topk"]] * b
        plan = mla.mla_decode_plan(lens, h, q_len, sm_count=torch.cuda.get_device_properties(s["q"].device).multi_processor_count)
        plan_d = torch.tensor([plan.splits.tolist(), plan.chunks.tolist()], dtype=torch.int32).cuda()
        size = mla.mla_decode_workspace_size(b, q_len, h, plan.max_splits)
        ws = torch.empty(size, device="cuda", dtype=torch.uint8)
        mla.mla_decode_workspace_init(ws, size)
        k = s["kept"] = (plan_d[0], plan_d[1], plan.max_splits, plan.kv_split, ws, size,
                         torch.empty(b, q_len, h, LATENT, device="cuda", dtype=torch.bfloat16),
                         torch.empty(b, q_len, h, device="cuda", dtype=torch.float32))
    splits, chunks, max_splits, kv_split, ws, size, out, lse = k
    head = (s["q"], s["pool"], s["pool"].shape[0], s["table"], s["table"].shape[1], s["lens_d"])
    tail = (splits, chunks, max_splits, kv_split, b, q_len, h, s["causal"], s["q_scale"], s["kv_scale"], s["softmax_scale"], ws, size, out, lse)
    if s["block_idx"] is None:
        mla.mla_decode_fp4(*head, *tail)
    else:
        mla.mla_decode_fp4_sparse(*head, s["block_idx"], s["topk"], *tail)
    return {"out": out, "lse": lse}


def _own_prologue(s):
    import split_kv_mla_paged_gb300 as mla
    if "q_out" not in s:
        s["q_out"] = torch.empty(s["q"].shape, device="cuda", dtype=torch.bfloat16 if s["kind"] == "bf16" else torch.uint8)
    wide = s["kind"] == "bf16"
    mla.mla_prologue(s["pos"].shape[0], positions=s["pos"], cos_sin=s["cos_sin"], rope_rows=s["cos_sin"].shape[0], rope_halves=s["halves"],
                     kv_rows=s["rows"], norm_weight=s["weight"], norm_eps=EPS, req_idx=s["req"], page_table=s["table"],
                     max_pages_per_req=s["table"].shape[1], batch=s["table"].shape[0], kv_pages=s["pool"], num_pages=s["pages"],
                     cache_kind=KIND[s["kind"]], kv_scale=1.0 if wide else s["kv_scale"],
                     q_rows=s["q"], num_heads=s["heads"], q_out=s["q_out"], q_kind=KIND["bf16" if wide else "fp8"],
                     q_scale=1.0 if wide else s["q_scale"])
    if wide:
        return {"pool": s["pool"], "q": s["q_out"]}
    q = s["q_out"].view(torch.float8_e4m3fn)
    if s["kind"] == "fp8":
        return {"pool": s["pool"].view(torch.float8_e4m3fn), "q": q}
    mla.mla_pages_copy(s["pool"], s["pages"], KIND["fp4"], s["wide"], s["wide"].shape[0], KIND["fp8"], s["src_ids"], s["dst_ids"], s["src_ids"].shape[0])
    return {"pool": s["wide"].view(torch.float8_e4m3fn), "q": q}


def _own_pages(s):
    import split_kv_mla_paged_gb300 as mla
    mla.mla_pages_copy(s["pool"], s["pool"].shape[0], KIND[s["src"]], s["to"], s["to"].shape[0], KIND[s["dst"]], s["src_ids"], s["dst_ids"], s["n"],
                       rows=s["row_counts"])
    if not s["remap"]:
        return {"pool": s["to"]}
    mla.mla_pages_remap(s["table"], s["table"].numel(), s["map"], s["pool"].shape[0])
    return {"pool": s["to"], "table": s["table"]}


# --------------------------------------------------------------------------------------- the definition in 64 bits
def _exact_fp4(page):
    """One request's pages [p, 10752] -> [32 p, 576] doubles: each value from its bits, by the format's definition."""
    word = page[:, :FP4_CODES].reshape(-1, PAGE, LATENT // 8, 4).long()
    word = word[..., 0] + (word[..., 1] << 8) + (word[..., 2] << 16) + (word[..., 3] << 24)
    lat = torch.empty(page.shape[0], PAGE, LATENT // 8, 8, device=page.device, dtype=torch.float64)
    for j in range(8):
        e, m = (word >> (4 * j + 1)) & 3, (word >> (4 * j)) & 1
        sign = (word >> (4 * SIGN_ORDER[j] + 3)) & 1
        mag = torch.where(e == 0, 0.5 * m, (1.0 + 0.5 * m) * 2.0 ** (e - 1).double())
        lat[..., j] = mag * (1.0 - 2.0 * sign)
    sc = (page[:, FP4_CODES:FP4_CODES + FP4_SCALES].reshape(-1, NBLK, PAGE) % 16).permute(0, 2, 1).double()
    step = torch.where(sc > 14, float("nan"), 2.0 ** (sc - 8.0))
    lat = lat.reshape(-1, NBLK, BLOCK) * step.reshape(-1, NBLK, 1)
    rope = page[:, FP4_CODES + FP4_SCALES:].contiguous().view(torch.float8_e4m3fn).double()
    return torch.cat((lat.reshape(-1, LATENT), rope.reshape(-1, ROPE)), dim=1)


def _exact_round(x, low, high, bits):
    """Nearest value with `bits` fraction bits, ties to even; steps no finer than 2^(low - bits), magnitudes at most `high`."""
    _, e = torch.frexp(x)
    step = ((torch.clamp(e.long() - 1, min=low) - bits + 1023) << 52).view(torch.float64)  # an exact power of two
    return (torch.round(x / step) * step).clamp(-high, high)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attn":
        out = torch.zeros(case["batch"], case["q"], case["heads"], LATENT, dtype=torch.float64)
        lse = torch.full(out.shape[:3], -math.inf, dtype=torch.float64)
        for i, n in enumerate(s["lens"]):
            pages = torch.arange(_pages_of(n), device="cuda")
            if s["block_idx"] is not None:
                pages = s["block_idx"][i].long()
                pages = pages[(pages >= 0) & (pages < _pages_of(n))]
            at = (pages[:, None] * PAGE + torch.arange(PAGE, device="cuda")).reshape(-1)
            k = _exact_fp4(s["pool"][s["table"][i, pages].long()])[at < n] * case["kv_scale"]
            at = at[at < n]
            for t in range(case["q"]):
                last = n - case["q"] + t if case["causal"] else n - 1
                kt = k[at <= last]
                if not len(kt):
                    continue
                z = (s["q"][i, t].view(torch.float8_e4m3fn).double() * s["q_scale"]) @ kt.T * s["softmax_scale"]
                lse[i, t] = torch.logsumexp(z, -1).cpu()
                out[i, t] = (torch.softmax(z, -1) @ kt[:, :LATENT]).cpu()
        return {"out": out, "lse": lse}
    if case["op"] == "prologue":
        angles = s["cos_sin"].double()[s["pos"].long()]
        turn = torch.complex(angles[:, :ROPE // 2], angles[:, ROPE // 2:])

        def turned(x, w):
            z = torch.complex(x[..., :32], x[..., 32:]) if case["halves"] else torch.view_as_complex(x.reshape(*x.shape[:-1], 32, 2).contiguous())
            z = torch.view_as_real(z * w)
            return torch.cat((z[..., 0], z[..., 1]), dim=-1) if case["halves"] else z.flatten(-2)

        x, q = s["rows"].double(), s["q"].double()
        lat = x[:, :LATENT]
        if s["weight"] is not None:
            lat = lat / torch.sqrt((lat ** 2).sum(1, keepdim=True) / LATENT + EPS) * s["weight"].double()
        x = torch.cat((lat, turned(x[:, LATENT:], turn)), dim=1)
        q = torch.cat((q[..., :LATENT], turned(q[..., LATENT:], turn[:, None])), dim=-1)
        page = s["table"][s["req"].long(), (s["pos"] // PAGE).long()].long()
        slot = (s["pos"] % PAGE).long()
        if case["kind"] == "bf16":
            pool = s["pool"].double()
            pool[page, slot] = _exact_round(x, -126, 3.3895313892515355e38, 7)
            return {"pool": pool, "q": _exact_round(q, -126, 3.3895313892515355e38, 7)}
        q = _exact_round(q / s["q_scale"], -6, 448.0, 3)
        x = x / case["kv_scale"]
        if case["kind"] == "fp8":
            pool = s["pool"].view(torch.float8_e4m3fn).double()
            pool[page, slot] = _exact_round(x, -6, 448.0, 3)
            return {"pool": pool, "q": q}
        blocks = x[:, :LATENT].reshape(-1, BLOCK)
        big = blocks.abs().max(1).values
        power = torch.zeros_like(big) - 8  # the smallest scale under which no value is more than half a step off its code
        for e in range(-8, 6):
            power = torch.where(big > 7.0 * 2.0 ** e, float(e + 1), power)
        step = (2.0 ** power)[:, None]
        lat = _exact_round(blocks / step, 0, 6.0, 1) * step
        new = torch.cat((lat.reshape(-1, LATENT), _exact_round(x[:, LATENT:], -6, 448.0, 3)), dim=1)
        pool = _exact_fp4(s["pool"]).reshape(-1, PAGE, DIM)
        pool[page, slot] = new
        wide = torch.zeros(s["wide"].shape, device="cuda", dtype=torch.float64)
        wide[s["dst_ids"].long()] = pool[s["src_ids"].long()]
        return {"pool": wide, "q": q}
    return None  # bytes and page ids: nothing in them is a computed number
