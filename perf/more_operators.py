"""Measured cases of a speculative decode step over forked requests and of the cache's eviction.

Four operators around the paged cache of 576-value rows (512 latent + 64 rope, 32 rows a page):

* shared   attention for requests whose page tables begin with the same pages: the shared prefix is attended once for
           all rows of its group, each request's own suffix by itself, and both are merged;
* weights  the attention weight that every cached key received in a step: the rows' exp(score - lse), summed per key
           and added to what it had;
* evict    the keys with the largest accumulated weight selected (the first and last ones are protected), and their
           rows moved to fresh pages;
* verify   drafted tokens checked against the target's probabilities with given random numbers, and the next token.

A 4-bit page of 32 rows is 10,752 bytes: 32 x 256 B of E2M1 codes, 16 x 32 scale codes (one byte per block of 32
latent values and row), 32 x 64 E4M3 codes of the rope part.  Value = kv_scale * 2^(scale code - 8) * E2M1 code.
In a 32-bit word of 8 values, nibble j's low 3 bits are value j's magnitude code; the nibbles' top bits, taken in
the order 1 3 5 7 0 2 4 6, are the signs of values 0 to 7.
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
SCALE = 0.0722                          # softmax scale


# ------------------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # Four samples of one short prompt, their first own tokens: latency.
        dict(name="shared_short", op="shared", kind="fp8", batch=4, groups=1, heads=12, q=1, prefix=1024, suffix=23, causal=False, kv_scale=1.0),
        # Sixteen samples of one long prompt, some thousand own tokens each.
        dict(name="shared_samples_128k", op="shared", kind="fp8", batch=16, groups=1, heads=12, q=1, prefix=131072, suffix=2001, causal=False, kv_scale=0.5),
        # Verification of 8 drafted tokens in eight samples over a 4-bit cache.
        dict(name="shared_verify_fp4", op="shared", kind="fp4", batch=8, groups=1, heads=12, q=8, prefix=32768, suffix=517, causal=True, kv_scale=1.0),
        # Three prompts of uneven length and popularity in one batch, BF16 cache.
        dict(name="shared_groups_bf16", op="shared", kind="bf16", batch=15, groups=3, heads=12, q=1, prefix=65536, suffix=700, causal=False, kv_scale=1.0),
        # Two short requests over a 4-bit cache.
        dict(name="weights_short_fp4", op="weights", kind="fp4", batch=2, heads=12, q=1, len=1000, causal=False, decay=1.0, kv_scale=1.0),
        # A serving batch at 128K context, single tokens.
        dict(name="weights_b16_128k", op="weights", kind="fp8", batch=16, heads=12, q=1, len=131072, causal=False, decay=1.0, kv_scale=0.5),
        # The observation window at a prompt's end: the last 8 tokens, BF16 cache, ragged lengths.
        dict(name="weights_window_bf16", op="weights", kind="bf16", batch=4, heads=12, q=8, len=32777, causal=True, decay=0.0, kv_scale=1.0),
        # Few requests just above their budget.
        dict(name="evict_short", op="evict", kind="fp8", batch=4, len=2111, keep=1024, first=4, last=64),
        # A serving batch at 128K context brought down to an eighth.
        dict(name="evict_b16_128k", op="evict", kind="fp8", batch=16, len=131072, keep=16384, first=32, last=1024),
        # One request with a million tokens, 4-bit cache.
        dict(name="evict_b1_1m_fp4", op="evict", kind="fp4", batch=1, len=1048576, keep=131072, first=4, last=4096),
        # One request, 3 drafted tokens, a small vocabulary: latency.
        dict(name="verify_b1", op="verify", batch=1, q=4, vocab=32000, dtype="fp32", drafts="sampled"),
        # A serving batch with 7 drafted tokens each, a large vocabulary.
        dict(name="verify_b64", op="verify", batch=64, q=8, vocab=131072, dtype="fp32", drafts="sampled"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["shared", "weights", "evict", "verify"])
    if op == "shared":
        kind, heads, q = rng.choice(["fp8", "fp4", "bf16"]), rng.choice([4, 8, 12, 12, 16]), rng.choice([1, 1, 2, 3, 8])
        batch = _log(rng, 2, 40)
        prefix = max(32, min(_log(rng, 32, 131072), 24_000_000 // (batch * heads * q)) // PAGE * PAGE)
        suffix = max(q, min(_log(rng, 1, 4000), 200_000 // batch, 20_000_000 // (batch * heads * q)))
        return dict(op=op, kind=kind, batch=batch, groups=rng.randint(1, min(4, batch)), heads=heads, q=q, prefix=prefix, suffix=suffix,
                    causal=q > 1, kv_scale=1.0 if kind == "bf16" else rng.choice([1.0, 0.5, 0.37]))
    if op == "weights":
        kind, heads, q = rng.choice(["fp8", "fp4", "bf16"]), rng.choice([4, 8, 12, 12, 16, 32]), rng.choice([1, 1, 2, 5, 8, 16])
        batch = _log(rng, 1, 32)
        length = max(q, min(_log(rng, 1, 1 << 20), 1_000_000 // batch, 24_000_000 // (batch * heads * q)))
        return dict(op=op, kind=kind, batch=batch, heads=heads, q=q, len=length, causal=q > 1, decay=rng.choice([0.0, 1.0, 0.9]),
                    kv_scale=1.0 if kind == "bf16" else rng.choice([1.0, 0.5, 0.37]))
    if op == "evict":
        batch = _log(rng, 1, 48)
        length = min(_log(rng, 1, 1 << 20), 2_000_000 // batch)
        keep = min(_log(rng, 1, length) if length > 1 else 1, 250_000 // batch)
        return dict(op=op, kind=rng.choice(["fp8", "fp4", "bf16"]), batch=batch, len=length, keep=keep,
                    first=rng.choice([0, 4, 32]), last=rng.choice([0, 64, 1000]))
    vocab, q = rng.choice([1000, 32000, 50021, 65536, 100003, 131072]), rng.choice([1, 2, 3, 4, 5, 8])
    return dict(op=op, batch=min(_log(rng, 1, 64), 67_000_000 // (vocab * q)), q=q, vocab=vocab, dtype=rng.choice(["fp32", "bf16"]),
                drafts=rng.choice(["sampled", "sampled", "fixed"]))


def _pages_of(n):
    return (n + PAGE - 1) // PAGE


def _spread(n, count, least):
    """count lengths from n down to about half of it, none below least."""
    return [max(least, n - (n * i) // (2 * count) - (i % 3 if i else 0)) for i in range(count)]


def _groups(case):
    """Requests per group (growing) and the groups' prefix lengths (falling, whole pages)."""
    g, b = case["groups"], case["batch"]
    total = g * (g + 1) // 2
    sizes = [max(1, b * (i + 1) // total) for i in range(g)]
    while sum(sizes) > b:
        sizes[sizes.index(max(sizes))] -= 1
    sizes[-1] += b - sum(sizes)
    return sizes, [max(PAGE, case["prefix"] * (g - i) // g // PAGE * PAGE) for i in range(g)]


def _suffixes(case):
    return _spread(case["suffix"], case["batch"], case["q"])


def _lens(case):
    return _spread(case["len"], case["batch"], case.get("q", 1))


def work(case):
    op = case["op"]
    if op == "shared":
        sizes, prefixes = _groups(case)
        per = case["heads"] * case["q"]
        keys = sum(prefixes) + sum(_suffixes(case))
        pairs = per * (sum(s * p for s, p in zip(sizes, prefixes)) + sum(_suffixes(case)))
        if case["causal"]:
            pairs -= case["batch"] * case["heads"] * case["q"] * (case["q"] - 1) // 2
        rows = case["batch"] * per
        return {"bytes": keys * ROW_BYTES[case["kind"]] + rows * (DIM * (2 if case["kind"] == "bf16" else 1) + 2 * LATENT + 4),
                "flops": 2 * pairs * (DIM + LATENT)}
    if op == "weights":
        n = sum(_lens(case))
        rows = case["batch"] * case["heads"] * case["q"]
        return {"bytes": n * (ROW_BYTES[case["kind"]] + (8 if case["decay"] else 4)) + rows * (DIM * (2 if case["kind"] == "bf16" else 1) + 4),
                "flops": 2 * n * case["heads"] * case["q"] * DIM}
    if op == "evict":
        lens = _lens(case)
        kept = sum(min(n, case["keep"]) for n in lens)
        return {"bytes": 4 * sum(lens) + kept * (2 * ROW_BYTES[case["kind"]] + 8), "flops": 0}
    size = 4 if case["dtype"] == "fp32" else 2
    rows = 2 if case["drafts"] == "sampled" and case["q"] > 1 else 1  # the probabilities that the next token is drawn from
    return {"bytes": case["batch"] * (rows * case["vocab"] * size + 32 * case["q"]), "flops": 2 * case["batch"] * case["vocab"]}


# ------------------------------------------------------------------------------------- the formats, plain form
_MAG = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _values(kind, pages):
    """Pages of a pool -> [..., 32, 576] 32-bit values, before kv_scale."""
    if kind == "bf16":
        return pages.float()
    if kind == "fp8":
        return pages.view(torch.float8_e4m3fn).float()
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


def _queries(kind, q):
    return q.float() if kind == "bf16" else q.view(torch.float8_e4m3fn).float()


def _e4m3(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


# ------------------------------------------------------------------------------------------------ the inputs
def _latents(n, gen):
    """n cache rows as a model has them: unit variance after the norm, with the spread between channel blocks that trained models show."""
    x = torch.randn(n, DIM, device="cuda", generator=gen)
    spread = torch.exp2(torch.randn(DIM // BLOCK, device="cuda", generator=gen))
    return x * spread.repeat_interleave(BLOCK)


def _pool(kind, pages, gen, kv_scale=1.0):
    if kind == "fp4":  # any codes are values; scales from 2^-2 to 2^0, as rows of unit variance have them
        pool = torch.randint(0, 256, (pages, FP4_PAGE), device="cuda", dtype=torch.uint8, generator=gen)
        pool[:, FP4_CODES:FP4_CODES + FP4_SCALES] = torch.randint(5, 8, (pages, FP4_SCALES), device="cuda", dtype=torch.uint8, generator=gen)
        for a in range(0, pages, 8192):
            m = min(8192, pages - a)
            rope = torch.randn(m, PAGE * ROPE, device="cuda", generator=gen)
            pool[a:a + m, FP4_CODES + FP4_SCALES:] = _e4m3(rope / kv_scale).view(torch.uint8)
        return pool
    pool = torch.empty(pages, PAGE, DIM, device="cuda", dtype=torch.bfloat16 if kind == "bf16" else torch.uint8)
    for a in range(0, pages, 2048):
        m = min(2048, pages - a)
        x = _latents(m * PAGE, gen)
        pool[a:a + m] = (x.bfloat16() if kind == "bf16" else _e4m3(x / kv_scale).view(torch.uint8)).view(m, PAGE, DIM)
    return pool


def _spoil(kind, pool, page, slot):
    """What lies behind a sequence in its last page is rubbish."""
    if kind == "bf16":
        pool[page, slot:] = float("nan")
    elif kind == "fp8":
        pool[page, slot:] = 255
    else:
        pool[page, :FP4_CODES].view(PAGE, 256)[slot:] = 255
        pool[page, FP4_CODES:FP4_CODES + FP4_SCALES].view(NBLK, PAGE)[:, slot:] = 255
        pool[page, FP4_CODES + FP4_SCALES:].view(PAGE, ROPE)[slot:] = 255


def _query_rows(kind, case, gen):
    q = torch.randn(case["batch"], case["q"], case["heads"], DIM, device="cuda", generator=gen) * 0.7
    return q.bfloat16() if kind == "bf16" else _e4m3(q).view(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    s = dict(case)
    op, kind = case["op"], case.get("kind")
    if op == "shared":
        sizes, prefixes = _groups(case)
        suffixes = _suffixes(case)
        lens, need = [], sum(p // PAGE for p in prefixes) + sum(_pages_of(n) for n in suffixes)
        order = torch.randperm(need + 3, device="cuda", generator=gen, dtype=torch.int32)
        pool = _pool(kind, need + 3, gen, case["kv_scale"])
        table = torch.full((case["batch"], max(prefixes) // PAGE + _pages_of(max(suffixes))), -1, device="cuda", dtype=torch.int32)
        at, r, offsets = 0, 0, [0]
        for size, prefix in zip(sizes, prefixes):
            k = prefix // PAGE
            table[r:r + size, :k] = order[at:at + k]
            at += k
            for _ in range(size):
                n, m = suffixes[r], _pages_of(suffixes[r])
                table[r, k:k + m] = order[at:at + m]
                at += m
                if n % PAGE:
                    _spoil(kind, pool, int(table[r, k + m - 1]), n % PAGE)
                lens.append(prefix + n)
                r += 1
            offsets.append(r)
        s.update(lens=lens, offsets=offsets, prefixes=prefixes, lens_d=torch.tensor(lens, device="cuda", dtype=torch.int32), table=table, pool=pool,
                 q=_query_rows(kind, case, gen), q_len=case["q"])
        return s
    if op == "verify":
        b, n, v = case["batch"], case["q"], case["vocab"]
        dt = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
        target, draft = torch.empty(b, n, v, device="cuda", dtype=dt), torch.empty(b, n - 1, v, device="cuda", dtype=dt)
        for i in range(b):  # a model's next-token logits, and those of a smaller model that mostly agrees
            z = 3.0 * torch.randn(n, v, device="cuda", generator=gen)
            target[i] = torch.softmax(z, -1)
            draft[i] = torch.softmax(z[:n - 1] + 0.4 * torch.randn(n - 1, v, device="cuda", generator=gen), -1)
        if n == 1:  # single tokens: nothing was drafted
            tokens = torch.zeros(b, 0, device="cuda")
        elif case["drafts"] == "sampled":
            tokens = torch.stack([torch.multinomial(draft[i].float(), 1, generator=gen)[:, 0] for i in range(b)])
        else:  # drafts that were looked up: no probabilities of their own
            tokens = target[:, :n - 1].float().argmax(-1)
        if case["drafts"] != "sampled":
            draft = None
        s.update(target=target, draft=draft, tokens=tokens.int().contiguous(), u=torch.rand(b, n, device="cuda", generator=gen),
                 lens_d=torch.randint(n, 100000, (b,), device="cuda", generator=gen).int(), q_len=n)
        return s
    lens = _lens(case)
    need = [_pages_of(n) for n in lens]
    order = torch.randperm(sum(need) + 3, device="cuda", generator=gen, dtype=torch.int32)
    table = torch.full((len(lens), max(need)), -1, device="cuda", dtype=torch.int32)
    at = 0
    for i, k in enumerate(need):
        table[i, :k] = order[at:at + k]
        at += k
    pool = _pool(kind, sum(need) + 3, gen, case.get("kv_scale", 1.0))
    width = max(lens) + 5
    s.update(lens=lens, lens_d=torch.tensor(lens, device="cuda", dtype=torch.int32), table=table, pool=pool)
    # What the keys have gathered so far: heavy-tailed, and nothing at all for some.
    had = torch.exp(2.5 * torch.randn(len(lens), width, device="cuda", generator=gen) - 8.0)
    had[torch.rand(len(lens), width, device="cuda", generator=gen) < 0.05] = 0.0
    if op == "weights":
        for i, n in enumerate(lens):
            if n % PAGE:
                _spoil(kind, pool, int(table[i, need[i] - 1]), n % PAGE)
        s.update(q=_query_rows(kind, case, gen), q_len=case["q"], had=had, out=torch.zeros_like(had))
        s["lse"] = torch.stack([torch.logsumexp(_scores(s, i), -1) for i in range(len(lens))]).view(len(lens), case["q"], case["heads"])
        return s
    keep = case["keep"]
    new_pages = sum(_pages_of(min(n, keep)) for n in lens)
    fresh = torch.randperm(new_pages + 1, device="cuda", generator=gen, dtype=torch.int32)
    to_table = torch.full((len(lens), _pages_of(keep)), -1, device="cuda", dtype=torch.int32)
    at = 0
    for i, n in enumerate(lens):
        k = _pages_of(min(n, keep))
        to_table[i, :k] = fresh[at:at + k]
        at += k
    s.update(had=had, keep_d=torch.full((len(lens),), keep, device="cuda", dtype=torch.int32), to_table=to_table,
             to=torch.zeros(new_pages + 1, *pool.shape[1:], device="cuda", dtype=pool.dtype),
             kept=torch.full((len(lens), keep), -1, device="cuda", dtype=torch.int32), new_lens=torch.zeros(len(lens), device="cuda", dtype=torch.int32),
             new_had=torch.zeros(len(lens), keep, device="cuda"))
    return s


def _scores(s, i, pos0=0, pos1=None):
    """Scores of request i's rows with its keys [pos0, pos1), natural-log units; -inf where a key is not visible."""
    n = s["lens"][i]
    pos1 = n if pos1 is None else pos1
    at = torch.arange(pos0, pos1, device=s["q"].device)
    k = _values(s["kind"], s["pool"][s["table"][i, pos0 // PAGE:_pages_of(pos1)].long()]).reshape(-1, DIM)[:pos1 - pos0]
    q = _queries(s["kind"], s["q"][i]).reshape(-1, DIM)
    t = (q @ k.T) * (SCALE * s["kv_scale"])
    if s["causal"]:
        limit = n - s["q_len"] + torch.arange(1, s["q_len"] + 1, device=q.device).repeat_interleave(s["heads"])
        t = torch.where(at < limit[:, None], t, -math.inf)
    return t


# ------------------------------------------------------------------------------------------------ the passes
def run(s):
    if own:
        return {"shared": _own_shared, "weights": _own_weights, "evict": _own_evict, "verify": _own_verify}[s["op"]](s)
    return {"shared": _shared, "weights": _weights, "evict": _evict, "verify": _verify}[s["op"]](s)


def _part(q, k, see, scale):
    """Softmax over one part of the keys: its maximum, sum and unnormalised output."""
    t = (q @ k.T) * scale
    if see is not None:
        t = torch.where(see, t, -math.inf)
    top = t.amax(-1, keepdim=True)
    p = torch.exp(t - torch.where(torch.isinf(top), 0.0, top))
    return top, p.sum(-1, keepdim=True), p @ k[:, :LATENT]


def _shared(s):
    q_len, heads, kind = s["q_len"], s["heads"], s["kind"]
    q = _queries(kind, s["q"])
    scale = SCALE * s["kv_scale"]
    out = torch.empty(s["batch"], q_len, heads, LATENT, device=q.device, dtype=torch.bfloat16)
    lse = torch.empty(s["batch"], q_len, heads, device=q.device)
    for g, prefix in enumerate(s["prefixes"]):
        a, b = s["offsets"][g], s["offsets"][g + 1]
        k = _values(kind, s["pool"][s["table"][a, :prefix // PAGE].long()]).reshape(-1, DIM)
        m0, l0, o0 = (x.view(b - a, q_len * heads, -1) for x in _part(q[a:b].reshape(-1, DIM), k, None, scale))
        del k
        for r in range(a, b):
            n = s["lens"][r]
            k = _values(kind, s["pool"][s["table"][r, prefix // PAGE:_pages_of(n)].long()]).reshape(-1, DIM)[:n - prefix]
            see = None
            if s["causal"]:
                limit = n - prefix - q_len + torch.arange(1, q_len + 1, device=q.device).repeat_interleave(heads)
                see = torch.arange(n - prefix, device=q.device) < limit[:, None]
            m1, l1, o1 = _part(q[r].reshape(-1, DIM), k, see, scale)
            top = torch.maximum(m0[r - a], m1)
            w0, w1 = torch.exp(m0[r - a] - top), torch.exp(m1 - top)
            den = w0 * l0[r - a] + w1 * l1
            out[r] = ((w0 * o0[r - a] + w1 * o1) * (s["kv_scale"] / den)).view(q_len, heads, LATENT).bfloat16()
            lse[r] = (top + torch.log(den)).view(q_len, heads)
    return {"out": out, "lse": lse}


def _weights(s):
    for i, n in enumerate(s["lens"]):
        w = torch.exp(_scores(s, i) - s["lse"][i].view(-1, 1)).sum(0)
        s["out"][i, :n] = s["had"][i, :n] * s["decay"] + w if s["decay"] else w
    return {"weights": s["out"]}


def _rows(kind, pool, page, slot):
    if kind != "fp4":
        return (pool[page, slot],)
    b = FP4_CODES + FP4_SCALES
    return (pool[:, :FP4_CODES].view(-1, PAGE, 256)[page, slot], pool[:, FP4_CODES:b].view(-1, NBLK, PAGE)[page, :, slot],
            pool[:, b:].view(-1, PAGE, ROPE)[page, slot])


def _put_rows(kind, pool, page, slot, rows):
    if kind != "fp4":
        pool[page, slot] = rows[0]
        return
    b = FP4_CODES + FP4_SCALES
    pool[:, :FP4_CODES].view(-1, PAGE, 256)[page, slot] = rows[0]
    pool[:, FP4_CODES:b].view(-1, NBLK, PAGE)[page, :, slot] = rows[1]
    pool[:, b:].view(-1, PAGE, ROPE)[page, slot] = rows[2]


def _evict(s):
    for i, n in enumerate(s["lens"]):
        k = min(n, s["keep"])
        w = s["had"][i, :n]
        rank = w.clone()
        rank[:s["first"]] = math.inf
        rank[max(0, n - s["last"]):] = math.inf
        pos = torch.sort(torch.sort(rank, descending=True, stable=True).indices[:k]).values
        s["kept"][i, :k] = pos.int()
        s["new_had"][i, :k] = w[pos]
        s["new_lens"][i] = k
        to = torch.arange(k, device=w.device)
        rows = _rows(s["kind"], s["pool"], s["table"][i, pos // PAGE].long(), pos % PAGE)
        _put_rows(s["kind"], s["to"], s["to_table"][i, to // PAGE].long(), to % PAGE, rows)
    pool = s["to"].view(torch.float8_e4m3fn) if s["kind"] == "fp8" else s["to"]
    return {"kept": s["kept"], "lens": s["new_lens"], "weights": s["new_had"], "pool": pool}


def _verify(s):
    b, n = s["batch"], s["q_len"]
    dev = s["target"].device
    at = torch.arange(b, device=dev)
    x = s["tokens"].long()
    p = s["target"][:, :n - 1].gather(2, x[..., None])[..., 0].double()
    q = s["draft"][:, :n - 1].gather(2, x[..., None])[..., 0].double() if s["draft"] is not None else torch.ones_like(p)
    good = (s["u"][:, :n - 1].double() * q < p).int()
    acc = torch.cumprod(good, 1).sum(1)
    w = s["target"][at, acc].double()
    if n > 1:
        cut = acc < n - 1
        if s["draft"] is not None:
            rest = (w - s["draft"][at, acc.clamp(max=n - 2)].double()).clamp(min=0.0)
        else:
            rest = w.scatter(1, x.gather(1, acc.clamp(max=n - 2)[:, None]), 0.0)
        w = torch.where((cut & (rest.sum(1) > 0.0))[:, None], rest, w)
    total = torch.cumsum(w, 1)
    # The first token whose sum exceeds the threshold.
    nxt = (total <= s["u"][:, n - 1:].double() * total[:, -1:]).sum(1)
    col = torch.arange(n, device=dev)
    tokens = torch.cat((s["tokens"], torch.full((b, 1), -1, device=dev, dtype=torch.int32)), 1)
    tokens = torch.where(col < acc[:, None], tokens, torch.where(col == acc[:, None], nxt[:, None], -1))
    return {"tokens": tokens.int(), "accepted": acc.int(), "lens": (s["lens_d"] - n + 1 + acc).int()}


# ------------------------------------------------------------------- the passes through the framework's operators
def _own_shared(s):
    import split_kv_mla_paged_gb300 as mla
    b, n, h = s["batch"], s["q_len"], s["heads"]
    k = s.get("kept_call")
    if k is None:  # the plan, workspace and outputs that a serving loop keeps for a batch
        plan = mla.mla_shared_plan(s["lens"], s["offsets"], s["prefixes"], h, n, causal=s["causal"], cache_kind=KIND[s["kind"]],
                                   sm_count=torch.cuda.get_device_properties(s["q"].device).multi_processor_count)
        ws = torch.empty(plan.workspace_bytes, device="cuda", dtype=torch.uint8)
        mla.mla_decode_workspace_init(ws, plan.workspace_bytes)
        k = s["kept_call"] = (plan, torch.from_numpy(plan.data).cuda(), ws, torch.empty(b, n, h, LATENT, device="cuda", dtype=torch.bfloat16),
                              torch.empty(b, n, h, device="cuda"))
    plan, plan_d, ws, out, lse = k
    mla.mla_decode_shared(s["q"], s["pool"], s["pool"].shape[0], s["table"], s["table"].shape[1], s["lens_d"], plan, plan_d, b, n, h, s["causal"],
                          1.0, s["kv_scale"], SCALE, ws, plan.workspace_bytes, out, lse)
    return {"out": out, "lse": lse}


def _own_weights(s):
    import split_kv_mla_paged_gb300 as mla
    mla.mla_key_weights(s["q"], s["pool"], s["pool"].shape[0], s["table"], s["table"].shape[1], s["lens_d"], s["lse"], s["out"], s["batch"],
                        s["q_len"], s["heads"], s["causal"], 1.0, s["kv_scale"], SCALE, cache_kind=KIND[s["kind"]],
                        previous=s["had"] if s["decay"] else None, decay=s["decay"])
    return {"weights": s["out"]}


def _own_evict(s):
    import split_kv_mla_paged_gb300 as mla
    mla.mla_evict_select(s["had"], s["lens_d"], s["keep_d"], s["kept"], s["new_lens"], first=s["first"], last=s["last"], new_weights=s["new_had"])
    mla.mla_rows_move(s["pool"], s["pool"].shape[0], s["table"], s["to"], s["to"].shape[0], s["to_table"], s["kept"], s["new_lens"],
                      cache_kind=KIND[s["kind"]])
    pool = s["to"].view(torch.float8_e4m3fn) if s["kind"] == "fp8" else s["to"]
    return {"kept": s["kept"], "lens": s["new_lens"], "weights": s["new_had"], "pool": pool}


def _own_verify(s):
    import split_kv_mla_paged_gb300 as mla
    k = s.get("kept_call")
    if k is None:  # the outputs that a serving loop keeps
        k = s["kept_call"] = (torch.empty(s["batch"], s["q_len"], device="cuda", dtype=torch.int32),
                              torch.empty(s["batch"], device="cuda", dtype=torch.int32), torch.empty(s["batch"], device="cuda", dtype=torch.int32))
    mla.mla_verify_drafts(s["target"], s["tokens"], s["u"], k[0], k[1], draft_probs=s["draft"], kv_lens=s["lens_d"], new_lens=k[2])
    return {"tokens": k[0], "accepted": k[1], "lens": k[2]}


# --------------------------------------------------------------------------------------- the definition in 64 bits
def _exact_rows(kind, page):
    """Pages of a pool -> [32 p, 576] doubles: each value from its bits, by the format's definition."""
    if kind != "fp4":
        return (page if kind == "bf16" else page.view(torch.float8_e4m3fn)).double().reshape(-1, DIM)
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


def exact(case, seed):
    if case["op"] == "evict":
        return None  # positions, and bytes and weights that are copied: nothing in them is a computed number
    s = prepare(case, seed)
    if case["op"] == "verify":
        got = {"tokens": torch.full((case["batch"], case["q"]), -1, dtype=torch.int32), "accepted": torch.zeros(case["batch"], dtype=torch.int32),
               "lens": torch.zeros(case["batch"], dtype=torch.int32)}
        for i in range(case["batch"]):
            a = 0
            while a < case["q"] - 1:
                x = int(s["tokens"][i, a])
                q = 1.0 if s["draft"] is None else float(s["draft"][i, a, x])
                if not float(s["u"][i, a]) * q < float(s["target"][i, a, x]):
                    break
                got["tokens"][i, a] = x
                a += 1
            w = s["target"][i, a].cpu().double()
            if a < case["q"] - 1:
                rest = w.clone()
                if s["draft"] is None:
                    rest[int(s["tokens"][i, a])] = 0.0
                else:
                    rest = torch.relu(w - s["draft"][i, a].cpu().double())
                w = rest if float(rest.sum()) > 0 else w
            run_sum = w.cumsum(0)
            got["tokens"][i, a] = int(torch.searchsorted(run_sum, float(s["u"][i, -1]) * run_sum[-1], right=True))
            got["accepted"][i] = a
            got["lens"][i] = int(s["lens_d"][i]) - case["q"] + 1 + a
        return got
    kind, heads, n_q = case["kind"], case["heads"], case["q"]
    out = torch.zeros(case["batch"], n_q, heads, LATENT, dtype=torch.float64)
    lse = torch.zeros(case["batch"], n_q, heads, dtype=torch.float64)
    gathered = s["out"].double().clone() if case["op"] == "weights" else None
    for i, n in enumerate(s["lens"]):
        k = _exact_rows(kind, s["pool"][s["table"][i, :_pages_of(n)].long()])[:n] * case["kv_scale"]
        if gathered is not None:
            gathered[i, :n] = s["had"][i, :n].double() * case["decay"] if case["decay"] else 0.0
        for t in range(n_q):
            last = n - n_q + t if case["causal"] else n - 1
            q = s["q"][i, t].double() if kind == "bf16" else s["q"][i, t].view(torch.float8_e4m3fn).double()
            z = q @ k[:last + 1].T * SCALE
            if gathered is not None:
                gathered[i, :last + 1] += torch.exp(z - s["lse"][i, t].double()[:, None]).sum(0)
            else:
                lse[i, t] = torch.logsumexp(z, -1).cpu()
                out[i, t] = (torch.softmax(z, -1) @ k[:last + 1, :LATENT]).cpu()
    return {"weights": gathered} if gathered is not None else {"out": out, "lse": lse}
