"""Workloads of the paged operators: norms of Queries and Keys with the rotation in the same pass, page
tables and slot maps, the paged 8- and 4-bit cache (written and read back), and attention of packed
batches over it.

`run(state)` computes one pass: in elementary torch operations (`own` false), or through the package's
calls (`own` true).  `exact(case, seed)` computes the same from the definitions in 64 bits.

The definitions.
- Norm and rotation: a row x of 128 channels of one head becomes x / sqrt(mean(x^2) + eps) * w, then pair
  i of axis a turns by position_a * theta^(-2 i / dim_a); rounded to bf16 once.
- Pages: a sequence of n tokens holds ceil(n / page) pages, entry i of its row of the table the page of
  tokens i page .. (i + 1) page - 1, the others -1.  An update first shortens every sequence to keep[b] tokens,
  then appends count[b].  Free pages are a stack: the new pages, numbered i = 0, 1, ... by sequence and
  place, come from the top down, and the pages given up, numbered the same way, go back so that they
  would come out again in that order; places above the top hold -1.  A sequence is refused (granted 0) when its rows or pages do not fit, or when it
  needs pages and the stack does not hold those of all sequences up to it.  Row first[b] + i of the packed batch
  is new token i, at position at = length + i and in slot table[..] * page + at % page (-1: no token).
- Cache: per token and head, groups of 32 channels; the step s is the smallest number with 5 exponent and
  3 mantissa bits with Q s >= max|x|, Q = 127 or 7, at most 56 (8 bits) or 896 (4 bits); the code is
  rint(x / s), stored plus 128 or 8.  Four-bit codes: channel 8 j + 2 k + t is nibble k + 4 t of 32-bit word
  j.  Keys are normed, turned and rounded to bf16 before they are quantised.
- Attention: new token i of a sequence of `length` tokens stands at p = length - count + i, in frame
  p // tpf, and sees token j when frame(j) <= frame(p) and (frame(p) - frame(j) < frames or j < sink).
"""
import functools
import math

import torch

own = False

D, GROUP = 128, 32
LOG2E = 1.4426950408889634
EPS = 1e-6

# ------------------------------------------------------------------ cases


def listed():
    # 40 heads, frames of 30 x 52 (480p) and 45 x 80 (720p) latent tokens and chunks of three frames are
    # the layer shapes of this repository's workloads; the others are generic serving shapes.
    wan = dict(axis_t=44, axis_y=42, axis_x=42, theta=10000.0, pairing="interleaved")
    text = dict(axis_t=128, axis_y=0, axis_x=0, theta=1000000.0, pairing="half")
    return [
        # Queries of one generated token of each of 32 sequences: latency
        dict(text, name="norm_token", op="norm", batch=32, heads=32, n=1, gh=1, gw=1, start=9000, packed=False, per_head=False),
        # the Queries of one 720p chunk as the projection leaves them (token-major), positions given per token
        dict(wan, name="norm_chunk_720p", op="norm", batch=1, heads=40, n=10800, gh=45, gw=80, start=75600, packed=True, per_head=True),
        # a decoding step of 64 sequences: some end, some lose rejected drafts, each gets one token
        dict(name="pages_token", op="pages", batch=64, page=64, length=4000, count=1, pad=0, drafts=3, tight=False),
        # prompts of many sequences admitted at once, more than the pool holds: the last ones are refused
        dict(name="pages_prompts", op="pages", batch=256, page=16, length=1500, count=250, pad=100, drafts=5, tight=True),
        # one token of each of 64 sequences normed, turned, written and read back: latency
        dict(text, name="write_token", op="write", bits=8, kv_heads=8, n=64, page=64, gh=1, gw=1, start=9000, norm=True, rope=True, skip=0),
        # one 720p chunk: normed, turned, quantised and handed back in bf16 (for packing)
        dict(wan, name="write_chunk_720p", op="write", bits=4, kv_heads=40, n=10800, page=128, gh=45, gw=80, start=75600, norm=True, rope=True,
             skip=0),
        # one token of each of 64 sequences of 125 to 8,000 tokens, grouped heads
        dict(name="attend_token_batch", op="attend", bits=8, page=64, batch=64, heads=32, kv_heads=8, count=1, chunk=0, length=8000, ragged=True,
             empty=False, tpf=1, frames=1 << 20, sink=0, pad=0),
        # one token of one stream over 39,000 tokens: the cache's bytes count
        dict(name="attend_token_stream", op="attend", bits=4, page=128, batch=1, heads=40, kv_heads=40, count=1, chunk=0, length=39000, ragged=False,
             empty=False, tpf=1, frames=1 << 20, sink=0, pad=0),
        # a few drafted tokens of sequences of different lengths, one of them empty, under a window with sinks
        dict(name="attend_drafts_window", op="attend", bits=4, page=16, batch=7, heads=24, kv_heads=8, count=5, chunk=0, length=2777, ragged=True,
             empty=True, tpf=1, frames=1500, sink=3, pad=2),
        # the next 2,048 tokens of a prompt over the 30,000 before them
        dict(name="attend_prompt_chunk", op="attend", bits=8, page=64, batch=1, heads=32, kv_heads=8, count=2048, chunk=0, length=32048,
             ragged=False, empty=False, tpf=1, frames=1 << 20, sink=0, pad=0),
        # 24 sequences generate a token each while one is given the next 777 tokens of its prompt
        dict(name="attend_mixed", op="attend", bits=8, page=32, batch=25, heads=32, kv_heads=8, count=1, chunk=777, length=6001, ragged=True,
             empty=False, tpf=1, frames=1 << 20, sink=0, pad=7),
        # one 480p chunk over the first frame and the 24 before it, block-causal over frames
        dict(name="attend_chunk_480p", op="attend", bits=4, page=256, batch=1, heads=40, kv_heads=40, count=4680, chunk=0, length=60840,
             ragged=False, empty=False, tpf=1560, frames=24, sink=1560, pad=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "pages", "write", "attend", "attend", "attend"])
    axes = rng.choice([dict(axis_t=44, axis_y=42, axis_x=42, theta=10000.0), dict(axis_t=16, axis_y=56, axis_x=56, theta=256.0),
                       dict(axis_t=128, axis_y=0, axis_x=0, theta=500000.0), dict(axis_t=32, axis_y=16, axis_x=16, theta=10000.0)])
    turn = dict(axes, pairing=rng.choice(["interleaved", "half"]), gh=rng.randint(1, 45), gw=rng.randint(1, 80))
    page, bits = rng.choice([16, 32, 64, 128, 256]), rng.choice([8, 4])
    if op == "norm":
        heads, packed = rng.choice([1, 8, 24, 32, 40]), rng.random() < 0.5
        batch = 1 if packed else rng.choice([1, 2, 3, 5, 8, 16])
        return dict(turn, op=op, batch=batch, heads=heads, n=max(1, _log(rng, 1, 432000) // (heads * batch)), start=_log(rng, 1, 2000000),
                    packed=packed, per_head=rng.random() < 0.5)
    if op == "pages":
        batch = _log(rng, 1, 512)
        return dict(op=op, batch=batch, page=page, length=_log(rng, 1, 20000), count=max(1, _log(rng, 1, 60000) // batch), pad=rng.choice([0, 1, 37]),
                    drafts=rng.randint(0, 9), tight=rng.random() < 0.3)
    kv = rng.choice([1, 2, 4, 8, 40])
    if op == "write":
        return dict(turn, op=op, bits=bits, kv_heads=kv, n=max(1, _log(rng, 1, 432000) // kv), page=page, start=_log(rng, 1, 200000),
                    norm=rng.random() < 0.6, rope=rng.random() < 0.6, skip=rng.choice([0, 0, 3]))
    heads = kv * (rng.choice([1, 2, 3, 4, 5, 8]) if kv <= 8 else 1)
    kind = rng.choice(["token", "drafts", "chunk", "mixed"])
    batch = _log(rng, 1, 80) if kind != "chunk" else rng.choice([1, 1, 2, 3])
    count = {"token": 1, "drafts": rng.randint(2, 8), "chunk": _log(rng, 9, 4700), "mixed": 1}[kind]
    chunk = _log(rng, 9, 2000) if kind == "mixed" else 0
    length = _log(rng, 10, 60000)
    while batch * heads * max(count, chunk) * length > 6_000_000_000 or batch * kv * length > 3_500_000:   # (as the largest listed case, padded)
        length, batch = max(10, length // 2), max(1, batch * 2 // 3)
    tpf = rng.choice([1, 1, 1, 16, 390, 1560])
    window = rng.random() < 0.4
    return dict(op=op, bits=bits, page=page, batch=batch, heads=heads, kv_heads=kv, count=count, chunk=chunk, length=length,
                ragged=rng.random() < 0.6, empty=batch > 1 and rng.random() < 0.3, tpf=tpf,
                frames=max(1, _log(rng, 1, length) // tpf) if window else 1 << 20, sink=rng.choice([0, 4, rng.randint(5, 300)]) if window else 0,
                pad=rng.choice([0, 0, 5]))


def _sequences(case):
    """Tokens of each sequence with the new ones, and the new ones."""
    b, n = case["batch"], case["length"]
    lengths = [max(1, n * (b - i) // b) if case["ragged"] else n for i in range(b)]
    if case["empty"]:
        lengths[-1] = 0
    counts = [min(case["count"], m) for m in lengths]
    if case["chunk"]:
        counts[b // 3] = min(case["chunk"], lengths[b // 3])
    return lengths, counts


def _requests(case):
    """The pages case: tokens held, tokens kept, new tokens, and free pages that are missing."""
    b, c = case["batch"], case["count"]
    held = [(case["length"] * (2 * i + 1) * 7919) % (case["length"] + 1) for i in range(b)]
    keep = [0 if i % 11 == 5 else max(0, n - i % (case["drafts"] + 1)) for i, n in enumerate(held)]
    count = [c if c < 3 else max(0, c - (i * 37) % c) if i % 13 else 0 for i in range(b)]
    return held, keep, count


def _pages_of(n, page):
    return -(-n // page)


def _row_bytes(bits):
    return D * bits // 8 + D // GROUP   # a cached Key or Value row of one head


def work(case):
    op = case["op"]
    if op == "norm":
        rows = case["batch"] * case["heads"] * case["n"]
        return {"bytes": 4 * D * rows, "flops": 7 * D * rows}
    if op == "pages":
        held, keep, count = _requests(case)
        entries = sum(_pages_of(n, case["page"]) - _pages_of(min(n, k), case["page"]) + _pages_of(c, case["page"]) for n, k, c in zip(held, keep, count))
        return {"bytes": 16 * (sum(count) + case["pad"]) + 12 * entries + 40 * case["batch"], "flops": 0}
    if op == "write":
        rows = case["n"] * case["kv_heads"]
        return {"bytes": rows * 4 * (2 * D + _row_bytes(case["bits"])), "flops": rows * 2 * D * 5}
    pairs = held = rows = 0
    for n, c in zip(*_sequences(case)):
        if not c:
            continue
        f = (torch.arange(c, dtype=torch.int64) + n - c) // case["tpf"]
        hi = torch.clamp((f + 1) * case["tpf"], max=n)
        sink = torch.clamp(hi, max=case["sink"])
        lo = torch.clamp((f - case["frames"] + 1) * case["tpf"], min=case["sink"])
        pairs += int((sink + torch.clamp(hi - lo, min=0)).sum())
        held += int(sink.max()) + max(0, int(hi.max()) - int(lo.min()))
        rows += c * case["heads"]
    return {"bytes": held * case["kv_heads"] * 2 * _row_bytes(case["bits"]) + rows * (4 * D + 4), "flops": 4 * D * pairs * case["heads"]}


# ------------------------------------------------------------------ inputs


def _activations(gen, n, h):
    """bf16 rows as a projection leaves them: unit noise, eight outlier channels, token-major memory
    seen as [heads][tokens][128]."""
    x = torch.randn(n, h, D, generator=gen, device="cuda", dtype=torch.float32)
    x[..., torch.randperm(D, generator=gen, device="cuda")[:8]] *= 4.0
    return x.to(torch.bfloat16).permute(1, 0, 2)


def _weight(gen, *shape):
    return 1.0 + 0.2 * torch.randn(*shape, generator=gen, device="cuda")


def _pool(gen, case, pages):
    """Codes and steps of written pages."""
    shape = (pages, case["kv_heads"], case["page"])
    out = {}
    for t in ("k", "v"):
        x = torch.randn(*shape, D, generator=gen, device="cuda", dtype=torch.float32)
        x[..., torch.randperm(D, generator=gen, device="cuda")[:8]] *= 4.0
        q, step = _quantise(x.to(torch.bfloat16).float(), case["bits"])
        out[t + "_codes"], out[t + "_step"] = _pack(q, case["bits"]), step
    return out


def _table(gen, lengths, page, extra, width):
    """A table [batch][width] whose pages are scattered over a pool, and the pool's free pages: a stack with a place
    for each of its pages."""
    need = [_pages_of(n, page) for n in lengths]
    total = sum(need)
    order = torch.randperm(total + extra, generator=gen, device="cuda").to(torch.int32)
    starts = torch.tensor([sum(need[:i]) for i in range(len(need))], device="cuda")
    i = torch.arange(width, device="cuda")
    mine = i < torch.tensor(need, device="cuda")[:, None]
    table = torch.where(mine, order[(starts[:, None] + i).clamp(max=total + extra - 1)], -1).to(torch.int32)
    return table, torch.cat([order[total:], torch.full((total,), -1, dtype=torch.int32, device="cuda")])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 11)
    s = {"case": dict(case)}
    whole = lambda v, t: torch.tensor(v, dtype=t, device="cuda")
    op = case["op"]
    if op == "norm":
        b, n = case["batch"], case["n"]
        x = _activations(gen, b * n, case["heads"])
        s["x"] = x.unflatten(1, (b, n)).permute(1, 0, 2, 3)
        s["weight"] = _weight(gen, case["heads"], D) if case["per_head"] else _weight(gen, D)
        start = whole([case["start"] + 37 * i for i in range(b)], torch.int64)
        s["at"] = start[:, None] + torch.arange(n, device="cuda") if case["packed"] else None
        s["start"] = None if case["packed"] else start
        return s
    if op == "pages":
        held, keep, count = _requests(case)
        page = case["page"]
        width = max(_pages_of(max(n, min(n, k) + c), page) for n, k, c in zip(held, keep, count)) + 1
        # as many free pages as are needed, or (tight) about half of them
        extra = sum(_pages_of(c, page) + 1 for c in count) // (2 if case["tight"] else 1)
        s["table"], s["free"] = _table(gen, held, page, extra, width)
        s["free_count"] = whole([extra], torch.int32)
        s["length"], s["keep"], s["count"] = whole(held, torch.int64), whole(keep, torch.int64), whole(count, torch.int32)
        rows = max(1, sum(count) + case["pad"])
        s["slot"], s["at"] = (torch.zeros(rows, dtype=torch.int64, device="cuda") for _ in range(2))
        s["first"], s["granted"] = (torch.zeros(case["batch"], dtype=torch.int32, device="cuda") for _ in range(2))
        return s
    if op == "write":
        n = case["n"]
        s["k"], s["v"] = (_activations(gen, n, case["kv_heads"]) for _ in range(2))
        pages = _pages_of(n, case["page"]) + 5
        make = lambda w: torch.zeros(pages, case["kv_heads"], case["page"], w, dtype=torch.uint8, device="cuda")
        w = (D * case["bits"] // 8, D // GROUP)
        s["pool"] = dict(k_codes=make(w[0]), k_step=make(w[1]), v_codes=make(w[0]), v_step=make(w[1]))
        order = torch.randperm(pages, generator=gen, device="cuda")
        i = torch.arange(n, device="cuda")
        slot = order[i // case["page"]] * case["page"] + i % case["page"]
        s["slot"] = torch.where(i % 7 < 7 - case["skip"], slot, -1)
        s["at"] = i + case["start"] if case["rope"] else None
        s["weight"] = _weight(gen, D) if case["norm"] else None
        s["k_hat"], s["v_hat"] = (torch.zeros(case["kv_heads"], n, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        return s
    lengths, counts = _sequences(case)
    need = sum(_pages_of(n, case["page"]) for n in lengths)
    width = max(_pages_of(n, case["page"]) for n in lengths) + 1
    s["table"], s["free"] = _table(gen, lengths, case["page"], need // 10 + 1, width)
    s["free_count"] = whole([need // 10 + 1], torch.int32)
    s["pool"] = _pool(gen, case, need + need // 10 + 1)
    s["length"], s["count"] = whole(lengths, torch.int64), whole(counts, torch.int32)
    s["first"] = (torch.cumsum(s["count"], 0) - s["count"]).to(torch.int32)
    n = sum(counts) + case["pad"]
    s["q"] = _activations(gen, n, case["heads"])
    s["out"] = torch.zeros(n, case["heads"], D, dtype=torch.bfloat16, device="cuda").permute(1, 0, 2)
    s["lse"] = torch.zeros(case["heads"], n, dtype=torch.float32, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms


def _axes(case):
    """Per channel pair: its axis and the exponent of its frequency, and the pair's two channels."""
    dims = [case["axis_t"], case["axis_y"], case["axis_x"]]
    axis = torch.cat([torch.full((m // 2,), a) for a, m in enumerate(dims)])
    power = torch.cat([torch.arange(m // 2, dtype=torch.float64) * 2 / max(m, 1) for m in dims])
    half = axis.numel()
    i = torch.arange(half)
    first, second = (2 * i, 2 * i + 1) if case["pairing"] == "interleaved" else (i, i + half)
    return axis.cuda(), power.cuda(), first.cuda(), second.cuda()


def _turn(x, case, p):
    """x fp32 [..][n][128] turned by the positions p [..][n] (angles in 64 bits)."""
    axis, power, first, second = _axes(case)
    pos = torch.stack([p // (case["gh"] * case["gw"]), p // case["gw"] % case["gh"], p % case["gw"]], -1)[..., axis].double()
    angle = torch.remainder(pos * case["theta"] ** -power, 2 * math.pi)
    c, s = torch.cos(angle).float(), torch.sin(angle).float()
    out = x.clone()
    a, b = x[..., first], x[..., second]
    out[..., first] = a * c - b * s
    out[..., second] = a * s + b * c
    return out


def _norm(x, w):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w


def _grid(bits):
    """The steps (fp32) in the order of their bytes, up to the largest."""
    table = (torch.arange(248, dtype=torch.int16) << 7).view(torch.float16).float()
    return table[table <= (56.0 if bits == 8 else 896.0)].cuda()


def _quantise(x, bits):
    """fp32 rows [..][128] -> signed codes (fp32) and the steps' bytes."""
    top, table = 127 if bits == 8 else 7, _grid(bits)
    g = x.reshape(*x.shape[:-1], D // GROUP, GROUP)
    step = torch.searchsorted(table * top, g.abs().amax(-1)).clamp(max=table.numel() - 1)
    s = table[step][..., None]
    q = torch.where(s > 0, torch.round(g / torch.where(s > 0, s, 1.0)), 0.0).clamp(-top, top)
    return q.reshape(x.shape), step.to(torch.uint8)


def _pack(q, bits):
    if bits == 8:
        return (q + 128).to(torch.uint8)
    u = (q + 8).to(torch.uint8).reshape(*q.shape[:-1], D // 8, 4, 2)   # word, k, t
    n = u.transpose(-1, -2).reshape(*q.shape[:-1], D // 8, 4, 2)       # nibble k + 4 t, two to a byte
    return (n[..., 0] | (n[..., 1] << 4)).reshape(*q.shape[:-1], D // 2)


def _values(codes, step, bits):
    """What the cache stands for, fp32 [..][128]."""
    if bits == 8:
        q = codes.float() - 128
    else:
        n = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], D // 8, 2, 4)   # t, k
        q = n.transpose(-1, -2).reshape(*codes.shape[:-1], D).float() - 8
    s = (step.to(torch.int16) << 7).view(torch.float16).float()
    return (q.reshape(*q.shape[:-1], D // GROUP, GROUP) * s[..., None]).reshape(q.shape)


def _plain_pages(s):
    page, table, length = s["case"]["page"], s["table"], s["length"]
    rows, pages, b = s["slot"].numel(), s["free"].numel(), table.shape[0]
    held = lambda n: (n + page - 1) // page
    i = torch.arange(table.shape[1], device="cuda")
    sums = lambda v: torch.cumsum(v, 0)
    # the free pages, and one more place for what is not to be written
    free = torch.cat([s["free"], s["free"].new_zeros(1)])
    kept = torch.minimum(length, s["keep"].clamp(min=0))
    drop = held(length) - held(kept)
    gone = (i >= held(kept)[:, None]) & (i < held(length)[:, None])
    number = (sums(drop) - drop - held(kept))[:, None] + i
    count = s["free_count"][0].long() + drop.sum()
    free[torch.where(gone, count - 1 - number, pages)] = table
    table.masked_fill_(gone, -1)
    # new tokens
    want = s["count"].clamp(min=0).long()
    first = sums(want) - want
    fits = (first + want <= rows) & (held(kept + want) <= table.shape[1])
    need = torch.where(fits, held(kept + want) - held(kept), 0)
    granted = torch.where(fits & ((need == 0) | (sums(need) <= count)), want, 0)
    after = kept + granted
    fresh = (i >= held(kept)[:, None]) & (i < held(after)[:, None])
    number = (sums(need) - need - held(kept))[:, None] + i
    table.copy_(torch.where(fresh, free[torch.where(fresh, count - 1 - number, pages)], table))
    left = count - (held(after) - held(kept)).sum()
    s["free"].copy_(torch.where(torch.arange(pages, device="cuda") < left, free[:pages], -1))
    s["free_count"].copy_(left[None])
    length.copy_(after)
    s["first"].copy_(first)
    s["granted"].copy_(granted)
    r = torch.arange(rows, device="cuda")
    seq = (torch.searchsorted(first, r, right=True) - 1).clamp(0, b - 1)
    live = r - first[seq] < granted[seq]
    at = torch.where(live, kept[seq] + r - first[seq], -1)
    s["at"].copy_(at)
    s["slot"].copy_(torch.where(live, table[seq, (at // page).clamp(min=0)].long() * page + at % page, -1))
    return {"table": table, "length": length, "free": s["free"], "free_count": s["free_count"], "first": s["first"],
            "granted": s["granted"], "slot": s["slot"], "at": s["at"]}


def _plain_write(s):
    case, pool, slot = s["case"], s["pool"], s["slot"]
    page, bits = case["page"], case["bits"]
    k = s["k"].float()
    if case["norm"]:
        k = _norm(k, s["weight"])
    if case["rope"]:
        k = _turn(k, case, s["at"][None])
    kept = slot >= 0
    there, within = slot[kept].div(page, rounding_mode="floor"), slot[kept] % page
    out = {}
    for t, x in (("k", k.to(torch.bfloat16).float()), ("v", s["v"].float())):
        q, step = _quantise(x, bits)
        pool[t + "_codes"][there, :, within] = _pack(q, bits).transpose(0, 1)[kept]
        pool[t + "_step"][there, :, within] = step.transpose(0, 1)[kept]
        hat = _values(pool[t + "_codes"][there, :, within], pool[t + "_step"][there, :, within], bits)
        s[t + "_hat"].zero_()
        s[t + "_hat"][:, kept] = hat.transpose(0, 1).to(torch.bfloat16)
        out[t + "_hat"] = s[t + "_hat"]
    return out


def _plain_attend(s):
    case, pool = s["case"], s["pool"]
    b, h, kv, tpf = case["batch"], case["heads"], case["kv_heads"], case["tpf"]
    counts = _sequences(case)[1]
    nq, n = max(1, max(counts)), s["q"].shape[1]
    table = s["table"].clamp(min=0).long()
    dense = lambda t: pool[t][table].transpose(2, 3).flatten(1, 2).transpose(1, 2)   # [batch][kv_heads][tokens][..]
    k = _values(dense("k_codes"), dense("k_step"), case["bits"])
    v = _values(dense("v_codes"), dense("v_step"), case["bits"])
    i = torch.arange(nq, device="cuda")
    row = (s["first"].long()[:, None] + i).clamp(max=n - 1)
    fq = ((s["length"] - s["count"])[:, None] + i).div(tpf, rounding_mode="floor")[:, :, None]
    j = torch.arange(k.shape[2], device="cuda")
    fk = j // tpf
    hidden = ~((j < s["length"][:, None])[:, None] & (fk <= fq) & ((fq - fk < case["frames"]) | (j < case["sink"])))
    q = s["q"].float()[:, row].transpose(0, 1).reshape(b, kv, (h // kv) * nq, D)
    x = torch.matmul(q, k.transpose(-1, -2)).view(b, kv, h // kv, nq, -1)
    x.mul_(LOG2E / math.sqrt(D)).masked_fill_(hidden[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x.sub_(torch.where(m == -math.inf, 0.0, m)).exp2_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(b, kv, (h // kv) * nq, -1), v).view(b, h, nq, D) / torch.where(total > 0, total, 1.0).view(b, h, nq, 1)
    lse = (m + torch.log2(total)).view(b, h, nq)
    r = torch.arange(n, device="cuda")
    seq = torch.searchsorted(s["first"], r.to(torch.int32), right=True) - 1
    place = r - s["first"][seq]
    live = place < s["count"][seq]
    place = place.clamp(max=nq - 1)
    s["out"].copy_(torch.where(live[:, None], o[seq, :, place].transpose(0, 1), s["out"].float()))
    s["lse"].copy_(torch.where(live, lse[seq, :, place].transpose(0, 1), s["lse"]))
    return {"out": s["out"], "lse": s["lse"]}


def _plain(s):
    op = s["case"]["op"]
    if op == "norm":
        p = s["at"] if s["at"] is not None else s["start"][:, None] + torch.arange(s["case"]["n"], device="cuda")
        w = s["weight"][:, None] if s["case"]["per_head"] else s["weight"]
        return _turn(_norm(s["x"].float(), w), s["case"], p[:, None]).to(torch.bfloat16)
    return _plain_pages(s) if op == "pages" else _plain_write(s) if op == "write" else _plain_attend(s)


# ------------------------------------------------------------------ the package's calls


@functools.lru_cache(maxsize=None)
def _context(heads):
    import bit_kv_cache_qsac_gb300 as qwm
    return qwm.Context(heads=heads)


@functools.lru_cache(maxsize=None)
def _spec(dims, theta, pairing, gh, gw):
    import bit_kv_cache_qsac_gb300 as qwm
    return qwm.RopeSpec(dims, theta=theta, pairing=pairing, grid=(gh, gw))


@functools.lru_cache(maxsize=None)
def _largest(items):
    """The largest number of new tokens of a sequence, which a program that plans its batches knows."""
    return max(_sequences(dict(items))[1])


def _spec_of(case):
    return _spec((case["axis_t"], case["axis_y"], case["axis_x"]), case["theta"], case["pairing"], case["gh"], case["gw"])


def _own(s):
    import bit_kv_cache_qsac_gb300 as qwm
    case = s["case"]
    if case["op"] == "norm":
        out = torch.empty(s["x"].shape, dtype=torch.bfloat16, device="cuda")
        qwm.qwm_norm_rope(_context(case["heads"]), _spec_of(case), s["x"], s["weight"], EPS, out, start=s["start"], at=s["at"])
        return out
    if case["op"] == "write":
        ctx, pool = _context(case["kv_heads"]), qwm.PagePool(case["bits"], **s["pool"])
        qwm.qwm_paged_write(ctx, pool, s["k"], s["v"], s["slot"], at=s["at"], rope=_spec_of(case) if case["rope"] else None, weight=s["weight"], eps=EPS)
        qwm.qwm_paged_read(ctx, pool, s["slot"], s["k_hat"], s["v_hat"])
        return {"k_hat": s["k_hat"], "v_hat": s["v_hat"]}
    tab = qwm.PageTable(case["page"], s["table"], s["length"], s["free"], s["free_count"])
    if case["op"] == "pages":
        qwm.qwm_pages_update(_context(1), tab, s["first"], s["granted"], s["slot"], s["at"], count=s["count"], keep=s["keep"])
        return {"table": tab.table, "length": tab.length, "free": tab.free, "free_count": tab.free_count, "first": s["first"],
                "granted": s["granted"], "slot": s["slot"], "at": s["at"]}
    qwm.qwm_paged_attend(_context(case["heads"]), qwm.PagePool(case["bits"], **s["pool"]), tab, s["q"], s["first"], s["count"], 1.0 / math.sqrt(D),
                         s["out"], lse=s["lse"], tpf=case["tpf"], frames=case["frames"], sink=case["sink"], max_count=_largest(tuple(case.items())))
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ the definitions in 64 bits


def _rotated64(x, case, p):
    """x float64 [heads][n][128] of tokens at positions p: each pair as a complex number."""
    dims = (case["axis_t"], case["axis_y"], case["axis_x"])
    half = sum(dims) // 2
    coord = (p // (case["gh"] * case["gw"]), (p // case["gw"]) % case["gh"], p % case["gw"])
    y, i = x.clone(), 0
    for a, m in enumerate(dims):
        for j in range(m // 2):
            c0, c1 = (2 * i, 2 * i + 1) if case["pairing"] == "interleaved" else (i, i + half)
            turn = torch.polar(torch.ones_like(p, dtype=torch.float64), coord[a].double() * case["theta"] ** -(2.0 * j / m))
            z = torch.complex(x[..., c0], x[..., c1]) * turn
            y[..., c0], y[..., c1] = z.real, z.imag
            i += 1
    return y


def _normed64(x, w):
    return x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + EPS) * w.double()


def _rounded64(x, bits):
    """Quantised float64 values of rows [..][128]."""
    top = 127.0 if bits == 8 else 7.0
    e, f = torch.meshgrid(torch.arange(31, dtype=torch.float64), torch.arange(8, dtype=torch.float64), indexing="ij")
    steps = torch.where(e > 0, (1 + f / 8) * 2 ** (e - 15), f / 8 * 2.0 ** -14).reshape(-1).to(x.device)
    steps = steps[steps <= (56 if bits == 8 else 896)]
    g = x.reshape(-1, D // GROUP, GROUP)
    s = steps[torch.bucketize(g.abs().amax(-1) / top, steps).clamp(max=steps.numel() - 1)][..., None]
    return torch.where(s > 0, (g / s.clamp(min=1e-30)).round().clamp(-top, top) * s, torch.zeros_like(g)).reshape(x.shape)


def _decoded64(codes, step, bits):
    c, d = codes.to(torch.int64), torch.arange(D, device=codes.device)
    if bits == 8:
        q = c - 128
    else:
        nibble = (d % 8) // 2 + 4 * (d % 2)
        q = ((c[:, (d // 8) * 4 + nibble // 2] >> (4 * (nibble % 2))) & 15) - 8
    b = step.to(torch.int64)
    e, f = b >> 3, (b & 7).double()
    s = torch.where(e > 0, (1 + f / 8) * 2.0 ** (e - 15).double(), f / 8 * 2.0 ** -14)
    return q.double() * s[:, d // GROUP]


def exact(case, seed):
    if case["op"] == "pages":
        return None   # whole numbers
    s = prepare(case, seed)
    if case["op"] == "norm":
        out = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda")
        for i in range(case["batch"]):
            p = s["at"][i] if case["packed"] else s["start"][i] + torch.arange(case["n"], device="cuda")
            w = s["weight"][:, None] if case["per_head"] else s["weight"]
            out[i] = _rotated64(_normed64(s["x"][i].double(), w), case, p)
        return out
    if case["op"] == "write":
        k = s["k"].double()
        if case["norm"]:
            k = _normed64(k, s["weight"])
        if case["rope"]:
            k = _rotated64(k, case, s["at"])
        kept = (s["slot"] >= 0)[:, None]
        return {"k_hat": torch.where(kept, _rounded64(k.to(torch.bfloat16).double(), case["bits"]), 0.0),
                "v_hat": torch.where(kept, _rounded64(s["v"].double(), case["bits"]), 0.0)}
    g, page, pool = case["heads"] // case["kv_heads"], case["page"], s["pool"]
    out, lse = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda"), torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    row = 0
    for b, (n, c) in enumerate(zip(*_sequences(case))):
        if not c:
            continue
        j = torch.arange(n, device="cuda")
        frame = (torch.arange(c, device="cuda") + n - c) // case["tpf"]
        seen = (j // case["tpf"] <= frame[:, None]) & ((j // case["tpf"] > frame[:, None] - case["frames"]) | (j < case["sink"]))
        held = seen.any(0).nonzero()[:, 0]
        seen, where = seen[:, held], (s["table"][b].long()[held // page], held % page)
        for h in range(case["kv_heads"]):
            kh, vh = (_decoded64(pool[t + "_codes"][where[0], h, where[1]], pool[t + "_step"][where[0], h, where[1]], case["bits"]) for t in "kv")
            for r in range(h * g, (h + 1) * g):
                logits = (s["q"][r, row:row + c].double() @ kh.T / math.sqrt(D)).masked_fill(~seen, -math.inf)
                out[r, row:row + c] = torch.softmax(logits, -1) @ vh
                lse[r, row:row + c] = torch.logsumexp(logits, -1) / math.log(2.0)
        row += c
    return {"out": out, "lse": lse}
