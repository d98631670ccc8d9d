"""Workloads of the recent-window operators: rotary positions with three axes, the 8- and 4-bit
window cache (quantised as it is written, read back), and attention over that cache with a sliding
window and sink tokens.

`run(state)` computes one pass: in elementary torch operations in 32 bits (`own` false), or through
the package's calls (`own` true).  `exact(case, seed)` computes the same from the definitions in 64
bits.

The definitions.
- Rotary: token (t, y, x) turns channel pair i of axis a by position_a * theta^(-2 i / dim_a).
- Cache: per token and head, groups of 32 channels; the step s is the smallest number with 5
  exponent and 3 mantissa bits (the top byte of an fp16 below its sign) with Q s >= max|x|, Q = 127
  or 7, at most 56 (8 bits) or 896 (4 bits); the code is rint(x / s), stored plus 128 or 8; the cache
  stands for s times the code.  Four-bit codes: channel 8 j + 2 k + t is nibble k + 4 t of 32-bit word
  j.  Keys are turned and rounded to bf16 before they are quantised.  Token p lives in slot p while p < sink, else in slot
  sink + (p - sink) % ring.
- Attention: Query row i stands at position q_start + i, in frame position // tpf.  It sees a key j
  that is still held when frame(j) <= frame(i) and (frame(i) - frame(j) < frames or j < sink).  The
  output of a row that sees none is 0 and its log-sum-exp -inf.
"""
import functools
import math

import torch

own = False

D, GROUP = 128, 32
LOG2E = 1.4426950408889634

# ------------------------------------------------------------------ cases


def listed():
    # 40 heads, frames of 30 x 52 (480p) and 45 x 80 (720p) latent tokens and chunks of three frames are
    # the layer shapes of this repository's workloads; the others are generic serving shapes.
    wan = dict(axis_t=44, axis_y=42, axis_x=42, theta=10000.0, pairing="interleaved", shared=False)
    text = dict(axis_t=128, axis_y=0, axis_x=0, theta=1000000.0, pairing="half", shared=False)
    return [
        # one generated token of each of 16 sequences, far into them: latency
        dict(text, name="rope_token", op="rope", batch=16, heads=32, n=1, gh=1, gw=1, start=900000),
        # the Queries of one 720p chunk as the projection leaves them (token-major)
        dict(wan, name="rope_chunk_720p", op="rope", batch=1, heads=40, n=10800, gh=45, gw=80, start=75600),
        # one token of each of 16 sequences written and read back: latency
        dict(text, name="write_token", op="write", bits=8, batch=16, kv_heads=8, n=1, gh=1, gw=1, sink=4, ring=4092,
             start=9000, rope=True, ragged=False),
        # a padded batch of odd lengths, written without rotation across the end of the ring
        dict(text, name="write_ragged", op="write", bits=4, batch=5, kv_heads=8, n=777, gh=1, gw=1, sink=3, ring=1999,
             start=1500, rope=False, ragged=True),
        # one 720p chunk: rotated, quantised and handed back in bf16 (for packing)
        dict(wan, name="write_chunk_720p", op="write", bits=4, batch=1, kv_heads=40, n=10800, gh=45, gw=80, sink=3600,
             ring=39600, start=75600, rope=True, ragged=False),
        # a 480p chunk read back as its frames leave the window
        dict(name="read_chunk_480p", op="read", bits=8, batch=1, kv_heads=40, n=4680, sink=1560, ring=37440,
             length=51480, back=14040),
        # one token of 16 sequences, grouped heads, a wrapped window of 4,092 tokens and 4 sinks
        dict(name="attend_token_batch", op="attend", bits=8, batch=16, heads=32, kv_heads=8, nq=1, sink=4, ring=4092,
             length=9001, tpf=1, frames=4092, ragged=False),
        # one token of one stream over 39,000 cached tokens: the cache's bytes count
        dict(name="attend_token_stream", op="attend", bits=4, batch=1, heads=40, kv_heads=40, nq=1, sink=1560,
             ring=37440, length=51480, tpf=1, frames=37440, ragged=False),
        # a few drafted tokens of sequences of different lengths, one of them empty
        dict(name="attend_drafts_ragged", op="attend", bits=4, batch=7, heads=24, kv_heads=8, nq=5, sink=3, ring=1999,
             length=2777, tpf=1, frames=1500, ragged=True),
        # a prompt under a sliding window of 1,024 tokens: most tiles are masked away
        dict(name="attend_prompt", op="attend", bits=8, batch=2, heads=32, kv_heads=8, nq=2111, sink=16, ring=4096,
             length=4103, tpf=1, frames=1024, ragged=False),
        # one 480p chunk over 24 frames of history, block-causal over frames
        dict(name="attend_chunk_480p", op="attend", bits=8, batch=1, heads=40, kv_heads=40, nq=4680, sink=1560,
             ring=40560, length=60840, tpf=1560, frames=24, ragged=False),
        # one 720p frame over ten frames of history and the first one
        dict(name="attend_frame_720p", op="attend", bits=4, batch=1, heads=40, kv_heads=40, nq=3600, sink=3600,
             ring=39600, length=79200, tpf=3600, frames=11, ragged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "attend", "attend"])
    axes = rng.choice([dict(axis_t=44, axis_y=42, axis_x=42, theta=10000.0), dict(axis_t=16, axis_y=56, axis_x=56, theta=256.0),
                       dict(axis_t=128, axis_y=0, axis_x=0, theta=500000.0), dict(axis_t=32, axis_y=16, axis_x=16, theta=10000.0)])
    turn = dict(axes, pairing=rng.choice(["interleaved", "half"]), shared=rng.random() < 0.3, gh=rng.randint(1, 45),
                gw=rng.randint(1, 80))
    batch = rng.choice([1, 1, 2, 3, 5, 8, 16])
    bits = rng.choice([8, 4])
    sink, ring = rng.choice([0, 1, 4, rng.randint(5, 200), rng.randint(200, 4000)]), _log(rng, 50, 40000)
    if op == "rope":
        heads = rng.choice([1, 8, 24, 32, 40])
        return dict(turn, op=op, batch=batch, heads=heads, n=max(1, _log(rng, 1, 432000) // (heads * batch)), start=_log(rng, 1, 2000000))
    kv = rng.choice([1, 2, 4, 8, 40])
    if op == "write":
        n = min(ring, max(1, _log(rng, 1, 432000) // (kv * batch)))
        return dict(turn, op=op, bits=bits, batch=batch, kv_heads=kv, n=n, sink=sink, ring=ring, start=_log(rng, 1, 200000),
                    rope=rng.random() < 0.6, ragged=rng.random() < 0.4)
    length = _log(rng, 1, 3 * (sink + ring))
    if op == "read":
        n = max(1, _log(rng, 1, 180000) // (kv * batch))
        return dict(op=op, bits=bits, batch=batch, kv_heads=kv, n=n, sink=sink, ring=ring, length=length,
                    back=rng.randint(1, length))
    heads = kv * rng.choice([1, 1, 2, 4, 5, 8] if kv <= 8 else [1])
    nq = _log(rng, 1, 4700)
    while batch * heads * nq * (sink + ring) > 6_000_000_000 or batch * heads * nq > 190_000:
        nq, batch = max(1, nq // 2), max(1, batch - 1)
        if nq == 1:
            ring = max(50, ring // 2)
            length = min(length, 3 * (sink + ring))
    tpf = rng.choice([1, 1, 1, 16, 390, 1560])
    return dict(op=op, bits=bits, batch=batch, heads=heads, kv_heads=kv, nq=nq, sink=sink, ring=ring, length=length, tpf=tpf,
                frames=max(1, _log(rng, 1, sink + ring) // tpf), ragged=rng.random() < 0.4)


def _lengths(case):
    """Tokens of each sequence: equal, or (ragged) falling to 0."""
    b, n = case["batch"], case["length"]
    return [n * (b - 1 - i) // max(1, b - 1) if b > 1 else n for i in range(b)] if case["ragged"] else [n] * b


def _counts(case):
    b, n = case["batch"], case["n"]
    return [n * (b - i) // b for i in range(b)] if case["ragged"] else None


def work(case):
    op, b = case["op"], case["batch"]
    if op == "rope":
        return {"bytes": 4 * D * b * case["heads"] * case["n"], "flops": 3 * D * b * case["heads"] * case["n"]}
    row = D * case["bits"] // 8 + D // GROUP   # a cached Key or Value row of one head
    if op in ("write", "read"):
        tokens = (sum(_counts(case) or [case["n"] * b]) if op == "write" else b * case["n"]) * case["kv_heads"]
        return {"bytes": tokens * 2 * (2 * D + row) + (tokens * 2 * (2 * D + row) if op == "write" else 0),
                "flops": tokens * 2 * D * (4 if op == "write" else 1)}
    pairs = held = 0
    for n in _lengths(case):
        p = torch.arange(case["nq"], dtype=torch.int64) + max(0, n - case["nq"])
        f = p // case["tpf"]
        hi = torch.clamp((f + 1) * case["tpf"], max=n)
        sink = torch.clamp(hi, max=case["sink"])
        lo = torch.clamp((f - case["frames"] + 1) * case["tpf"], min=max(case["sink"], n - case["ring"]))
        seen = torch.clamp(hi - lo, min=0)
        pairs += int((sink + seen).sum())
        held += int(sink.max()) + max(0, int(hi.max()) - int(lo.min()))
    rows = b * case["heads"] * case["nq"]
    return {"bytes": held * case["kv_heads"] * 2 * row + rows * (4 * D + 4), "flops": 4 * D * pairs * case["heads"]}


# ------------------------------------------------------------------ inputs


def _activations(gen, *shape):
    """bf16 rows as a projection leaves them: unit noise, eight outlier channels, token-major memory
    seen as [batch][heads][tokens][128]."""
    b, h, n, d = shape
    x = torch.randn(b, n, h, d, generator=gen, device="cuda", dtype=torch.float32)
    x[..., torch.randperm(d, generator=gen, device="cuda")[:8]] *= 4.0
    return x.to(torch.bfloat16).permute(0, 2, 1, 3)


def _cache(gen, case, codes_of):
    """A written cache of one tensor: (codes, steps)."""
    slots = case["sink"] + case["ring"]
    x = _activations(gen, case["batch"], case["kv_heads"], slots, D)
    q, step = codes_of(x.float(), case["bits"])
    return _pack(q, case["bits"]), step


def _empty_cache(case):
    shape = (case["batch"], case["kv_heads"], case["sink"] + case["ring"])
    make = lambda w: torch.zeros(*shape, w, dtype=torch.uint8, device="cuda")
    return dict(k_codes=make(D * case["bits"] // 8), v_codes=make(D * case["bits"] // 8), k_step=make(D // GROUP), v_step=make(D // GROUP))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 11)
    s = {"case": dict(case)}
    b = case["batch"]
    whole = lambda v, t: torch.tensor(v, dtype=t, device="cuda")
    if case["op"] == "rope":
        s["x"] = _activations(gen, b, case["heads"], case["n"], D)
        s["start"] = whole([case["start"] + 37 * i for i in range(b)], torch.int64)
        return s
    if case["op"] == "write":
        s["k"], s["v"] = (_activations(gen, b, case["kv_heads"], case["n"], D) for _ in range(2))
        s["cache"] = _empty_cache(case)
        s["start"] = whole([case["start"] + 37 * i for i in range(b)], torch.int64)
        counts = _counts(case)
        s["count"] = whole(counts, torch.int32) if counts else None
        s["length"] = s["start"] + (s["count"].to(torch.int64) if counts else case["n"])
        s["k_hat"], s["v_hat"] = (torch.zeros(b, case["kv_heads"], case["n"], D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        return s
    s["cache"] = {}
    s["cache"]["k_codes"], s["cache"]["k_step"] = _cache(gen, case, _quantise)
    s["cache"]["v_codes"], s["cache"]["v_step"] = _cache(gen, case, _quantise)
    if case["op"] == "read":
        s["length"] = whole([case["length"]] * b, torch.int64)
        s["start"] = s["length"] - case["back"]
        s["k_hat"], s["v_hat"] = (torch.zeros(b, case["kv_heads"], case["n"], D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        return s
    lengths = _lengths(case)
    s["length"] = whole(lengths, torch.int64)
    s["q_start"] = whole([max(0, n - case["nq"]) for n in lengths], torch.int64)
    s["q"] = _activations(gen, b, case["heads"], case["nq"], D)
    return s


# ------------------------------------------------------------------ plain forms


def _axes(case):
    """Per channel pair: its axis and the exponent of its frequency, and the pair's two channels."""
    dims = [case["axis_t"], case["axis_y"], case["axis_x"]]
    axis = torch.cat([torch.full((m // 2,), a) for a, m in enumerate(dims)])
    local = torch.cat([torch.arange(m // 2, dtype=torch.float64) * 2 / max(m, 1) for m in dims])
    half = axis.numel()
    i = torch.arange(half)
    power = 2.0 * i.double() / (2 * half) if case["shared"] else local
    first, second = (2 * i, 2 * i + 1) if case["pairing"] == "interleaved" else (i, i + half)
    return axis.cuda(), power.cuda(), first.cuda(), second.cuda()


def _turn(x, case, start):
    """x fp32 [b][h][n][128] turned by its positions (angles in 64 bits)."""
    axis, power, first, second = _axes(case)
    p = start[:, None] + torch.arange(x.shape[2], device=x.device)
    plane = case["gh"] * case["gw"]
    pos = torch.stack([p // plane, p // case["gw"] % case["gh"], p % case["gw"]], -1)[..., axis].double()
    angle = torch.remainder(pos * case["theta"] ** -power, 2 * math.pi)
    c, s = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    out = x.clone()
    a, b = x[..., first], x[..., second]
    out[..., first] = a * c - b * s
    out[..., second] = a * s + b * c
    return out


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


def _held(length, sink, ring):
    """Position of the token in each slot [b][slots], and whether there is one."""
    slot = torch.arange(sink + ring, device=length.device)
    n = length[:, None]
    last = n - 1 - torch.remainder(n - 1 - slot, ring)   # the latest p < n with (p - sink) % ring == slot - sink
    pos = torch.where(slot < sink, slot.expand(n.shape[0], -1), last)
    return pos, torch.where(slot < sink, slot < n, last >= sink)


def _plain(s):
    case = s["case"]
    if case["op"] == "rope":
        return _turn(s["x"].float(), case, s["start"]).to(torch.bfloat16)
    sink, ring, bits = case["sink"], case["ring"], case["bits"]
    if case["op"] == "write":
        k = s["k"].float()
        if case["rope"]:
            k = _turn(k, case, s["start"]).to(torch.bfloat16).float()
        i = torch.arange(case["n"], device="cuda")
        p = s["start"][:, None] + i
        mine = i < s["count"][:, None] if s["count"] is not None else torch.ones_like(p, dtype=torch.bool)
        kept = mine & ((p < sink) | (p >= s["length"][:, None] - ring))
        out = {}
        for name, x in (("k_hat", k), ("v_hat", s["v"].float())):
            q, step = _quantise(x, bits)
            g = (step.to(torch.int16) << 7).view(torch.float16).float()[..., None]
            val = (q.reshape(*q.shape[:-1], D // GROUP, GROUP) * g).reshape(q.shape)
            out[name] = torch.where(kept[:, None, :, None], val, 0.0).to(torch.bfloat16)
        return out
    c = s["cache"]
    if case["op"] == "read":
        p = s["start"][:, None] + torch.arange(case["n"], device="cuda")
        n = s["length"][:, None]
        held = (p < n) & ((p < sink) | (p >= n - ring))
        slot = torch.where(p < sink, p, sink + (p - sink).remainder(ring))
        at = slot[:, None, :, None].expand(-1, case["kv_heads"], -1, -1)
        pick = lambda t: torch.gather(t, 2, at.expand(-1, -1, -1, t.shape[-1]))
        return {name + "_hat": torch.where(held[:, None, :, None], _values(pick(c[name + "_codes"]), pick(c[name + "_step"]), bits), 0.0)
                .to(torch.bfloat16) for name in ("k", "v")}
    b, h, nq, _ = s["q"].shape
    kv = case["kv_heads"]
    k, v = _values(c["k_codes"], c["k_step"], bits), _values(c["v_codes"], c["v_step"], bits)
    pos, held = _held(s["length"], sink, ring)
    fq = (s["q_start"][:, None] + torch.arange(nq, device="cuda")).div(case["tpf"], rounding_mode="floor")[:, :, None]
    fk = pos.div(case["tpf"], rounding_mode="floor")[:, None, :]
    hidden = ~(held[:, None, :] & (fk <= fq) & ((fq - fk < case["frames"]) | (pos < sink)[:, None, :]))
    q = s["q"].float().reshape(b, kv, (h // kv) * nq, D)
    x = torch.matmul(q, k.transpose(-1, -2)).view(b, kv, h // kv, nq, -1)
    x.mul_(LOG2E / math.sqrt(D)).masked_fill_(hidden[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x.sub_(torch.where(m == -math.inf, 0.0, m)).exp2_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(b, kv, (h // kv) * nq, -1), v).view(b, kv, h // kv, nq, D) / torch.where(total > 0, total, 1.0)
    return {"out": o.reshape(b, h, nq, D).to(torch.bfloat16), "lse": (m + torch.log2(total)).reshape(b, h, nq)}


# ------------------------------------------------------------------ the package's calls


@functools.lru_cache(maxsize=None)
def _context(heads):
    import bit_kv_cache_qsac_gb300 as qwm
    return qwm.Context(heads=heads)


@functools.lru_cache(maxsize=None)
def _spec(dims, theta, pairing, shared, gh, gw):
    import bit_kv_cache_qsac_gb300 as qwm
    return qwm.RopeSpec(dims, theta=theta, pairing=pairing, shared_freq=shared, grid=(gh, gw))


def _own(s):
    import bit_kv_cache_qsac_gb300 as qwm
    case = s["case"]
    spec = None
    if case["op"] == "rope" or case.get("rope"):
        spec = _spec((case["axis_t"], case["axis_y"], case["axis_x"]), case["theta"], case["pairing"], case["shared"], case["gh"], case["gw"])
    if case["op"] == "rope":
        out = torch.empty(s["x"].shape, dtype=torch.bfloat16, device="cuda")
        qwm.qwm_rope(_context(case["heads"]), spec, s["x"], s["start"], out)
        return out
    win = qwm.Window(case["bits"], case["sink"], case["ring"], **s["cache"])
    ctx = _context(case.get("heads", case["kv_heads"]))
    if case["op"] == "write":
        qwm.qwm_window_write(ctx, win, s["k"], s["v"], s["start"], count=s["count"], rope=spec)
    if case["op"] in ("write", "read"):
        qwm.qwm_window_read(ctx, win, s["start"], s["length"], s["k_hat"], s["v_hat"], count=s.get("count"))
        return {"k_hat": s["k_hat"], "v_hat": s["v_hat"]}
    q = s["q"]
    out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device="cuda")
    qwm.qwm_window_attend(ctx, win, q, s["q_start"], s["length"], case["tpf"], case["frames"], 1.0 / math.sqrt(D), out, lse=lse)
    return {"out": out, "lse": lse}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ the definitions in 64 bits


def _rotated64(x, case, start):
    """x float64 [heads][n][128] of tokens start, start + 1, ...: each pair as a complex number."""
    dims = (case["axis_t"], case["axis_y"], case["axis_x"])
    half = sum(dims) // 2
    p = torch.arange(start, start + x.shape[1], dtype=torch.int64, device=x.device)
    coord = (p // (case["gh"] * case["gw"]), (p // case["gw"]) % case["gh"], p % case["gw"])
    y, i = x.clone(), 0
    for a, m in enumerate(dims):
        for j in range(m // 2):
            rate = case["theta"] ** (-(i / half if case["shared"] else 2.0 * j / m))
            c0, c1 = (2 * i, 2 * i + 1) if case["pairing"] == "interleaved" else (i, i + half)
            turn = torch.polar(torch.ones_like(p, dtype=torch.float64), coord[a].double() * rate)
            z = torch.complex(x[..., c0], x[..., c1]) * turn
            y[..., c0], y[..., c1] = z.real, z.imag
            i += 1
    return y


def _rounded64(x, bits):
    """Quantised float64 values of rows [n][128]."""
    top = 127.0 if bits == 8 else 7.0
    e, f = torch.meshgrid(torch.arange(31, dtype=torch.float64), torch.arange(8, dtype=torch.float64), indexing="ij")
    steps = torch.where(e > 0, (1 + f / 8) * 2 ** (e - 15), f / 8 * 2.0 ** -14).reshape(-1).to(x.device)
    steps = steps[steps <= (56 if bits == 8 else 896)]
    g = x.reshape(-1, D // GROUP, GROUP)
    amax = g.abs().amax(-1)
    s = steps[torch.bucketize(amax / top, steps).clamp(max=steps.numel() - 1)][..., None]
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
    s = prepare(case, seed)
    b = case["batch"]
    if case["op"] == "rope":
        out = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda")
        for i in range(b):
            out[i] = _rotated64(s["x"][i].double(), case, int(s["start"][i]))
        return out
    kv, sink, ring, bits = case["kv_heads"], case["sink"], case["ring"], case["bits"]
    if case["op"] in ("write", "read"):
        out = {n: torch.zeros(b, kv, case["n"], D, dtype=torch.float64, device="cuda") for n in ("k_hat", "v_hat")}
        for i in range(b):
            start, length = int(s["start"][i]), int(s["length"][i])
            count = min(case["n"], length - start)
            first = max(0, length - ring - start)      # the ring has lost the tokens before it
            keep = [j for j in range(count) if j >= first or start + j < sink]
            if not keep:
                continue
            at = torch.tensor(keep, device="cuda")
            p = at + start
            slot = torch.where(p < sink, p, sink + (p - sink) % ring)
            for n in ("k", "v"):
                rows = None
                if case["op"] == "write":
                    rows = s[n][i].double()
                    if n == "k" and case["rope"]:
                        rows = _rotated64(rows, case, start).to(torch.bfloat16).double()
                for h in range(kv):
                    out[n + "_hat"][i, h, at] = (_rounded64(rows[h, at], bits) if rows is not None else
                                                 _decoded64(s["cache"][n + "_codes"][i, h][slot], s["cache"][n + "_step"][i, h][slot], bits))
        return out
    g, nq = case["heads"] // kv, case["nq"]
    out = torch.zeros(b, case["heads"], nq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((b, case["heads"], nq), -math.inf, dtype=torch.float64, device="cuda")
    for i in range(b):
        length, q0 = int(s["length"][i]), int(s["q_start"][i])
        p = torch.cat([torch.arange(min(sink, length)), torch.arange(max(sink, length - ring), max(sink, length))]).cuda()
        if not p.numel():
            continue
        slot = torch.where(p < sink, p, sink + (p - sink) % ring)
        frame = (torch.arange(nq, device="cuda") + q0) // case["tpf"]
        seen = (p // case["tpf"] <= frame[:, None]) & ((p // case["tpf"] > frame[:, None] - case["frames"]) | (p < sink))
        some = seen.any(1)
        for h in range(kv):
            kh = _decoded64(s["cache"]["k_codes"][i, h][slot], s["cache"]["k_step"][i, h][slot], bits)
            vh = _decoded64(s["cache"]["v_codes"][i, h][slot], s["cache"]["v_step"][i, h][slot], bits)
            for r in range(h * g, (h + 1) * g):
                logits = (s["q"][i, r].double() @ kh.T / math.sqrt(D)).masked_fill(~seen, -math.inf)
                out[i, r][some] = torch.softmax(logits[some], -1) @ vh
                lse[i, r][some] = torch.logsumexp(logits[some], -1) / math.log(2.0)
    return {"out": out, "lse": lse}
