"""Cases of the 8-bit cache operators: rotary positions, packing records, sparse attention over
packed records, and the pages of the resident tier.

``run`` computes an operator in its plain form (elementary torch operations in 32 bits), or, where
``own`` is true, through the package's entry points on the same inputs.

Records are rows of e4m3 bytes, one per token: the K heads, then the V heads (or, ``latent``, one
head of ``k_dim`` values whose first ``v_dim`` are V as well).  ``scales[request][block][c]`` holds
the scale of head c (K heads, then V heads) over each block of ``block`` tokens.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn
TOP = 448.0            # the largest e4m3 value


# ---------------------------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------------------------
def _rotary(name, T, heads, k_heads, dim, rot, offset, interleaved, scaling, dtype, part, ctx):
    return dict(name=name, op="rotary", T=T, heads=heads, k_heads=k_heads, dim=dim, rot=rot,
                offset=offset, interleaved=interleaved, scaling=scaling, dtype=dtype,
                part=part, ctx=ctx)


def _pack(name, n, max_len, ragged, kv_heads, k_dim, v_dim, latent, block, start, rot, to, dtype):
    return dict(name=name, op="pack", n=n, max_len=max_len, ragged=ragged, kv_heads=kv_heads,
                k_dim=k_dim, v_dim=v_dim, latent=latent, block=block, start=start, rot=rot, to=to,
                dtype=dtype)


def _attend(name, R, V, n, pad, heads, kv_heads, k_dim, v_dim, latent, block, tokens, B, resident,
            ctx, dtype):
    return dict(name=name, op="attend", R=R, V=V, n=n, pad=pad, heads=heads, kv_heads=kv_heads,
                k_dim=k_dim, v_dim=v_dim, latent=latent, block=block, tokens=tokens, B=B,
                resident=resident, ctx=ctx, dtype=dtype)


def _pages(name, op, pages, layers, rows, row, R, blocks, live, n):
    return dict(name=name, op=op, pages=pages, layers=layers, rows=rows, row=row, R=R,
                blocks=blocks, live=live, n=n)


def listed():
    return [
        # The query of one decode step: 8 requests at 128K positions, 64 heads, the last 64 of 576
        # values rotated into the buffer whose first 512 another product has filled.
        _rotary("rotary_decode", 8, 64, 0, 576, 64, 512, False, "none", "bf16", True, 131072),
        # A prompt chunk with grouped heads: q and k, interleaved pairs, contexts stretched beyond
        # the trained length by parts; an odd token count.
        _rotary("rotary_prompt", 8191, 32, 8, 128, 128, 0, True, "parts", "bf16", False, 131072),
        # The new record of each of 64 requests in a decode step: latent head, rotated tail,
        # blocks that are open (their scale stands) and blocks that begin.
        _pack("pack_decode", 64, 1, False, 1, 576, 512, True, 64, "any", 64, "token", "bf16"),
        # Ragged prompts written by position: 8 heads of K and of V.
        _pack("pack_prompt", 8, 4096, True, 8, 128, 128, False, 64, "zero", 128, "position", "bf16"),
        # The smallest call: one request, 64 selections, 16 heads on one latent head.
        _attend("attend_tiny", 1, 1, 64, 3, 16, 1, 576, 512, True, 16, 1, 128, False, 4096, "bf16"),
        # One decode layer of token selection: 8 requests, 2048 of 128K positions.
        _attend("attend_tokens", 8, 1, 2048, 0, 64, 1, 576, 512, True, 64, 1, 4096, False, 131072,
                "bf16"),
        # The largest: 64 requests, 128 heads, some selections padded.
        _attend("attend_wide", 64, 1, 2048, 37, 128, 1, 576, 512, True, 64, 1, 4096, False,
                1048576, "bf16"),
        # Page selection: 16 requests, 128 pages of 16 tokens, 8 heads of 128 with groups of 4; the
        # newest page is part-filled.
        _attend("attend_pages", 16, 1, 128, 0, 32, 8, 128, 128, False, 16, 16, 256, False, 204793,
                "bf16"),
        # Verify rows in 16 bits: 4 rows of an odd 499 selections, every other row resident.
        _attend("attend_verify", 6, 4, 499, 11, 24, 4, 64, 64, False, 32, 1, 2304, True, 32768,
                "f16"),
        # Beams fork from their parents: the last, part-filled page of each is copied in 4 layers.
        _pages("pages_fork", "fork", 4096, 4, 64, 576, 96, 64, 0.5, 32),
        # A fragmented store is compacted: about a fifth of 1 GB moves.
        _pages("pages_compact", "compact", 7001, 4, 64, 576, 128, 96, 0.6, 0),
        # Requests end and others begin in a large store: only tables and counts change.
        _pages("pages_turnover", "turnover", 200003, 1, 1, 16, 256, 1024, 0.7, 40),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "pack", "attend", "attend", "pages"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op == "rotary":
        dim = rng.choice([64, 80, 128, 192, 256, 576])
        rot = rng.choice([32, 64, dim // 2 // 2 * 2]) if dim > 64 else rng.choice([32, 64])
        heads = rng.choice([1, 6, 16, 32, 64, 128])
        k_heads = rng.choice([0, 1, 8])
        T = max(1, min(_log(rng, 1, 16384), (20 << 20) // ((heads + k_heads) * dim)))
        c = _rotary("", T, heads, k_heads, dim, rot, rng.choice([0, dim - rot]),
                    rng.random() < 0.5, rng.choice(["none", "linear", "parts"]),
                    rng.choice(["bf16", "f16", "f32"]), rng.random() < 0.5,
                    _log(rng, 1024, 1 << 20))
    elif op == "pack":
        latent = rng.random() < 0.4
        n = _log(rng, 1, 64)
        long = rng.random() < 0.6
        heads, kd, vd = (1, 576, 512) if latent else (rng.choice([1, 2, 4, 8]),) + rng.choice(
            [(64, 64), (128, 128), (192, 128), (80, 80)])
        max_len = min(_log(rng, 1, 4096), 32768 // n) if long else 1
        to = "position" if max_len > 1 else "token"
        c = _pack("", n, max_len, max_len > 1 and rng.random() < 0.7, heads, kd, vd, latent,
                  rng.choice([1, 16, 64, 128]), "any" if rng.random() < 0.5 else "zero",
                  rng.choice([0, 32, 64]), to, dtype)
    elif op == "attend":
        latent = rng.random() < 0.5
        V = rng.choice([1, 1, 1, 2, 4])
        tokens = rng.choice([1, 1, 16])
        R = _log(rng, 1, 64)
        if latent:
            heads, kvh, kd, vd = rng.choice([8, 16, 64, 128]), 1, 576, 512
        else:
            kvh = rng.choice([1, 2, 4, 8])
            heads = kvh * rng.choice([1, 3, 4, 8, 16])
            kd, vd = rng.choice([(64, 64), (128, 128), (192, 128), (256, 256), (80, 80)])
        row = kvh * (kd + (0 if latent else vd))
        most = min(64 * 1984, (160 << 20) // row) // (R * V)
        n = max(1, min(_log(rng, 1, 8192), most) // tokens)
        B = 16 + V * n + rng.randrange(1, 512)
        c = _attend("", R, V, n, rng.choice([0, 0, n // 7]), heads, kvh, kd, vd, latent,
                    rng.choice([1, 16, 64]), tokens, B, rng.random() < 0.3,
                    (B + rng.randrange(1, 4096)) * 4 * tokens - rng.randrange(tokens), dtype)
    else:
        kind = rng.choice(["fork", "compact", "turnover"])
        R = _log(rng, 4, 256)
        blocks = _log(rng, 4, 256)
        live = rng.uniform(0.2, 0.85)
        pages = max(8, int(R * blocks * 0.6)) + rng.randrange(1, 64)
        rows = rng.choice([1, 16, 64])
        row = rng.choice([16, 576, 2048])
        layers = max(1, min(rng.choice([1, 2, 4, 8]), (900 << 20) // (pages * rows * row)))
        if pages * rows * row * layers > (1 << 30):
            rows, row = 16, 576
        c = _pages("", kind, pages, layers, rows, row, R, blocks, round(live, 3),
                   max(1, R // rng.choice([3, 4, 8])))
    del c["name"]
    return c


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _frequencies(rot, scaling, ctx):
    """Radians per position of each pair, base 10000.  "linear": positions interpolated by 4.
    "parts": pairs that turn often over the trained 4096 positions keep their frequency, those that
    turn less than once are interpolated by 32, a ramp between; the amplitude grows with it."""
    f = [10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        return [x / 4.0 for x in f], 1.0
    if scaling == "parts":
        turns = [4096 * x / (2 * math.pi) for x in f]
        keep = [min(1.0, max(0.0, (t - 1.0) / (32.0 - 1.0))) for t in turns]
        return [x * g + x / 32.0 * (1 - g) for x, g in zip(f, keep)], 0.1 * math.log(32.0) + 1.0
    return f, 1.0


def _turns(freqs):
    """Turns per position as 64-bit fractions (int64 that wraps): p * turns is the phase mod 1."""
    raw = [int(round(f / (2 * math.pi) * 2.0 ** 64)) & (2 ** 64 - 1) for f in freqs]
    return torch.tensor([x - 2 ** 64 if x >= 2 ** 63 else x for x in raw], dtype=torch.int64,
                        device="cuda")


def _prepare_rotary(c, g):
    dt = DT[c["dtype"]]
    f, amp = _frequencies(c["rot"], c["scaling"], c["ctx"])
    s = dict(q=torch.randn(c["T"], c["heads"], c["dim"], device="cuda", generator=g).to(dt),
             pos=torch.randint(0, c["ctx"], (c["T"],), device="cuda", generator=g).to(torch.int32),
             turns=_turns(f), amp=amp, k=None)
    if c["k_heads"]:
        s["k"] = torch.randn(c["T"], c["k_heads"], c["dim"], device="cuda", generator=g).to(dt)
    # where a part of each head is rotated the rest of the output is there before
    s["q_out"] = s["q"].clone()
    s["k_out"] = s["k"].clone() if s["k"] is not None else None
    return s


def _prepare_pack(c, g):
    dt = DT[c["dtype"]]
    n, m, S = c["n"], c["max_len"], c["block"]
    lens = torch.full((n,), m, dtype=torch.int64, device="cuda")
    if c["ragged"]:
        lens = torch.randint(m // 2, m + 1, (n,), device="cuda", generator=g)
        lens[0] = m
    cu = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    cu[1:] = torch.cumsum(lens, 0)
    T = int(cu[-1])
    start = torch.zeros(n, dtype=torch.int32, device="cuda")
    if c["start"] == "any":
        start = torch.randint(0, 4 * S + 1, (n,), device="cuda", generator=g).to(torch.int32)
    P = 4 * S + m + 1
    nblk = -(-P // S)
    cols = c["kv_heads"] * (1 if c["latent"] else 2)
    # the spread between tokens and heads that caches show
    k = torch.randn(T, c["kv_heads"], c["k_dim"], device="cuda", generator=g)
    k *= torch.exp(torch.randn(T, c["kv_heads"], 1, device="cuda", generator=g) * 0.5)
    s = dict(k=k.to(dt), v=None, start=start, cu=cu, nblk=nblk, P=P, turns=None, amp=1.0,
             reqs=torch.randperm(n, device="cuda", generator=g).to(torch.int32),
             scales=(0.5 + torch.rand(n, nblk, cols, device="cuda", generator=g)) * 0.006)
    if not c["latent"]:
        v = torch.randn(T, c["kv_heads"], c["v_dim"], device="cuda", generator=g)
        s["v"] = (v * torch.exp(torch.randn(T, 1, 1, device="cuda", generator=g) * 0.5)).to(dt)
    if c["rot"]:
        s["turns"] = _turns(_frequencies(c["rot"], "none", P)[0])
    rec = c["kv_heads"] * (c["k_dim"] + (0 if c["latent"] else c["v_dim"]))
    s["dst"] = torch.zeros((T, rec) if c["to"] == "token" else (n, P, rec), dtype=torch.uint8,
                           device="cuda")
    return s


def _e4m3(shape, g):
    """Random e4m3 values as packing leaves them: normal, their block's largest near 448 / 2."""
    return (torch.randn(shape, device="cuda", generator=g) * 60.0).clamp_(-TOP, TOP).to(E4M3)


def _prepare_attend(c, g):
    R, V, n, tok, B = c["R"], c["V"], c["n"], c["tokens"], c["B"]
    row = c["kv_heads"] * (c["k_dim"] + (0 if c["latent"] else c["v_dim"]))
    k = V * n
    places = -(-c["ctx"] // tok)                       # records of the context
    # distinct positions (or pages), the last one among them
    sel = torch.randint(0, max(1, places // k), (R, k), device="cuda", generator=g)
    sel += torch.arange(k, device="cuda") * (places // k)
    sel[:, k - 1] = places - 1
    sel = sel.gather(1, torch.rand(R, k, device="cuda", generator=g).argsort(1)).to(torch.int32)
    slots = torch.rand(R, B, device="cuda", generator=g).argsort(1)[:, :k].to(torch.int32)
    hot = _e4m3((R, B + 1, tok * row), g).view(torch.uint8)
    resident = None
    if c["resident"]:
        resident = _e4m3((R * k // 2 + 1, tok * row), g).view(torch.uint8)
        alt = torch.arange(R * k, device="cuda").view(R, k)
        slots = torch.where(alt % 2 == 1, B + 1 + alt // 2, slots).to(torch.int32)
    if c["pad"]:
        sel.view(R, V, n)[:, :, n - c["pad"]:] = -1
        slots.view(R, V, n)[:, :, n - c["pad"]:] = -1
    nblk = -(-places * tok // c["block"])
    cols = c["kv_heads"] * (1 if c["latent"] else 2)
    return dict(
        q=(torch.randn(R, V, c["heads"], c["k_dim"], device="cuda", generator=g) * 2).to(
            DT[c["dtype"]]),
        sel=sel, slots=slots, hot=hot, resident=resident,
        scales=(0.5 + torch.rand(R, nblk, cols, device="cuda", generator=g)) / 60.0,
        lens=torch.full((R,), c["ctx"], dtype=torch.int32, device="cuda"),
        scale=c["k_dim"] ** -0.5,
        out=torch.empty(R, V, c["heads"], c["v_dim"], dtype=DT[c["dtype"]], device="cuda"),
        lse=torch.empty(R, V, c["heads"], device="cuda"))


def _prepare_pages(c, g):
    """Requests with tables of shared and private pages, scattered over the store; the forks' and
    the newcomers' requests are empty."""
    N, R, M, n = c["pages"], c["R"], c["blocks"], c["n"]
    empty = n if c["op"] != "compact" else 0
    used = R - empty
    lens = torch.randint(1, M + 1, (R,), device="cuda", generator=g)
    budget = min(int(N * c["live"]), N - n - 1)
    col = torch.arange(M, device="cuda")
    held = (col[None] < lens[:, None]) & (torch.arange(R, device="cuda")[:, None] < used)
    order = torch.cumsum(held.view(-1).to(torch.int64), 0).view(R, M) - 1
    held &= order < budget
    pages = torch.randperm(N, device="cuda", generator=g)
    tables = torch.where(held, pages[order.clamp(0, N - 1)], -1)
    # every fourth request shares the first half of its neighbour's pages
    share = (torch.arange(R, device="cuda") % 4 == 3)[:, None] & held & (col[None] < M // 2)
    tables = torch.where(share & (tables.roll(1, 0) >= 0), tables.roll(1, 0), tables)
    refs = torch.bincount(tables[tables >= 0].view(-1), minlength=N)
    meta0 = torch.cat([refs, tables.view(-1)]).to(torch.int32)
    meta = meta0.clone()
    s = dict(meta0=meta0, meta=meta, refs=meta[:N], tables=meta[N:].view(R, M),
             store=torch.randint(-2 ** 31, 2 ** 31 - 1, (c["layers"], N, c["rows"] * c["row"] // 4),
                                 device="cuda", generator=g, dtype=torch.int32))
    if c["op"] == "fork":
        s["src"] = torch.randint(0, max(1, used), (n,), device="cuda", generator=g).to(torch.int32)
        s["dst"] = (used + torch.randperm(n, device="cuda", generator=g)).to(torch.int32)
        held_tokens = (tables >= 0).sum(1)[s["src"].long()] * c["rows"]
        s["tokens"] = (held_tokens - torch.randint(0, c["rows"], (n,), device="cuda", generator=g)
                       ).clamp_(min=0).to(torch.int32)
    if c["op"] == "turnover":
        s["out"] = torch.randperm(max(1, used), device="cuda", generator=g)[:n].to(torch.int32)
        s["into"] = (used + torch.randperm(n, device="cuda", generator=g)).to(torch.int32)
        s["want"] = torch.randint(1, M + 1, (n,), device="cuda", generator=g).to(torch.int32)
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    make = {"rotary": _prepare_rotary, "pack": _prepare_pack, "attend": _prepare_attend}
    return dict(make.get(case["op"], _prepare_pages)(case, g), case=case)


# ---------------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------------
def _rotated(x, pos, turns, offset, rot, interleaved, amp):
    """x [T][H][D] in 32 bits with its pairs turned by pos * turns."""
    ph = (pos.to(torch.int64)[:, None] * turns[None]).to(torch.float32) * (2 * math.pi / 2.0 ** 64)
    cos, sin = torch.cos(ph)[:, None] * amp, torch.sin(ph)[:, None] * amp
    y = x.to(torch.float32).clone()
    if interleaved:
        a, b = y[..., offset:offset + rot:2], y[..., offset + 1:offset + rot:2]
    else:
        a, b = y[..., offset:offset + rot // 2], y[..., offset + rot // 2:offset + rot]
    na, nb = a * cos - b * sin, a * sin + b * cos
    a.copy_(na)
    b.copy_(nb)
    return y


def _sides(c, s):
    """(input, output) of q and of k: whole heads, or the rotated part of each."""
    cut = slice(c["offset"], c["offset"] + c["rot"]) if c["part"] else slice(None)
    both = [(s["q"][..., cut], s["q_out"][..., cut])]
    if s["k"] is not None:
        both.append((s["k"][..., cut], s["k_out"][..., cut]))
    return both, 0 if c["part"] else c["offset"]


def _run_rotary(c, s):
    both, offset = _sides(c, s)
    args = (s["pos"], s["turns"], offset, c["rot"], c["interleaved"], s["amp"])
    [y.copy_(_rotated(x, *args)) for x, y in both]
    return {"q": s["q_out"], "k": s["k_out"]}


def _run_pack(c, s):
    S, n, H = c["block"], c["n"], c["kv_heads"]
    T = s["k"].shape[0]
    tok = torch.arange(T, device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["cu"][1:], tok, right=True)
    pos = (s["start"][seq] + tok - s["cu"][seq]).to(torch.int64)
    req = s["reqs"][seq].to(torch.int64)
    k = s["k"].to(torch.float32)
    if c["rot"]:
        k = _rotated(s["k"], pos, s["turns"], c["k_dim"] - c["rot"], c["rot"], False, 1.0)
    amax = k.abs().amax(-1)
    if s["v"] is not None:
        v = s["v"].to(torch.float32)
        amax = torch.cat([amax, v.abs().amax(-1)], 1)
    blk = req * s["nblk"] + pos // S
    cells = s["scales"].view(-1, amax.shape[1])
    top = torch.zeros_like(cells).scatter_reduce_(0, blk[:, None].expand_as(amax), amax, "amax")
    first = torch.zeros(cells.shape[0], device="cuda").index_add_(0, blk, (pos % S == 0).float())
    last = torch.zeros(cells.shape[0], device="cuda").index_add_(0, blk, (pos % S == S - 1).float())
    fresh = ((first > 0)[:, None] | (cells == 0)) & (top > 0)
    room = torch.where(last > 0, 1.0, 2.0)[:, None]
    cells.copy_(torch.where(fresh, top * (room / TOP), cells))
    inv = torch.where(cells > 0, 1 / cells, 0.0)[blk]
    parts = [(k * inv[:, :H, None]).view(T, -1)]
    if s["v"] is not None:
        parts.append((v * inv[:, H:, None]).view(T, -1))
    rows = torch.cat(parts, 1).clamp_(-TOP, TOP).to(E4M3).view(torch.uint8)
    if c["to"] == "token":
        s["dst"].copy_(rows)
    else:
        s["dst"].view(-1, rows.shape[1])[req * s["P"] + pos] = rows
    return {"rows": s["dst"].view(E4M3), "scales": s["scales"]}


def _run_attend(c, s):
    R, V, n, tok, H, KH = c["R"], c["V"], c["n"], c["tokens"], c["heads"], c["kv_heads"]
    Dk, Dv, B = c["k_dim"], c["v_dim"], c["B"]
    slot = s["slots"].to(torch.int64)
    rows = s["hot"].gather(1, slot.clamp(0, B)[:, :, None].expand(-1, -1, s["hot"].shape[2]))
    if s["resident"] is not None:
        far = s["resident"][(slot - B - 1).clamp(min=0)]
        rows = torch.where((slot > B)[:, :, None], far, rows)
    x = rows.view(E4M3).to(torch.float32).view(R, V, n * tok, -1)
    pos = s["sel"].to(torch.int64)[:, :, None] * tok + torch.arange(tok, device="cuda")
    ok = ((slot >= 0)[:, :, None] & (pos < s["lens"][:, None, None])).view(R, V, 1, 1, n * tok)
    blk = (pos.clamp(min=0) // c["block"]).view(R, -1)
    sc = s["scales"].gather(1, blk[:, :, None].expand(-1, -1, s["scales"].shape[2]))
    sc = sc.view(R, V, n * tok, -1)
    kk = (x[..., :KH * Dk].view(R, V, n * tok, KH, Dk) * sc[..., :KH, None]).permute(0, 1, 3, 2, 4)
    if c["latent"]:
        vv = kk[..., :Dv]
    else:
        vv = (x[..., KH * Dk:].view(R, V, n * tok, KH, Dv) * sc[..., KH:, None]).permute(
            0, 1, 3, 2, 4)
    q = s["q"].to(torch.float32).view(R, V, KH, H // KH, Dk)
    a = torch.matmul(q, kk.transpose(-1, -2)) * s["scale"]
    a = torch.where(ok, a, -math.inf)
    m = a.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, 0.0)
    p = torch.exp(a - m)
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p, vv) / torch.where(z > 0, z, 1.0)
    s["out"].copy_(o.view(R, V, H, Dv))
    s["lse"].copy_((torch.log(z) + m).view(R, V, H))
    return {"out": s["out"], "lse": s["lse"]}


def _run_fork(c, s):
    rows, N, M = c["rows"], c["pages"], c["blocks"]
    tables, refs, store = s["tables"], s["refs"], s["store"]
    src, dst = s["src"].long(), s["dst"].long()
    full, part = s["tokens"].long() // rows, s["tokens"].long() % rows
    have = tables[src]
    shared = torch.where(torch.arange(M, device="cuda")[None] < full[:, None], have, -1)
    refs.index_add_(0, shared.clamp(min=0).view(-1), (shared >= 0).view(-1).to(torch.int32))
    at = full.clamp(max=M - 1)[:, None]
    last = have.gather(1, at)[:, 0].long()
    need = (part > 0) & (last >= 0)
    # the lowest free pages, in the list's order
    free = torch.nonzero(refs == 0)[:, 0]
    free = free[(torch.cumsum(need.long(), 0) - 1).clamp(min=0)]
    page = torch.where(need, free, -1)
    tables[dst] = torch.where((torch.arange(M, device="cuda")[None] == at) & need[:, None],
                              page[:, None].to(torch.int32), shared)
    refs.index_add_(0, page.clamp(min=0), need.to(torch.int32))
    use = torch.arange(store.shape[2], device="cuda")[None] < (part * (c["row"] // 4))[:, None]
    new = torch.where(use[None], store[:, last.clamp(min=0)], store[:, page.clamp(min=0)])
    store[:, page[need]] = new[:, need]


def _run_compact(c, s):
    tables, refs, store = s["tables"], s["refs"], s["store"]
    live = refs > 0
    ids = torch.arange(c["pages"], device="cuda")
    low = ids < live.sum()
    src, dst = torch.nonzero(live & ~low)[:, 0], torch.nonzero(~live & low)[:, 0]
    to = ids.to(torch.int32)
    to[src] = dst.to(torch.int32)
    tables.copy_(torch.where(tables >= 0, to[tables.clamp(min=0).long()], -1))
    refs[dst] = refs[src]
    refs[src] = 0
    store[:, dst] = store[:, src]


def _run_turnover(c, s):
    tables, refs, M = s["tables"], s["refs"], c["blocks"]
    out, into = s["out"].long(), s["into"].long()
    gone = tables[out]
    refs.index_add_(0, gone.clamp(min=0).view(-1), -(gone >= 0).view(-1).to(torch.int32))
    tables[out] = -1
    # in the list's order each newcomer takes the lowest free pages; one that finds too few, none
    have = tables[into]
    need = (have < 0) & (torch.arange(M, device="cuda")[None] < s["want"].long()[:, None])
    free = torch.nonzero(refs == 0)[:, 0]
    fits = torch.cumsum(need.sum(1), 0) <= free.shape[0]
    need &= fits[:, None]
    rank = (torch.cumsum(need.view(-1).long(), 0) - 1).clamp(0, max(0, free.shape[0] - 1))
    page = free[rank].view(need.shape)
    tables[into] = torch.where(need, page.to(torch.int32), have)
    refs.index_add_(0, torch.where(need, page, 0).view(-1), need.view(-1).to(torch.int32))


# ---------------------------------------------------------------------------------------------
# the package's operators
# ---------------------------------------------------------------------------------------------
def _own_rotary(c, s):
    from host_offload_serving_gb300 import cache8
    both, offset = _sides(c, s)
    k, k_out = both[1] if len(both) > 1 else (None, None)
    cache8.rotate(both[0][0], s["pos"], s["turns"], k=k, offset=offset,
                  interleaved=c["interleaved"], amplitude=s["amp"], out=both[0][1], k_out=k_out)
    return {"q": s["q_out"], "k": s["k_out"]}


def _layout(c):
    from host_offload_serving_gb300 import cache8
    return cache8.Records(c["kv_heads"], c["k_dim"], c["v_dim"], c["block"], latent=c["latent"])


def _own_pack(c, s):
    from host_offload_serving_gb300 import cache8
    if "layout" not in s:
        s["layout"] = _layout(c)
    cache8.pack(s["layout"], s["k"], s["v"], s["dst"], s["scales"], s["start"], cu_lens=s["cu"],
                reqs=s["reqs"], max_len=c["max_len"], headroom=2.0, turns=s["turns"],
                rot_offset=c["k_dim"] - c["rot"])
    return {"rows": s["dst"].view(E4M3), "scales": s["scales"]}


def _own_attend(c, s):
    from host_offload_serving_gb300 import cache8
    if "layout" not in s:
        s["layout"] = _layout(c)
    cache8.attend(s["layout"], s["q"], s["sel"], s["slots"], s["hot"], s["scales"], s["out"],
                  softmax_scale=s["scale"], lse=s["lse"], record_tokens=c["tokens"],
                  seq_lens=s["lens"], resident=s["resident"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_pages(c, s):
    if "pool" not in s:
        from host_offload_serving_gb300 import pages
        s["pool"] = pages.PagePool(s["store"].view(torch.uint8), s["tables"], s["refs"],
                                   block_tokens=c["rows"])
    if c["op"] == "fork":
        s["pool"].fork(s["src"], s["dst"], s["tokens"])
    elif c["op"] == "compact":
        s["pool"].compact()
    else:
        s["pool"].free(s["out"])
        s["pool"].grow(s["into"], s["want"])


def run(state):
    c = state["case"]
    op = c["op"]
    if op in ("fork", "compact", "turnover"):
        # the tables and counts as they were: a pass changes them (and only fills pages that were
        # free, so the store needs no such copy)
        state["meta"].copy_(state["meta0"])
        if own:
            _own_pages(c, state)
        else:
            {"fork": _run_fork, "compact": _run_compact, "turnover": _run_turnover}[op](c, state)
        return {"tables": state["tables"], "refs": state["refs"], "store": state["store"]}
    if own:
        return {"rotary": _own_rotary, "pack": _own_pack, "attend": _own_attend}[op](c, state)
    return {"rotary": _run_rotary, "pack": _run_pack, "attend": _run_attend}[op](c, state)


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------
def work(c):
    size = 4 if c.get("dtype") == "f32" else 2
    if c["op"] == "rotary":
        part = c["rot"] if c["part"] else c["dim"]
        e = c["T"] * (c["heads"] + c["k_heads"])
        return {"bytes": e * part * size * 2 + 4 * c["T"] + 4 * c["rot"], "flops": e * c["rot"] * 3}
    if c["op"] == "pack":
        T = c["n"] * c["max_len"] * (0.75 if c["ragged"] else 1)
        vals = c["kv_heads"] * (c["k_dim"] + (0 if c["latent"] else c["v_dim"]))
        cells = T / min(c["block"], c["max_len"]) * c["kv_heads"] * (1 if c["latent"] else 2)
        return {"bytes": T * vals * (size + 1) + 4 * cells + 8 * c["n"], "flops": T * vals * 2}
    if c["op"] == "attend":
        n = c["R"] * c["V"] * (c["n"] - c["pad"])
        row = c["kv_heads"] * (c["k_dim"] + (0 if c["latent"] else c["v_dim"]))
        cols = c["kv_heads"] * (1 if c["latent"] else 2)
        q = c["R"] * c["V"] * c["heads"]
        cells = min(n * c["tokens"], c["R"] * -(-c["ctx"] // c["block"]))
        return {"bytes": n * c["tokens"] * row + q * (c["k_dim"] + c["v_dim"]) * size + 4 * q
                + c["R"] * c["V"] * c["n"] * 8 + cells * cols * 4,
                "flops": 2.0 * n * c["tokens"] * c["heads"] * (c["k_dim"] + c["v_dim"])}
    meta = 4 * (c["pages"] + c["R"] * c["blocks"])
    if c["op"] == "fork":
        # half a page in the mean, read and written; the parents' and the forks' table rows
        return {"bytes": c["n"] * c["layers"] * c["rows"] * c["row"] + 4 * c["pages"]
                + 8 * c["n"] * c["blocks"], "flops": 0}
    if c["op"] == "compact":
        # the live pages above the live count, in the mean, read and written
        live = min(c["live"], c["R"] * c["blocks"] / 2 / c["pages"]) * 0.9
        return {"bytes": 2.0 * c["pages"] * live * (1 - live) * c["layers"] * c["rows"] * c["row"]
                + 2 * meta, "flops": 0}
    return {"bytes": 4 * c["pages"] + 8 * c["n"] * c["blocks"], "flops": 0}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------
def _exact_turn(x, pos, freqs, offset, rot, interleaved, amp):
    """Each pair as a complex number times amp * e^(i * pos * f)."""
    ang = pos.double()[:, None] * torch.tensor(freqs, dtype=torch.float64, device="cuda")[None]
    w = torch.polar(torch.full_like(ang, amp), ang)[:, None]
    mid = x.double()[..., offset:offset + rot]
    if interleaved:
        z = torch.view_as_complex(mid.reshape(*mid.shape[:-1], rot // 2, 2).contiguous()) * w
        mid = torch.view_as_real(z).reshape(mid.shape)
    else:
        z = torch.complex(mid[..., :rot // 2], mid[..., rot // 2:]) * w
        mid = torch.cat([z.real, z.imag], -1)
    return torch.cat([x.double()[..., :offset], mid, x.double()[..., offset + rot:]], -1)


def exact(case, seed):
    c = case
    if c["op"] in ("fork", "compact", "turnover"):
        return None                                    # whole numbers only
    s = prepare(case, seed)
    if c["op"] == "rotary":
        f, amp = _frequencies(c["rot"], c["scaling"], c["ctx"])
        args = (s["pos"], f, c["offset"], c["rot"], c["interleaved"], amp)
        return {"q": _exact_turn(s["q"], *args),
                "k": None if s["k"] is None else _exact_turn(s["k"], *args)}
    if c["op"] == "pack":
        f = _frequencies(c["rot"], "none", 0)[0] if c["rot"] else []
        rows = torch.zeros(s["dst"].shape, dtype=torch.float64, device="cuda")
        scales = s["scales"].double()
        H, S = c["kv_heads"], c["block"]
        cu, start, reqs = s["cu"].tolist(), s["start"].tolist(), s["reqs"].tolist()
        for i, r in enumerate(reqs):
            lo, hi, p0 = cu[i], cu[i + 1], start[i]
            x = s["k"][lo:hi]
            pos = torch.arange(p0, p0 + hi - lo, device="cuda")
            x = _exact_turn(x, pos, f, c["k_dim"] - c["rot"], c["rot"], False, 1.0) if f else x.double()
            heads = [x[:, h] for h in range(H)]
            if s["v"] is not None:
                heads += [s["v"][lo:hi, h].double() for h in range(H)]
            for b in range(p0 // S, (p0 + hi - lo - 1) // S + 1):
                a, z = max(b * S, p0), min(b * S + S, p0 + hi - lo)
                if a == b * S:
                    grow = 1.0 if z == b * S + S else 2.0
                    tops = torch.stack([h[a - p0:z - p0].abs().max() for h in heads])
                    scales[r, b] = tops * grow / TOP
            per = scales[r][pos // S]
            row = torch.cat([h / per[:, j:j + 1] for j, h in enumerate(heads)], 1).clamp(-TOP, TOP)
            if c["to"] == "token":
                rows[lo:hi] = row
            else:
                rows[r, p0:p0 + hi - lo] = row
        return {"rows": rows, "scales": scales}
    R, V, n, tok, KH, Dk, Dv = (c[x] for x in ("R", "V", "n", "tokens", "kv_heads", "k_dim", "v_dim"))
    G = c["heads"] // KH
    out = torch.zeros(R, V, c["heads"], Dv, dtype=torch.float64, device="cuda")
    lse = torch.full((R, V, c["heads"]), -math.inf, dtype=torch.float64, device="cuda")
    row = KH * (Dk + (0 if c["latent"] else Dv))
    for r in range(R):
        both = s["hot"][r].view(E4M3).view(-1, tok, row)
        for v in range(V):
            slot = s["slots"][r, v * n:(v + 1) * n].long()
            sel = s["sel"][r, v * n:(v + 1) * n].long()
            slot, sel = slot[slot >= 0], sel[slot >= 0]
            x = torch.zeros(slot.numel(), tok, row, dtype=torch.float64, device="cuda")
            near = slot <= c["B"]
            x[near] = both[slot[near]].double()
            if s["resident"] is not None:
                x[~near] = s["resident"][slot[~near] - c["B"] - 1].view(E4M3).view(
                    -1, tok, row).double()
            pos = (sel[:, None] * tok + torch.arange(tok, device="cuda")).reshape(-1)
            x = x.view(-1, row)[pos < c["ctx"]]
            sc = s["scales"][r].double()[pos[pos < c["ctx"]] // c["block"]]
            for h in range(KH if x.shape[0] else 0):
                kh = x[:, h * Dk:(h + 1) * Dk] * sc[:, h, None]
                vh = kh[:, :Dv] if c["latent"] else (
                    x[:, KH * Dk + h * Dv:KH * Dk + (h + 1) * Dv] * sc[:, KH + h, None])
                a = s["q"][r, v, h * G:(h + 1) * G].double() @ kh.T * s["scale"]
                out[r, v, h * G:(h + 1) * G] = torch.softmax(a, -1) @ vh
                lse[r, v, h * G:(h + 1) * G] = torch.logsumexp(a, -1)
    return {"out": out, "lse": lse}
