"""The 8-bit record operators on the GPU against plain computations in 64 bits.

Tolerances follow from the formats: U is half a unit in the last place of the
output type; e4m3 rounds a value to 2^-4 of it (2^-10 below its normal
range); the probabilities and q enter as two (bf16) or three (f16) e4m3 terms, 2^-8 or
2^-12 of each; sums are in 32 bits.
"""
import numpy as np
import pytest
import torch

from host_offload_serving_gb300 import cache8, pages
from host_offload_serving_gb300 import hisparse as H

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
E4M3 = torch.float8_e4m3fn


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------------------------
# rotary
# ---------------------------------------------------------------------------------------------
def _rotated64(x, pos, freqs, offset, interleaved, amp, inverse=False):
    """x [T][H][D] in 64 bits; phases reduced by Python integers."""
    rot = 2 * len(freqs)
    y = x.double().cpu().numpy().copy()
    turns = [int(t) for t in freqs]
    ang = np.array([[((int(p) * t) % 2 ** 64) / 2.0 ** 64 * 2 * np.pi for t in turns]
                    for p in pos.tolist()])
    c, s = np.cos(ang)[:, None] * amp, np.sin(ang)[:, None] * amp * (-1 if inverse else 1)
    ia = offset + (2 * np.arange(rot // 2) if interleaved else np.arange(rot // 2))
    ib = ia + (1 if interleaved else rot // 2)
    a, b = y[..., ia].copy(), y[..., ib].copy()
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    norm = np.zeros_like(y)
    norm[..., ia] = norm[..., ib] = np.hypot(a, b) * amp
    return y, norm


def _rotary_close(got, want, norm, dtype):
    err = np.abs(got.double().cpu().numpy() - want)
    tol = U[dtype] * np.abs(want) + 1e-6 * norm * (norm > 0) + 2.0 ** -25 * (norm > 0)
    assert (err <= tol).all(), float((err - tol).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T,heads,k_heads,dim,rot,offset,interleaved", [
    (1, 1, 0, 64, 64, 0, False), (1, 128, 1, 576, 64, 512, False), (7, 3, 1, 80, 40, 40, False),
    (5, 2, 2, 96, 32, 8, True), (33, 6, 2, 128, 128, 0, True), (3, 2, 0, 10, 6, 1, False),
    (4, 5, 3, 9, 2, 7, True), (257, 4, 4, 64, 32, 32, False),
])
def test_rotary(T, heads, k_heads, dim, rot, offset, interleaved, dtype):
    g = _gen(T * 1000 + dim)
    turns, amp = cache8.rotary_turns(rot, scaling="parts", factor=4.0, original_len=64)
    q, k = _randn(g, T, heads, dim).to(dtype), None
    pos = torch.randint(0, 1 << 20, (T,), device="cuda", generator=g).to(torch.int32)
    pos[0] = 0
    if T > 2:
        pos[1], pos[2] = 2 ** 31 - 1, -5
    if k_heads:
        k = _randn(g, T, k_heads, dim).to(dtype)
    out = torch.full_like(q, float("nan"))
    k_out = torch.full_like(k, float("nan")) if k_heads else None
    cache8.rotate(q, pos, turns.cuda(), k=k, out=out, k_out=k_out, offset=offset,
                  interleaved=interleaved, amplitude=amp)
    for x, y in ((q, out), (k, k_out)):
        if x is None:
            continue
        want, norm = _rotated64(x, pos, turns, offset, interleaved, amp)
        _rotary_close(y, want, norm, dtype)
        # in place, the same bits
        z = x.clone()
        cache8.rotate(z, pos, turns.cuda(), offset=offset, interleaved=interleaved, amplitude=amp)
        assert torch.equal(z, y)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T,heads,k_heads,dim,rot,offset,interleaved", [
    (2501, 12, 3, 64, 64, 0, False), (1500, 33, 1, 128, 64, 32, True), (3, 1, 1, 8192, 8192, 0, False),
    (2, 1, 0, 8192, 8192, 0, True), (4099, 1, 0, 16, 8, 4, True), (700, 5, 5, 20, 12, 4, False),
])
def test_rotary_many_tokens(T, heads, k_heads, dim, rot, offset, interleaved, dtype):
    """Several tokens and CTAs for a thread's unit, and the widest rotated part."""
    test_rotary(T, heads, k_heads, dim, rot, offset, interleaved, dtype)


def test_rotary_strided_views_and_untouched_rest():
    """A part of wider heads, by views whose strides and alignment are odd."""
    g = _gen(5)
    wide = _randn(g, 9, 3, 131).to(torch.bfloat16)
    keep = wide.clone()
    turns, _ = cache8.rotary_turns(32)
    pos = torch.arange(9, device="cuda", dtype=torch.int32)
    for at in (3, 64):
        view = wide[:, :, at:at + 64]
        want, norm = _rotated64(view, pos, turns, 16, False, 1.0)
        cache8.rotate(view, pos, turns.cuda(), offset=16)
        _rotary_close(view, want, norm, torch.bfloat16)
        wide[:, :, at:at + 64] = keep[:, :, at:at + 64]
        assert torch.equal(wide, keep)


def test_rotary_inverse_is_the_gradient():
    """<rotate(x), y> has the gradient rotate(y, inverse) in x: against the
    formula, and against differences (the map is linear, so a difference is exact but for
    rounding in 32 bits)."""
    g = _gen(6)
    turns, _ = cache8.rotary_turns(16)
    t = turns.cuda()
    pos = torch.tensor([3, 70000], dtype=torch.int32, device="cuda")
    x, y = _randn(g, 2, 3, 24), _randn(g, 2, 3, 24)
    kw = dict(offset=4, interleaved=True, amplitude=1.25)
    grad = cache8.rotate(y, pos, t, out=torch.empty_like(y), inverse=True, **kw)[0]
    want, norm = _rotated64(y, pos, turns, 4, True, 1.25, inverse=True)
    _rotary_close(grad, want, norm, torch.float32)
    f = lambda v: float((cache8.rotate(v, pos, t, out=torch.empty_like(v), **kw)[0].double() * y.double()).sum())
    for at in ((0, 0, 4), (0, 2, 5), (1, 1, 12), (1, 0, 19), (1, 2, 2)):
        hi, lo = x.clone(), x.clone()
        hi[at] += 1.0
        lo[at] -= 1.0
        num = (f(hi) - f(lo)) / float(hi[at] - lo[at])
        assert abs(num - float(grad[at])) < 1e-4 * (1 + abs(num)) * float(y.abs().max())


def test_rotary_empty_and_many_heads():
    turns = cache8.rotary_turns(32)[0].cuda()
    x = torch.zeros(0, 4, 64, device="cuda")
    cache8.rotate(x, torch.zeros(0, dtype=torch.int32, device="cuda"), turns)
    g = _gen(8)
    q = _randn(g, 2, 700, 64)
    pos = torch.tensor([11, 131071], dtype=torch.int32, device="cuda")
    want, norm = _rotated64(q, pos, turns.cpu(), 0, False, 1.0)
    _rotary_close(cache8.rotate(q, pos, turns)[0], want, norm, torch.float32)


# ---------------------------------------------------------------------------------------------
# pack
# ---------------------------------------------------------------------------------------------
def _pack64(rec, k, v, scales, start, cu, reqs, headroom, turns, rot_offset, interleaved=False):
    """(values [tokens][columns] list per token of x / scale, scales) in 64 bits."""
    S, K = rec.block_tokens, rec.kv_heads
    scales = scales.double().cpu().numpy().copy()
    kk = k.double().cpu().numpy()
    vals = [None] * k.shape[0]
    for i, p0 in enumerate(start):
        lo, hi = cu[i], cu[i + 1]
        if hi == lo:
            continue
        x = kk[lo:hi]
        if turns is not None:
            x, _ = _rotated64(k[lo:hi], torch.arange(p0, p0 + hi - lo), turns, rot_offset,
                              interleaved, 1.0)
        heads = [x[:, h] for h in range(K)]
        if v is not None:
            heads += [v[lo:hi, h].double().cpu().numpy() for h in range(K)]
        pos = np.arange(p0, p0 + hi - lo)
        r = reqs[i]
        for b in range(p0 // S, (p0 + hi - lo - 1) // S + 1):
            m = pos // S == b
            for c, h in enumerate(heads):
                if (pos[m][0] == b * S) or scales[r, b, c] == 0:
                    a = np.abs(h[m])
                    a = a[np.isfinite(a)]
                    top = a.max() if a.size else 0.0
                    if top > 0:
                        scales[r, b, c] = top / 448 * (1 if pos[m][-1] == b * S + S - 1 else headroom)
        for t in range(hi - lo):
            row = []
            for c, h in enumerate(heads):
                s = scales[r, pos[t] // S, c]
                row.append(h[t] / s if s > 0 else h[t] * 0)
            vals[lo + t] = np.concatenate(row)
    return vals, scales


def _pack_close(rows, vals):
    """rows uint8 [n][row] against the values they round."""
    got = rows.view(E4M3).double().cpu().numpy()
    want = np.stack(vals)
    nan = np.isnan(want)
    assert (np.isnan(got) == nan).all()
    want = np.clip(np.where(nan, 0, want), -448, 448)
    tol = np.maximum(np.abs(want) * 2.0 ** -4, 2.0 ** -10) * (1 + 1e-4)
    err = np.abs(np.where(nan, 0, got) - want)
    assert (err <= tol).all(), float((err / tol).max())


PACK_RECORDS = [cache8.Records(1, 576, 512, 64, latent=True), cache8.Records(8, 128, 128, 64),
                cache8.Records(2, 80, 48, 16), cache8.Records(3, 16, 32, 1), cache8.Records(1, 64, 64, 300)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rec", PACK_RECORDS, ids=["latent", "heads", "odd", "one", "long"])
@pytest.mark.parametrize("rot", [0, 16])
def test_pack_by_position(rec, dtype, rot):
    """Ragged sequences, empty ones and ones that begin inside a block; open
    blocks keep their scale, unset ones get one."""
    g = _gen(rec.k_dim + rot)
    S = rec.block_tokens
    lens, start = [1, 2 * S + 5, 0, S, 97], [0, 3, 1, S - 1, 2 * S]
    reqs = [2, 0, 1, 4, 3]
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    k = (_randn(g, cu[-1], rec.kv_heads, rec.k_dim) * 3).to(dtype)
    v = None if rec.latent else _randn(g, cu[-1], rec.kv_heads, rec.v_dim).to(dtype)
    P = 4 * S + 100
    scales = torch.zeros(5, rec.blocks(P), rec.columns, device="cuda")
    scales[0, 0] = 0.004                       # an open block of request 0
    scales[4] = 0.01
    turns = cache8.rotary_turns(rot)[0] if rot else None
    want, want_s = _pack64(rec, k, v, scales, start, cu, reqs, 1.5, turns, rec.k_dim - rot)
    dst = torch.full((5, P, rec.row_bytes), 0x55, dtype=torch.uint8, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    st = _status()
    cache8.pack(rec, k, v, dst, scales, i32(start), cu_lens=i32(cu), reqs=i32(reqs), max_len=max(lens),
                headroom=1.5, turns=turns.cuda() if rot else None, rot_offset=rec.k_dim - rot, status=st)
    assert int(st) == 0
    np.testing.assert_allclose(scales.double().cpu().numpy(), want_s, rtol=4e-6)
    rows, seen = [], torch.zeros(5, P, dtype=torch.bool)
    for i, r in enumerate(reqs):
        rows.append(dst[r, start[i]:start[i] + lens[i]])
        seen[r, start[i]:start[i] + lens[i]] = True
    _pack_close(torch.cat(rows), want)
    assert (dst.cpu()[~seen] == 0x55).all()


@pytest.mark.parametrize("rec,lens,rot,offset,interleaved,dtype", [
    (cache8.Records(8, 64, 64, 1), [600, 3, 450, 599], 64, 0, True, torch.bfloat16),    # blocks of a token
    (cache8.Records(4, 128, 128, 16), [900, 701, 17, 640], 32, 8, False, torch.float16),
    (cache8.Records(5, 48, 80, 16), [333, 800], 16, 16, True, torch.float32),           # 5 heads, odd sizes
    (cache8.Records(2, 192, 128, 64), [400, 33, 64, 1], 64, 128, False, torch.bfloat16),
    (cache8.Records(1, 640, 512, 64, latent=True), [70, 131], 640, 0, False, torch.bfloat16),
    (cache8.Records(1, 640, 512, 128, latent=True), [129, 300], 320, 160, True, torch.float32),
    (cache8.Records(1, 16, 16, 4096), [5003, 4100], 16, 0, False, torch.bfloat16),      # blocks walked in parts
    (cache8.Records(3, 512, 16, 200), [900], 128, 256, True, torch.float16),
    (cache8.Records(17, 32, 16, 8), [90, 1, 64], 32, 0, False, torch.bfloat16),
])
def test_pack_blocks_and_heads_of_every_size(rec, lens, rot, offset, interleaved, dtype):
    """Blocks of one token to thousands, one head to many, the rotated part anywhere in the head."""
    g = _gen(sum(lens) + rot)
    n = len(lens)
    start = [(7 * i + 5) % (2 * rec.block_tokens) for i in range(n)]
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    k = (_randn(g, cu[-1], rec.kv_heads, rec.k_dim) * 2).to(dtype)
    v = None if rec.latent else _randn(g, cu[-1], rec.kv_heads, rec.v_dim).to(dtype)
    P = max(s + l for s, l in zip(start, lens))
    scales = torch.zeros(n, rec.blocks(P), rec.columns, device="cuda")
    turns = cache8.rotary_turns(rot)[0]
    want, want_s = _pack64(rec, k, v, scales, start, cu, list(range(n)), 2.0, turns, offset, interleaved)
    dst = torch.zeros(n, P, rec.row_bytes, dtype=torch.uint8, device="cuda")
    st = _status()
    cache8.pack(rec, k, v, dst, scales, torch.tensor(start, dtype=torch.int32, device="cuda"),
                cu_lens=torch.tensor(cu, dtype=torch.int32, device="cuda"), max_len=max(lens), turns=turns.cuda(),
                rot_offset=offset, interleaved=interleaved, status=st)
    assert int(st) == 0
    np.testing.assert_allclose(scales.double().cpu().numpy(), want_s, rtol=4e-6)
    _pack_close(torch.cat([dst[i, start[i]:start[i] + lens[i]] for i in range(n)]), want)


@pytest.mark.parametrize("rec", PACK_RECORDS[:3], ids=["latent", "heads", "odd"])
def test_pack_decode_steps(rec):
    """One token a step through a whole block: the first fixes the scale with
    its headroom, later ones keep it and saturate; a zero token sets none."""
    g = _gen(3)
    S, n = rec.block_tokens, 3
    scales = torch.zeros(n, 2, rec.columns, device="cuda")
    hist = []
    for step in range(S + 2):
        k = _randn(g, n, rec.kv_heads, rec.k_dim).to(torch.bfloat16)
        v = None if rec.latent else _randn(g, n, rec.kv_heads, rec.v_dim).to(torch.bfloat16)
        if step == 0:
            k[1] = 0
        if step == 5:
            k[2] *= 1000
        start = torch.full((n,), step, dtype=torch.int32, device="cuda")
        want, want_s = _pack64(rec, k, v, scales, [step] * n, list(range(n + 1)), list(range(n)), 2.0, None, 0)
        rows = torch.empty(n, rec.row_bytes, dtype=torch.uint8, device="cuda")
        cache8.pack(rec, k, v, rows, scales, start)
        np.testing.assert_allclose(scales.double().cpu().numpy(), want_s, rtol=4e-6)
        _pack_close(rows, want)
        hist.append(scales[:, 0].clone())
    assert float(hist[0][1, 0]) == 0.0 and float(hist[1][1, 0]) > 0.0
    assert torch.equal(hist[1], hist[S - 1])


def test_pack_pages_errors_and_specials():
    """Paged rows; tokens without a page, pages outside the store, positions
    outside the table; infinities and NaN."""
    rec = cache8.Records(1, 32, 16, 4)
    g = _gen(9)
    k, v = _randn(g, 12, 1, 32), _randn(g, 12, 1, 16)
    k[2, 0, 3] = float("inf")
    k[3, 0, 5] = float("-inf")
    k[5, 0, 7] = float("nan")
    scales = torch.zeros(2, 3, 2, device="cuda")
    table = torch.tensor([[2, -1, 0, 7], [1, 1, 1, 1]], dtype=torch.int32, device="cuda")
    store = torch.full((9, 48), 0x11, dtype=torch.uint8, device="cuda")    # 3 pages of 3 rows
    start = torch.zeros(1, dtype=torch.int32, device="cuda")
    st = _status()
    want, want_s = _pack64(rec, k, v, scales, [0], [0, 12], [0], 2.0, None, 0)
    cache8.pack(rec, k, v, store, scales, start, max_len=12, blocks=table, page_tokens=3, status=st)
    assert int(st) == H.ERR_RANGE                                          # page 7 of 3
    np.testing.assert_allclose(scales[0].double().cpu().numpy(), want_s[0], rtol=4e-6)
    assert bool((scales[1] == 0).all())
    _pack_close(store[6:9], want[0:3])
    _pack_close(store[0:3], want[6:9])
    assert bool((store[3:6] == 0x11).all())
    for bad in (dict(start=torch.tensor([-1], dtype=torch.int32, device="cuda")),
                dict(start=torch.tensor([8], dtype=torch.int32, device="cuda")),       # past the scales
                dict(reqs=torch.tensor([2], dtype=torch.int32, device="cuda"))):
        st = _status()
        rows = torch.full((4, 48), 0x22, dtype=torch.uint8, device="cuda")
        kw = dict(dict(start=start), **bad)
        n = 4
        cache8.pack(rec, k[:n], v[:n], rows, scales[:, :2], kw.pop("start"), max_len=n, status=st, **kw)
        assert int(st) == H.ERR_RANGE
        assert bool((rows == 0x22).all())


# ---------------------------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------------------------
def _attend64(rec, q, sel, slots, hot, scales, softmax_scale, tok=1, sel_block=1, seq_lens=None,
              resident=None):
    """(out, lse, sum of p|v|, bound on a score's error) in 64 bits."""
    R, V, Hq, Dk = q.shape
    B, K, Dv = hot.shape[1] - 1, rec.kv_heads, rec.v_dim
    n = slots.shape[1] // V
    sel, slots = sel.cpu().numpy().astype(np.int64), slots.cpu().numpy().astype(np.int64)
    sc = scales.double().cpu().numpy()
    out = np.zeros((R, V, Hq, Dv))
    lse = np.full((R, V, Hq), -np.inf)
    mass, ds = np.zeros_like(out), np.zeros_like(lse)
    qs = q.double().cpu().numpy()
    val = lambda t: t.view(E4M3).double().cpu().numpy()
    for r in range(R):
        for v in range(V):
            rows, pos = [], []
            for j in range(v * n, (v + 1) * n):
                s = slots[r, j]
                if s < 0 or n == 0:
                    continue
                p = sel[r, j] if sel_block == 1 else sel[r, j // sel_block] * sel_block + j % sel_block
                rec_row = hot[r, s] if s <= B else resident[s - B - 1]
                for u in range(tok):
                    if seq_lens is not None and p * tok + u >= int(seq_lens[r]):
                        continue
                    rows.append(rec_row[u * rec.row_bytes:(u + 1) * rec.row_bytes])
                    pos.append(p * tok + u)
            if not rows:
                continue
            x = val(torch.stack(rows))
            s8 = sc[r, np.array(pos) // rec.block_tokens]
            for h in range(Hq):
                g = h // (Hq // K)
                kh = x[:, g * Dk:(g + 1) * Dk] * s8[:, g:g + 1]
                vh = kh[:, :Dv] if rec.latent else \
                    x[:, K * Dk + g * Dv:K * Dk + (g + 1) * Dv] * s8[:, K + g:K + g + 1]
                a = kh @ qs[r, v, h] * softmax_scale
                m = a.max()
                p = np.exp(a - m)
                z = p.sum()
                out[r, v, h], lse[r, v, h] = p @ vh / z, m + np.log(z)
                mass[r, v, h] = p @ np.abs(vh) / z
                ds[r, v, h] = 2.0 ** -16 * abs(softmax_scale) * np.abs(qs[r, v, h]).max() * np.abs(kh).sum(1).max()
    return out, lse, mass, ds


def _attend_close(out, lse, want, dtype):
    o, l, mass, ds = want
    terms = 2.0 ** -8 if dtype is torch.bfloat16 else 2.0 ** -12
    got = out.double().cpu().numpy()
    tol = U[dtype] * np.abs(o) + (terms + 2 * ds[..., None] + 1e-5) * mass + 2.0 ** -24
    assert np.isfinite(got).all()
    assert (np.abs(got - o) <= tol).all(), float((np.abs(got - o) / tol).max())
    if lse is not None:
        g = lse.double().cpu().numpy()
        assert (np.isneginf(g) == np.isneginf(l)).all()
        f = np.isfinite(l)
        assert (np.abs(g[f] - l[f]) <= ds[f] + 1e-5 * np.abs(l[f]) + 1e-5).all()


def _attend_case(rec, heads, dtype, R, V, n, tok=1, B=None, seed=0, q_std=1.0, pad=0.1):
    g = _gen(seed + n)
    B = B or V * n + 5
    hot = (_randn(g, R, B + 1, tok * rec.row_bytes) * 60).clamp(-448, 448).to(E4M3).view(torch.uint8)
    places = V * n * 3 + 1
    sel = torch.stack([torch.randperm(places, device="cuda", generator=g)[:V * n] for _ in range(R)])
    slots = torch.stack([torch.randperm(B + 1, device="cuda", generator=g)[:V * n] for _ in range(R)])
    drop = torch.rand(R, V * n, device="cuda", generator=g) < pad
    sel, slots = sel.masked_fill(drop, -1).int(), slots.masked_fill(drop, -1).int()
    scales = (0.2 + torch.rand(R, rec.blocks(places * tok), rec.columns, device="cuda", generator=g)) / 60
    q = (_randn(g, R, V, heads, rec.k_dim) * q_std).to(dtype)
    out = torch.full((R, V, heads, rec.v_dim), float("nan"), dtype=dtype, device="cuda")
    lse = torch.full((R, V, heads), float("nan"), device="cuda")
    return dict(rec=rec, q=q, sel=sel, slots=slots, hot=hot, scales=scales, out=out, lse=lse)


def _attend(c, **kw):
    scale = c["rec"].k_dim ** -0.5
    st = _status()
    cache8.attend(c["rec"], c["q"], c["sel"], c["slots"], c["hot"], c["scales"], c["out"], lse=c["lse"],
                  softmax_scale=scale, status=st, **kw)
    return int(st)


LATENT = cache8.Records(1, 576, 512, 64, latent=True)
HEADS = cache8.Records(4, 128, 128, 16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rec,heads,R,V,n", [
    (LATENT, 16, 1, 1, 1), (LATENT, 64, 2, 1, 95), (LATENT, 128, 1, 1, 513), (LATENT, 8, 3, 2, 128),
    (LATENT, 1, 1, 1, 129), (LATENT, 40, 1, 1, 257), (LATENT, 128, 9, 1, 64),
    (HEADS, 16, 2, 1, 2), (HEADS, 4, 3, 1, 97), (HEADS, 32, 1, 3, 640), (HEADS, 12, 2, 2, 33),
    (HEADS, 64, 40, 1, 130), (HEADS, 256, 1, 1, 70),
    (cache8.Records(2, 64, 64, 32), 6, 2, 4, 127), (cache8.Records(3, 80, 80, 1), 9, 2, 1, 200),
    (cache8.Records(1, 16, 16, 4096), 1, 1, 1, 31), (cache8.Records(2, 192, 128, 64), 16, 2, 1, 300),
    (cache8.Records(1, 256, 256, 16), 5, 2, 1, 161), (cache8.Records(5, 48, 112, 7), 10, 2, 1, 66),
    (cache8.Records(1, 640, 512, 16), 17, 1, 1, 99), (cache8.Records(2, 96, 96, 16, latent=True), 8, 2, 1, 77),
    (cache8.Records(1, 128, 16, 64, latent=True), 70, 1, 1, 40), (cache8.Records(1, 64, 512, 64), 24, 1, 1, 140),
])
def test_attend(rec, heads, R, V, n, dtype):
    c = _attend_case(rec, heads, dtype, R, V, n, q_std=2.0)
    assert _attend(c) == 0
    want = _attend64(rec, c["q"], c["sel"], c["slots"], c["hot"], c["scales"], rec.k_dim ** -0.5)
    _attend_close(c["out"], c["lse"], want, dtype)
    first, lse = c["out"].clone(), c["lse"].clone()
    assert _attend(c) == 0                       # the same bits again
    assert torch.equal(first, c["out"]) and torch.equal(lse, c["lse"])


@pytest.mark.parametrize("rec,heads", [(HEADS, 16), (cache8.Records(2, 192, 128, 16), 8), (LATENT, 16)])
def test_attend_many_tiles_of_many_rows(rec, heads):
    """So many rows that none is split, each long enough to go round every stage and table of a
    CTA several times."""
    c = _attend_case(rec, heads, torch.bfloat16, 64, 1, 3001)
    assert _attend(c) == 0
    first = c["out"].clone()
    assert _attend(c) == 0 and torch.equal(first, c["out"])
    some = [0, 37, 63]
    want = _attend64(rec, c["q"][some], c["sel"][some], c["slots"][some], c["hot"][some], c["scales"][some],
                     rec.k_dim ** -0.5)
    _attend_close(c["out"][some], c["lse"][some], want, torch.bfloat16)


@pytest.mark.parametrize("rec,heads", [(LATENT, 64), (HEADS, 16)])
def test_attend_long(rec, heads):
    """One request whose whole long selection is attended, and the same with a peaked
    softmax whose maximum comes late."""
    c = _attend_case(rec, heads, torch.bfloat16, 1, 1, 16000, q_std=4.0)
    c["hot"].view(E4M3)[0, 7] = 448.0
    c["slots"][0, 15000] = 7
    c["sel"][0, 15000] = 5
    assert _attend(c) == 0
    want = _attend64(rec, c["q"], c["sel"], c["slots"], c["hot"], c["scales"], rec.k_dim ** -0.5)
    _attend_close(c["out"], c["lse"], want, torch.bfloat16)


@pytest.mark.parametrize("rec,heads,dtype", [(LATENT, 32, torch.bfloat16), (HEADS, 8, torch.float16)])
def test_attend_empty_rows_and_masked_specials(rec, heads, dtype):
    """Rows that a mask empties give 0 and -inf; NaN and infinities in rows
    that nothing selects, behind the length, or in unused slots stay out."""
    c = _attend_case(rec, heads, dtype, 4, 2, 150, tok=3, pad=0.3)
    c["sel"][1] = c["slots"][1] = -1             # a request that failed
    c["sel"][2, :150] = c["slots"][2, :150] = -1  # one of two rows
    lens = torch.tensor([450, 900, 700, 0], dtype=torch.int32, device="cuda")
    hot = c["hot"].view(4, -1, 3, rec.row_bytes)
    used = torch.zeros(4, hot.shape[1], 3, dtype=torch.bool, device="cuda")
    for r in range(4):
        for s, p in zip(c["slots"][r].tolist(), c["sel"][r].tolist()):
            for u in range(3):
                if s >= 0 and p * 3 + u < int(lens[r]):
                    used[r, s, u] = True
    hot[~used] = 0x7F                            # NaN
    assert _attend(c, record_tokens=3, seq_lens=lens) == 0
    want = _attend64(rec, c["q"], c["sel"], c["slots"], c["hot"], c["scales"], rec.k_dim ** -0.5, tok=3,
                     seq_lens=lens)
    assert bool(torch.isneginf(c["lse"][1]).all()) and bool((c["out"][3] == 0).all())
    _attend_close(c["out"], c["lse"], want, dtype)


def test_attend_no_entries():
    c = _attend_case(HEADS, 8, torch.bfloat16, 2, 1, 4)
    c["sel"], c["slots"] = c["sel"][:, :0].contiguous(), c["slots"][:, :0].contiguous()
    assert _attend(c) == 0
    assert bool((c["out"] == 0).all()) and bool(torch.isneginf(c["lse"]).all())


@pytest.mark.parametrize("rec,heads", [(LATENT, 24), (HEADS, 12)])
def test_attend_pages_residents_blocks_and_strides(rec, heads):
    """Records of 5 tokens with a part-filled last page, every third row
    resident, block-id selections, and views with padding everywhere."""
    g = _gen(21)
    R, V, n, tok = 3, 2, 90, 5
    c = _attend_case(rec, heads, torch.bfloat16, R, V, n, tok=tok, pad=0.0)
    B = c["hot"].shape[1] - 1
    wide = torch.zeros(R, B + 1, tok * rec.row_bytes + 32, dtype=torch.uint8, device="cuda")
    wide[:, :, :tok * rec.row_bytes] = c["hot"]
    res = (_randn(g, 200, tok * rec.row_bytes + 16) * 60).clamp(-448, 448).to(E4M3).view(torch.uint8)
    blocks = torch.stack([torch.randperm(200, device="cuda", generator=g)[:V * n // 3] for _ in range(R)]).int()
    blocks[1, 4] = -1
    slots = c["slots"].clone()
    slots[:, ::3] = B + 1 + torch.randint(0, 200, (R, V * n // 3), device="cuda", generator=g).int()
    slots[1, 12:15] = -1
    qw = torch.zeros(R, V, heads, rec.k_dim + 8, dtype=torch.bfloat16, device="cuda")
    qw[..., :rec.k_dim] = c["q"]
    ow = torch.zeros(R, V, heads, rec.v_dim + 24, dtype=torch.bfloat16, device="cuda")
    scales = (0.2 + torch.rand(R, rec.blocks(600 * tok), rec.columns, device="cuda", generator=g)) / 60
    lens = torch.tensor([2999, 2400, 3000], dtype=torch.int32, device="cuda")
    st = _status()
    cache8.attend(rec, qw[..., :rec.k_dim], blocks, slots, wide[:, :, :tok * rec.row_bytes], scales,
                  ow[..., :rec.v_dim], lse=c["lse"], record_tokens=tok, sel_block_tokens=3, seq_lens=lens,
                  resident=res[:, :tok * rec.row_bytes], status=st)
    assert int(st) == 0
    want = _attend64(rec, c["q"], blocks, slots, c["hot"], scales, rec.k_dim ** -0.5, tok=tok, sel_block=3,
                     seq_lens=lens, resident=res)
    _attend_close(ow[..., :rec.v_dim], c["lse"], want, torch.bfloat16)
    assert bool((ow[..., rec.v_dim:] == 0).all())


@pytest.mark.parametrize("rec,heads,dtype,tok", [(LATENT, 32, torch.bfloat16, 1), (HEADS, 16, torch.bfloat16, 1),
                                                 (HEADS, 8, torch.float16, 4)])
def test_attend_residents_mixed_every_way(rec, heads, dtype, tok):
    """Rows of both stores side by side: runs of one, alternating ones, masked ones between."""
    g = _gen(31)
    c = _attend_case(rec, heads, dtype, 3, 1, 320, tok=tok, pad=0.15)
    B = c["hot"].shape[1] - 1
    res = (_randn(g, 77, tok * rec.row_bytes) * 60).clamp(-448, 448).to(E4M3).view(torch.uint8)
    pick = torch.randint(0, 77, (3, 320), device="cuda", generator=g).int() + B + 1
    far = torch.zeros(3, 320, dtype=torch.bool, device="cuda")
    far[:, 64:128] = True
    far[:, 128:200:2] = True
    far[:, 200:260] = torch.rand(3, 60, device="cuda", generator=g) < 0.5
    c["slots"] = torch.where(far & (c["slots"] >= 0), pick, c["slots"]).contiguous()
    assert _attend(c, record_tokens=tok, resident=res) == 0
    want = _attend64(rec, c["q"], c["sel"], c["slots"], c["hot"], c["scales"], rec.k_dim ** -0.5, tok=tok,
                     resident=res)
    _attend_close(c["out"], c["lse"], want, dtype)


def test_attend_reports_what_is_out_of_range():
    c = _attend_case(HEADS, 8, torch.bfloat16, 2, 1, 50, pad=0.0)
    B = c["hot"].shape[1] - 1
    good = dict(c, sel=c["sel"].clone(), slots=c["slots"].clone(), out=c["out"].clone(), lse=c["lse"].clone())
    for j, (s, p) in enumerate(((B + 1, 3), (-7, 4), (2 ** 31 - 1, 5), (4, 10 ** 8), (5, -3), (-2 ** 31, 1))):
        c["slots"][0, j], c["sel"][0, j] = s, p
        good["slots"][0, j] = good["sel"][0, j] = -1
    assert _attend(c) == H.ERR_RANGE
    assert _attend(good) == 0
    assert torch.equal(c["out"], good["out"]) and torch.equal(c["lse"], good["lse"])


def test_attend_num_reqs_streams_and_graphs():
    c = _attend_case(HEADS, 8, torch.bfloat16, 4, 1, 200)
    n = torch.tensor([3], dtype=torch.int32, device="cuda")
    want = _attend64(HEADS, c["q"], c["sel"], c["slots"], c["hot"], c["scales"], 128 ** -0.5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        cache8.attend(HEADS, c["q"], c["sel"], c["slots"], c["hot"], c["scales"], c["out"], lse=c["lse"], num_reqs=n)
    s.synchronize()
    _attend_close(c["out"][:3], c["lse"][:3], [x[:3] for x in want], torch.bfloat16)
    assert bool(torch.isnan(c["out"][3]).all()) and bool(torch.isnan(c["lse"][3]).all())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache8.attend(HEADS, c["q"], c["sel"], c["slots"], c["hot"], c["scales"], c["out"], lse=c["lse"], num_reqs=n)
    n.fill_(4)
    c["out"].zero_()
    graph.replay()
    torch.cuda.synchronize()
    _attend_close(c["out"], c["lse"], want, torch.bfloat16)


def test_attend_offsets_beyond_32_bits():
    """Requests whose hot rows lie more than 4 GB apart."""
    rec, B, R, n = LATENT, 9, 3, 200
    far = torch.empty(2 * (5 << 29) + (B + 1) * 576, dtype=torch.uint8, device="cuda")   # 5.4 GB
    hot = far.as_strided((R, B + 1, 576), (5 << 29, 576, 1))
    c = _attend_case(rec, 16, torch.bfloat16, R, 1, 10, B=B)
    hot.copy_(c["hot"])
    c["hot"] = hot
    assert _attend(c) == 0
    want = _attend64(rec, c["q"], c["sel"], c["slots"], c["hot"], c["scales"], 576 ** -0.5)
    _attend_close(c["out"], c["lse"], want, torch.bfloat16)


@pytest.mark.parametrize("rec,heads", [(LATENT, 64), (HEADS, 16)])
def test_attend_extreme_scores_and_scales(rec, heads):
    """Scores far apart (one-hot rows), all equal ones, tiny q, and block scales that differ by 2^12."""
    c = _attend_case(rec, heads, torch.bfloat16, 3, 1, 300, pad=0.0)
    c["q"][0] *= 200
    c["q"][1] = 0
    c["q"][2] *= 2.0 ** -60
    c["scales"][0] *= torch.where(torch.arange(c["scales"].shape[1], device="cuda") % 2 == 0, 1.0,
                                  2.0 ** -12)[:, None]
    assert _attend(c) == 0
    want = _attend64(rec, c["q"], c["sel"], c["slots"], c["hot"], c["scales"], rec.k_dim ** -0.5)
    _attend_close(c["out"], c["lse"], want, torch.bfloat16)


# ---------------------------------------------------------------------------------------------
# pages
# ---------------------------------------------------------------------------------------------
class PageModel:
    """The pool by plain lists."""

    def __init__(self, pages, R, M, bt, layers, row, seed):
        rng = np.random.default_rng(seed)
        self.bt, self.row, self.M = bt, row, M
        self.tables = np.full((R, M), -1, np.int32)
        self.refs = np.zeros(pages, np.int32)
        self.store = rng.integers(0, 256, (layers, pages, bt * row), dtype=np.uint8)
        self.full = False

    def _take(self, need, free):
        if need > len(free):
            self.full = True
            free.clear()
            return None
        return [free.pop(0) for _ in range(need)]

    def grow(self, reqs, blocks):
        free = np.flatnonzero(self.refs == 0).tolist()
        for r, b in zip(reqs, blocks):
            holes = [j for j in range(b) if self.tables[r, j] == -1]
            got = self._take(len(holes), free) if holes else []
            for j, p in zip(holes, got or []):
                self.tables[r, j], self.refs[p] = p, 1

    def fork(self, src, dst, tokens):
        free = np.flatnonzero(self.refs == 0).tolist()
        copies = []
        for s, d, t in zip(src, dst, tokens):
            full, part = divmod(t, self.bt)
            last = self.tables[s, full] if part else -1
            if last >= 0:
                got = self._take(1, free)
                if got is None:
                    continue
            self.tables[d, :full] = self.tables[s, :full]
            for p in self.tables[s, :full]:
                if p >= 0:
                    self.refs[p] += 1
            if last >= 0:
                self.tables[d, full], self.refs[got[0]] = got[0], 1
                copies.append((last, got[0], part * self.row))
        for a, b, n in copies:
            self.store[:, b, :n] = self.store[:, a, :n]

    def free(self, reqs):
        for r in reqs:
            for p in self.tables[r]:
                if p >= 0:
                    self.refs[p] -= 1
            self.tables[r] = -1

    def compact(self):
        used = np.flatnonzero(self.refs > 0)
        m = len(used)
        movers, holes = used[used >= m], np.flatnonzero(self.refs[:m] == 0)
        for a, b in zip(movers, holes):
            self.store[:, b] = self.store[:, a]
            self.refs[b], self.refs[a] = self.refs[a], 0
            self.tables[self.tables == a] = b


def _same(pool, model, st):
    np.testing.assert_array_equal(pool.tables.cpu().numpy(), model.tables)
    np.testing.assert_array_equal(pool.refs.cpu().numpy(), model.refs)
    np.testing.assert_array_equal(pool.store.cpu().numpy(), model.store)
    assert int(st) == (H.ERR_FULL if model.full else 0)
    st.zero_()
    model.full = False


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("pages_,R,M,bt,layers,row,seed", [
    (1, 1, 1, 1, 1, 16, 0), (37, 6, 9, 16, 2, 48, 1), (500, 24, 31, 4, 3, 16, 2), (64, 40, 3, 7, 1, 144, 3),
    (9001, 128, 100, 1, 1, 16, 4), (40000, 300, 150, 1, 1, 16, 5), (130, 10, 16, 64, 4, 576, 6),
])
def test_pages_random_life(pages_, R, M, bt, layers, row, seed):
    """Random requests begin, branch, end and are compacted; everything equals
    the plain lists after every call, exhaustion included."""
    rng = np.random.default_rng(seed)
    model = PageModel(pages_, R, M, bt, layers, row, seed)
    st = _status()
    pool = pages.PagePool(torch.from_numpy(model.store.copy()).cuda(), block_tokens=bt, requests=R,
                          max_blocks=M, status=st)
    for step in range(24):
        kind = step % 4 if step < 8 else int(rng.integers(0, 4))
        empty = np.flatnonzero((model.tables == -1).all(1))
        some = rng.permutation(R)[:max(1, R // 3)]
        if kind == 0:
            b = rng.integers(0, M + 1, len(some))
            model.grow(some, b)
            pool.grow(_i32(some), _i32(b))
        elif kind == 1 and 0 < len(empty) < R:
            dst = rng.permutation(empty)[:max(1, len(empty) // 2)]
            src = rng.choice(np.setdiff1d(np.arange(R), empty), len(dst))
            t = rng.integers(0, M * bt + 1, len(dst))
            model.fork(src, dst, t)
            pool.fork(_i32(src), _i32(dst), _i32(t))
        elif kind == 2:
            model.free(some[:max(1, len(some) // 2)])
            pool.free(_i32(some[:max(1, len(some) // 2)]))
        else:
            model.compact()
            pool.compact()
        _same(pool, model, st)


@pytest.mark.parametrize("pages_,R,M,bt,layers,row,seed", [
    (20011, 24, 1300, 2, 1, 16, 7), (3000, 9, 2047, 1, 2, 16, 8), (70001, 100, 700, 1, 1, 16, 9),
    (33000, 41, 1024, 1, 1, 16, 10),
])
def test_pages_long_tables(pages_, R, M, bt, layers, row, seed):
    """The same with tables so long that an entry has 2, 4 or 8 warps, each with its own part
    of the blocks; odd lengths, and a pool that runs out."""
    test_pages_random_life(pages_, R, M, bt, layers, row, seed)


def test_pages_refusals_on_the_device():
    """Bad indices and a destination that holds pages are skipped and reported."""
    model = PageModel(32, 5, 4, 8, 2, 16, 1)
    st = _status()
    pool = pages.PagePool(torch.from_numpy(model.store.copy()).cuda(), block_tokens=8, requests=5,
                          max_blocks=4, status=st)
    model.grow([0, 1], [4, 2])
    pool.grow(_i32([0, 1]), _i32([4, 2]))
    _same(pool, model, st)
    pool.fork(_i32([0, 0, 9, 0, 0]), _i32([1, -1, 2, 3, 4]), _i32([8, 8, 8, 33, -1]))
    assert int(st) == H.ERR_RANGE
    st.zero_()
    _same(pool, model, st)
    pool.grow(_i32([5, -1, 2]), _i32([1, 1, 5]))
    pool.free(_i32([7, -2]))
    assert int(st) == H.ERR_RANGE
    st.zero_()
    _same(pool, model, st)


def test_pages_strided_store_and_free_twice():
    """A store inside a larger one, a request listed twice by free, and a graph."""
    big = torch.zeros(2, 50, 8 * 32 + 64, dtype=torch.uint8, device="cuda")
    g = _gen(2)
    big.copy_(torch.randint(0, 256, big.shape, device="cuda", generator=g).to(torch.uint8))
    rest = big[:, :, 256:].clone()
    model = PageModel(50, 8, 6, 8, 2, 32, 2)
    model.store[:] = big[:, :, :256].cpu().numpy()
    st = _status()
    pool = pages.PagePool(big[:, :, :256], block_tokens=8, requests=8, max_blocks=6, status=st)
    model.grow([0, 1, 2, 3], [6, 5, 6, 3])
    pool.grow(_i32([0, 1, 2, 3]), _i32([6, 5, 6, 3]))
    model.fork([0, 2], [5, 6], [41, 20])
    pool.fork(_i32([0, 2]), _i32([5, 6]), _i32([41, 20]))
    model.free([0, 1])
    pool.free(_i32([0, 1, 0]))
    _same(pool, model, st)
    graph = torch.cuda.CUDAGraph()
    pool.compact()                               # warm
    model.compact()
    with torch.cuda.graph(graph):
        pool.compact()
    model.free([2])
    pool.free(_i32([2]))
    graph.replay()
    model.compact()
    _same(pool, model, st)
    assert torch.equal(big[:, :, 256:], rest)
