"""The 8-bit record operators at the edges of their ranges, against plain computations in 64
bits: sizes that divide nothing, block scales that are no numbers, probabilities far below a
row's largest.  Tolerances follow from the formats, as in test_cache8_gpu.py."""
import numpy as np
import pytest
import torch

from host_offload_serving_gb300 import cache8, pages
from host_offload_serving_gb300 import hisparse as H
from test_cache8_gpu import (E4M3, HEADS, LATENT, U, PageModel, _attend, _attend64, _attend_case, _attend_close,
                             _gen, _pack64, _pack_close, _randn, _rotated64, _same, _status)

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------------------------
# rotary
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_sines_of_small_angles(interleaved):
    """The sine of an angle far below a turn is as fine, relatively, as its 32 bits."""
    rot, T = 64, 6
    turns, _ = cache8.rotary_turns(rot, base=1e9)
    pos = _i32([1, 3, 100, -1, -7, 4097])
    x = torch.zeros(T, 1, rot, device="cuda")
    even = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    x[..., even + (1 if interleaved else rot // 2)] = 1.0    # pairs (0, 1) -> (-sin, cos)
    y = cache8.rotate(x, pos, turns.cuda(), interleaved=interleaved, out=torch.empty_like(x))[0]
    want, _ = _rotated64(x, pos, turns, 0, interleaved, 1.0)
    got, want = y.double().cpu().numpy()[..., even], want[..., even]
    # the phase rounded to 24 bits, sincospif (2 units in the last place), one product
    rel = np.abs(got - want) / np.abs(want)
    small = np.abs(want) < 0.25
    assert small.sum() > 50 and rel[small].max() <= 4 * 2.0 ** -23


# ---------------------------------------------------------------------------------------------
# pack
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("rec,rot", [
    (cache8.Records(1, 384, 256, 128, latent=True), 64), (cache8.Records(1, 608, 512, 128, latent=True), 608),
    (cache8.Records(1, 560, 512, 200, latent=True), 128), (cache8.Records(2, 176, 128, 256), 176),
    (cache8.Records(1, 96, 96, 512, latent=True), 32),
])
def test_pack_blocks_walked_by_teams_with_threads_left_over(rec, rot):
    """Blocks that a CTA walks twice, with heads whose units do not divide its 640 threads: the
    threads left over turn nothing."""
    g = _gen(rec.k_dim)
    lens = [3 * rec.block_tokens + 7, 2 * rec.block_tokens]
    start, cu = [5, 0], [0, lens[0], sum(lens)]
    k = (_randn(g, cu[-1], rec.kv_heads, rec.k_dim) * 2).to(torch.bfloat16)
    v = None if rec.latent else _randn(g, cu[-1], rec.kv_heads, rec.v_dim).to(torch.bfloat16)
    P = 4 * rec.block_tokens + 12
    scales = torch.zeros(2, rec.blocks(P), rec.columns, device="cuda")
    turns = cache8.rotary_turns(rot)[0]
    want, want_s = _pack64(rec, k, v, scales, start, cu, [0, 1], 2.0, turns, rec.k_dim - rot)
    dst = torch.zeros(2, P, rec.row_bytes, dtype=torch.uint8, device="cuda")
    st = _status()
    cache8.pack(rec, k, v, dst, scales, _i32(start), cu_lens=_i32(cu), max_len=max(lens), turns=turns.cuda(),
                rot_offset=rec.k_dim - rot, status=st)
    assert int(st) == 0
    np.testing.assert_allclose(scales.double().cpu().numpy(), want_s, rtol=4e-6)
    _pack_close(torch.cat([dst[i, start[i]:start[i] + lens[i]] for i in range(2)]), want)


@pytest.mark.parametrize("rec", [LATENT, HEADS, cache8.Records(2, 80, 48, 1)], ids=["latent", "heads", "one"])
def test_pack_blocks_whose_only_values_are_infinite(rec):
    """Infinities saturate also where nothing else sets a scale; it stays unset."""
    k = torch.zeros(3, rec.kv_heads, rec.k_dim, device="cuda")
    k[0, 0, 3], k[1, 0, 5], k[2, 0, 7] = float("inf"), float("-inf"), float("nan")
    v = None if rec.latent else torch.zeros(3, rec.kv_heads, rec.v_dim, device="cuda")
    scales = torch.zeros(1, rec.blocks(3), rec.columns, device="cuda")
    rows = torch.full((3, rec.row_bytes), 0x55, dtype=torch.uint8, device="cuda")
    cache8.pack(rec, k, v, rows, scales, _i32([0]), max_len=3)
    want = torch.zeros_like(rows)
    want[0, 3], want[1, 5], want[2, 7] = 0x7E, 0xFE, 0x7F
    got = rows.clone()
    got[2, 7] &= 0x7F
    assert torch.equal(got, want)
    assert bool((scales == 0).all())


# ---------------------------------------------------------------------------------------------
# where tensors lie
# ---------------------------------------------------------------------------------------------
def test_host_tensors_are_refused_and_pinned_rows_written():
    """One pageable host tensor among device tensors is refused by every call; rows may go to
    pinned host memory."""
    g = _gen(1)
    rec = cache8.Records(1, 64, 64, 16)
    turns, pos = cache8.rotary_turns(32)[0], _i32([0, 1, 2])
    x = _randn(g, 3, 1, 64)
    for bad in (dict(turns=turns), dict(pos=pos.cpu()), dict(k=x.cpu()), dict(out=x.cpu())):
        kw = dict(dict(pos=pos, turns=turns.cuda()), **bad)
        with pytest.raises(ValueError, match="is on cpu"):
            cache8.rotate(x, kw.pop("pos"), kw.pop("turns"), **kw)
    scales, start = torch.zeros(1, 1, 2, device="cuda"), _i32([0])
    dst = torch.zeros(3, 128, dtype=torch.uint8, device="cuda")
    for bad in (dict(turns=turns), dict(start=start.cpu()), dict(cu_lens=_i32([0, 3]).cpu()), dict(dst=dst.cpu()),
                dict(scales=scales.cpu()), dict(v=x.cpu()), dict(status=start.cpu())):
        kw = dict(dict(v=x, dst=dst, scales=scales, start=start), **bad)
        with pytest.raises(ValueError, match="is on cpu"):
            cache8.pack(rec, x, kw.pop("v"), kw.pop("dst"), kw.pop("scales"), kw.pop("start"), max_len=3, **kw)
    q, sel = _randn(g, 1, 1, 1, 64).bfloat16(), _i32([[0, 1, 2]])
    for bad in (dict(sel=sel.cpu()), dict(slots=sel.cpu()), dict(hot=dst[None].cpu()), dict(out=q.cpu()),
                dict(scales=scales.cpu()), dict(lse=torch.zeros(1, 1, 1)), dict(seq_lens=start.cpu()),
                dict(resident=dst.cpu()), dict(num_reqs=start.cpu()), dict(status=start.cpu())):
        kw = dict(dict(sel=sel, slots=sel, hot=dst[None], scales=scales, out=q.clone()), **bad)
        with pytest.raises(ValueError, match="is on cpu"):
            cache8.attend(rec, q, kw.pop("sel"), kw.pop("slots"), kw.pop("hot"), kw.pop("scales"), kw.pop("out"), **kw)
    pool = pages.PagePool(dst.view(1, 3, 128), block_tokens=1, requests=2, max_blocks=2)
    for call in (lambda: pool.grow(start.cpu(), start), lambda: pool.grow(start, start.cpu()),
                 lambda: pool.fork(start, start.cpu(), start), lambda: pool.free(start.cpu())):
        with pytest.raises(ValueError, match="is on cpu"):
            call()
    pinned = torch.zeros(3, 128, dtype=torch.uint8).pin_memory()
    cache8.pack(rec, x, x, dst, scales, start, max_len=3)
    cache8.pack(rec, x, x, pinned, scales, start, max_len=3)
    torch.cuda.synchronize()
    assert bool(dst.any()) and torch.equal(dst.cpu(), pinned)


# ---------------------------------------------------------------------------------------------
# pages
# ---------------------------------------------------------------------------------------------
def test_pages_grow_by_more_than_31_bits():
    """A list that asks for more than 2^31 pages: the entries before the first that finds too few
    get theirs, the others none."""
    R, M, n = 8192, 262300, 100
    assert 15 + (R - 2) * M > 2 ** 31
    st = _status()
    pool = pages.PagePool(torch.zeros(1, n, 16, dtype=torch.uint8, device="cuda"), block_tokens=1, requests=R,
                          max_blocks=M, status=st)
    want = torch.full((R,), M, dtype=torch.int32, device="cuda")
    want[0], want[1] = 10, 5
    pool.grow(torch.arange(R, dtype=torch.int32, device="cuda"), want)
    assert int(st) == H.ERR_FULL
    assert pool.tables[0, :11].tolist() == [*range(10), -1] and pool.tables[1, :6].tolist() == [*range(10, 15), -1]
    assert pool.refs.tolist() == [1] * 15 + [0] * (n - 15)
    assert int((pool.tables != -1).sum()) == 15


def test_pages_compact_reports_entries_that_no_count_stands_for():
    """A table entry whose page has no count is reported and stays, whatever an earlier call left in
    the workspace."""
    model = PageModel(64, 4, 8, 4, 1, 16, 3)
    st = _status()
    pool = pages.PagePool(torch.from_numpy(model.store.copy()).cuda(), block_tokens=4, requests=4, max_blocks=8,
                          status=st)
    pool.grow(_i32([0, 1]), _i32([3, 4]))
    model.grow([0, 1], [3, 4])
    pool.free(_i32([0]))
    model.free([0])
    pool.tables[2, 5] = 40
    model.tables[2, 5] = 40
    pool.work.fill_(1)
    pool.compact()
    model.compact()
    assert int(st) == H.ERR_RANGE
    st.zero_()
    _same(pool, model, st)


# ---------------------------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------------------------
def _bits(pattern):
    return torch.tensor(pattern, dtype=torch.int32, device="cuda").view(torch.float32)


@pytest.mark.parametrize("rec,heads", [(LATENT, 16), (HEADS, 16), (cache8.Records(2, 64, 64, 16), 64),
                                       (cache8.Records(1, 128, 128, 16), 64)])
@pytest.mark.parametrize("pattern", [0x7FFFFFFF, 0x7FC00000, -1])
def test_attend_scales_of_k_that_are_nan(rec, heads, pattern):
    """Whatever its bits, a NaN scale of K makes the rows that read it NaN, and no others."""
    c = _attend_case(rec, heads, torch.bfloat16, 2, 1, 200, pad=0.1)
    assert _attend(c) == 0
    out, lse = c["out"].clone(), c["lse"].clone()
    j = int((c["slots"][1] >= 0).nonzero()[100])
    c["scales"][1, int(c["sel"][1, j]) // rec.block_tokens, rec.kv_heads - 1] = _bits(pattern)
    assert _attend(c) == 0
    hit = torch.zeros(2, 1, heads, dtype=torch.bool, device="cuda")
    hit[1, 0, heads - heads // rec.kv_heads:] = True
    assert bool(torch.isnan(c["out"][hit]).all()) and bool(torch.isnan(c["lse"][hit]).all())
    assert torch.equal(c["out"][~hit], out[~hit]) and torch.equal(c["lse"][~hit], lse[~hit])


@pytest.mark.parametrize("heads", [8, 16, 128, 256])
@pytest.mark.parametrize("pattern", [0x7FFFFFFF, 0x7FC00000, 0x7F800000])
def test_attend_scales_of_v_that_are_no_numbers(heads, pattern):
    """... and one of V their outputs; the softmax and its lse have nothing of V in them."""
    c = _attend_case(HEADS, heads, torch.bfloat16, 2, 1, 200, pad=0.1)
    assert _attend(c) == 0
    out = c["out"].clone()
    want = _attend64(HEADS, c["q"], c["sel"], c["slots"], c["hot"], c["scales"], 128 ** -0.5)
    j = int((c["slots"][1] >= 0).nonzero()[100])
    c["scales"][1, int(c["sel"][1, j]) // 16, HEADS.columns - 1] = _bits(pattern)
    assert _attend(c) == 0
    hit = torch.zeros(2, 1, heads, dtype=torch.bool, device="cuda")
    hit[1, 0, heads - heads // 4:] = True
    assert bool((~torch.isfinite(c["out"][hit])).all())
    assert torch.equal(c["out"][~hit], out[~hit])
    _attend_close(out, c["lse"], want, torch.bfloat16)


def test_attend_infinite_scales_of_k():
    """Scores of minus infinity have no weight; a score of plus infinity leaves no number."""
    c = _attend_case(HEADS, 16, torch.bfloat16, 2, 1, 200, pad=0.1)
    j = int((c["slots"][1] >= 0).nonzero()[100])
    clean = c["scales"].clone()
    blk = int(c["sel"][1, j]) // 16
    same = (c["sel"][1] // 16 == blk) & (c["sel"][1] >= 0)
    same[j] = False
    c["sel"][1, same] = c["slots"][1, same] = -1           # the block's only token
    c["scales"][1, blk, :4] = float("inf")
    assert _attend(c) == 0
    gone = c["slots"].clone()
    gone[1, j] = -1
    want = _attend64(HEADS, c["q"], c["sel"], gone, c["hot"], clean, 128 ** -0.5)
    row = c["hot"][1, c["slots"][1, j]].view(E4M3).double()[:4 * 128].view(4, 128)
    up = torch.einsum("hgd,hd->hg", c["q"][1, 0].double().view(4, 4, 128), row).view(16) > 0
    low = torch.ones(2, 1, 16, dtype=torch.bool, device="cuda")
    low[1, 0] = ~up
    assert 0 < int(up.sum()) < 16
    assert bool((~torch.isfinite(c["out"][~low])).all()) and bool((~torch.isfinite(c["lse"][~low])).all())
    m = low.cpu().numpy()
    _attend_close(c["out"][low][None, None], c["lse"][low][None, None], [x[m][None, None] for x in want], torch.bfloat16)


def _beside_dominant_tokens(rec, heads, R, at, weight, dtype, floor):
    """Rows of 2048 tokens of which those of entries `at` have `weight` together and a V of 0, so that
    the output is made of the others' small probabilities.  Its error is bounded by itself: the rounding of
    the output (at most U / 3^0.5 of its norm, 2^-25 a value at the lower end of f16) with half as much
    again, 2^-11 of each probability, and `floor` of the largest probability times its scale of V (half as
    much again over 3^0.5), by the norm of V's bytes."""
    n, D, K = 2048, rec.k_dim, rec.kv_heads
    c = _attend_case(rec, heads, dtype, R, 1, n, pad=0.0)
    hot, scales = c["hot"].view(E4M3), c["scales"]
    far = torch.arange(K, device="cuda") * D + D - 1
    hot[..., far] = torch.tensor(0.0, device="cuda").to(E4M3)
    c["q"][..., D - 1] = 1.0
    # a block of their own, whose scale makes their scores what the weight asks for
    blk = scales.shape[1]
    for i, entry in enumerate(at):
        slot = c["slots"][:, entry].long()
        hot[torch.arange(R, device="cuda"), slot] = torch.tensor(0.0, device="cuda").to(E4M3)
        for f in far.tolist():
            hot[torch.arange(R, device="cuda"), slot, f] = torch.tensor(448.0, device="cuda").to(E4M3)
        c["sel"][:, entry] = blk * rec.block_tokens + i
    c["scales"] = torch.cat([scales, torch.full((R, 1, rec.columns), 1 / 60, device="cuda")], 1).contiguous()
    some = [0, R - 1] if R > 1 else [0]
    pick = lambda: _attend64(rec, c["q"][some], c["sel"][some], c["slots"][some], c["hot"][some], c["scales"][some], D ** -0.5)
    c["scales"][:, blk, :K] = -50.0
    rest = float(np.median(pick()[1]))                    # lse of the others
    c["scales"][:, blk, :K] = (rest + np.log(weight / (1 - weight) / len(at))) * D ** 0.5 / 448
    assert _attend(c) == 0
    want, lse, _, _ = pick()
    got = c["out"][some].double().cpu().numpy()
    size = np.linalg.norm(want, axis=-1)
    err = np.linalg.norm(got - want, axis=-1) / size
    v_cols = rec.v_dim if rec.latent else K * rec.v_dim
    bytes_v = hot[some][..., :v_cols] if rec.latent else hot[some][..., K * D:]
    norm_v = float(bytes_v.double().norm(dim=(1, 2)).max()) / (1 if rec.latent else K ** 0.5)
    s_v = float(c["scales"][:, blk, 0 if rec.latent else K].max())
    low = 0.0 if dtype is torch.bfloat16 else 2.0 ** -25 * rec.v_dim ** 0.5 / size
    tol = 1.5 * (U[dtype] + low) / 3 ** 0.5 + 2.0 ** -11 \
        + 1.5 * floor / 3 ** 0.5 * weight / len(at) * s_v * norm_v / size
    assert (err <= tol).all(), (float((err / tol).max()), float(err.max()), float(tol.min()))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rec,heads,R,at", [
    (LATENT, 128, 1, 0), (LATENT, 128, 80, 5), (LATENT, 16, 160, 2040), (LATENT, 64, 2, 700),
    (HEADS, 16, 40, 0), (HEADS, 16, 1, 1300), (HEADS, 128, 1, 0), (cache8.Records(2, 64, 64, 32), 6, 160, 1),
])
@pytest.mark.parametrize("weight", [0.5, 0.95, 0.997, 0.9999])
def test_attend_beside_a_dominant_token_without_values(rec, heads, R, at, weight, dtype):
    """One token far above the others of its tile."""
    _beside_dominant_tokens(rec, heads, R, [at], weight, dtype, 2.0 ** -32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rec,heads,R", [(HEADS, 16, 40), (HEADS, 16, 1), (cache8.Records(1, 128, 128, 64), 64, 160)])
@pytest.mark.parametrize("weight", [0.9, 0.997])
def test_attend_beside_dominant_tokens_in_every_warp(rec, heads, R, weight, dtype):
    """Several, so placed in the first tile that each warp has one and none stands out."""
    _beside_dominant_tokens(rec, heads, R, [3, 35, 67, 99], weight, dtype, 2.0 ** -25)


@pytest.mark.parametrize("rec,heads", [(HEADS, 16), (cache8.Records(1, 128, 128, 16), 64)])
def test_attend_first_tile_of_scores_of_minus_infinity(rec, heads):
    """A head whose first tile has only a score of minus infinity takes its offset from later tiles
    (other heads of the tile have one of plus infinity, and no result)."""
    c = _attend_case(rec, heads, torch.bfloat16, 1, 1, 4096, pad=0.0)
    K, D = rec.kv_heads, rec.k_dim
    hot = c["hot"].view(E4M3)
    far = torch.arange(K, device="cuda") * D + D - 1      # the last value of each K head
    hot[..., far] = torch.tensor(-448.0, device="cuda").to(E4M3)
    c["scales"][..., :K] = 1 / 64
    c["q"][..., D - 1] = 300.0 * D ** 0.5 / 7.0           # scores of about -300
    c["q"][:, :, 1::2, D - 1] *= -1.0                     # and of 300
    c["scales"] = torch.cat([c["scales"], torch.ones(1, 1, rec.columns, device="cuda")], 1).contiguous()
    c["scales"][0, -1, :K] = float("inf")
    c["sel"][0, :128] = c["slots"][0, :128] = -1
    c["slots"][0, 128:][c["slots"][0, 128:] == 0] = -1
    hot[0, 0, :K * D] = torch.tensor(0.0, device="cuda").to(E4M3)
    hot[0, 0, far] = torch.tensor(-448.0, device="cuda").to(E4M3)
    gone = c["slots"].clone()
    c["slots"][0, 77], c["sel"][0, 77] = 0, (c["scales"].shape[1] - 1) * rec.block_tokens
    assert _attend(c) == 0
    want = _attend64(rec, c["q"], c["sel"], gone, c["hot"], c["scales"], D ** -0.5)
    even = [x[:, :, ::2] for x in want]
    _attend_close(c["out"][:, :, ::2], c["lse"][:, :, ::2], even, torch.bfloat16)
    assert bool(torch.isnan(c["out"][:, :, 1::2]).all())


@pytest.mark.parametrize("seq,tok,block", [(100, 16, 1), (1000, 64, 16), (7, 5, 2)])
def test_attend_last_page_beyond_the_scale_table(seq, tok, block):
    """Tokens of a part-filled last page do not count, whether or not the scale table reaches them."""
    rec = cache8.Records(2, 64, 64, block)
    n = -(-seq // tok)
    c = _attend_case(rec, 8, torch.bfloat16, 2, 1, n, tok=tok, pad=0.0)
    c["sel"] = torch.stack([torch.randperm(n, device="cuda") for _ in range(2)]).int()
    c["scales"] = c["scales"][:, :rec.blocks(seq)].contiguous()
    lens = _i32([seq, seq])
    assert rec.blocks(seq) * block < n * tok
    assert _attend(c, record_tokens=tok, seq_lens=lens) == 0
    want = _attend64(rec, c["q"], c["sel"], c["slots"], c["hot"], c["scales"], 64 ** -0.5, tok=tok, seq_lens=lens)
    _attend_close(c["out"], c["lse"], want, torch.bfloat16)
    assert _attend(c, record_tokens=tok) == H.ERR_RANGE      # without lengths they are selected


@pytest.mark.parametrize("share", [0.02, 0.5, 1.0])
@pytest.mark.parametrize("heads,R,n", [(16, 1, 9000), (16, 64, 3001), (128, 2, 700)])
def test_attend_blocks_without_a_scale_of_v(heads, R, n, share):
    """Blocks whose V is all 0 have a scale of 0; their tokens have their weight all the same."""
    c = _attend_case(HEADS, heads, torch.bfloat16, R, 1, n)
    none = torch.rand(R, c["scales"].shape[1], 1, device="cuda", generator=_gen(n)) < share
    c["scales"][..., 4:] = c["scales"][..., 4:].masked_fill(none, 0.0)
    assert _attend(c) == 0
    some = [0, R - 1] if R > 1 else [0]
    want = _attend64(HEADS, c["q"][some], c["sel"][some], c["slots"][some], c["hot"][some], c["scales"][some],
                     128 ** -0.5)
    _attend_close(c["out"][some], c["lse"][some], want, torch.bfloat16)
