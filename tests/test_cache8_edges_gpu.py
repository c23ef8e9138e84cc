"""The 8-bit record operators at the edges of their ranges, against plain computations in 64
bits: sizes that divide nothing, block scales that are no numbers, probabilities far below a
row's largest.  Tolerances follow from the formats, as in test_cache8_gpu.py."""
import numpy as np
import pytest
import torch

from host_offload_serving_gb300 import cache8
from test_cache8_gpu import _gen, _pack64, _pack_close, _randn, _status

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


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
