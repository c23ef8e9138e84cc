"""Decode over 8-bit records end to end, on a small latent-attention model of random weights.

A prompt is packed once: its first pages into a resident store, all of its rows into the
host pool.  The prompt's request is forked, so that two continuations share the resident pages.
Then, in every layer of every step, q is turned, the new token's record is packed, the positions
that an indexer picks are resolved (resident store, hot buffer, host pool), and
attention reads the rows where they lie.  At the end one request's pages are freed and the
store is compacted.

    python examples/decode_8bit.py [--steps 8] [--check]
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
from host_offload_serving_gb300 import cache8, pages, runtime  # noqa: E402

R, LAYERS, HEADS, DIM = 3, 2, 16, 256          # requests (one stays idle), layers, query heads, width
REC = cache8.Records(kv_heads=1, k_dim=576, v_dim=512, block_tokens=64, latent=True)
ROT = 64                                       # values at the end of a K head that turn
PROMPT, TOP_K, HOT, PAGE, PAGES = 1000, 256, 512, 64, 40
RESIDENT = 5                                   # pages of the prompt that stay in HBM, the last part-filled
INDEX = 32                                     # width of the indexer's keys


class Model:
    """Random weights, the caches of R requests, and the two calls that use them."""

    def __init__(self, steps, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def rand(*shape):
            return (torch.randn(*shape, device="cuda", generator=g) * shape[-2] ** -0.5).bfloat16()
        self.w_q = [rand(DIM, HEADS * REC.k_dim) for _ in range(LAYERS)]
        self.w_k = [rand(DIM, REC.k_dim) for _ in range(LAYERS)]
        self.w_o = [rand(HEADS * REC.v_dim, DIM) for _ in range(LAYERS)]
        self.w_i = [rand(DIM, INDEX) for _ in range(LAYERS)]
        self.prompt = rand(PROMPT, DIM)
        self.P = PROMPT + steps
        self.mem = runtime.WorkloadMemory(R, LAYERS, HOT, self.P, REC.row_bytes)
        self.hs = runtime.HiSparse(R, LAYERS, TOP_K, HOT, self.P, REC.row_bytes, self.mem.layer_buffers())
        self.scales = torch.zeros(LAYERS, R, REC.blocks(self.P), REC.columns, device="cuda")
        self.index = torch.zeros(LAYERS, R, self.P, INDEX, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        store = torch.zeros(LAYERS, PAGES, PAGE * REC.row_bytes, dtype=torch.uint8, device="cuda")
        self.pool = pages.PagePool(store, block_tokens=PAGE, requests=R, max_blocks=-(-self.P // PAGE),
                                   status=self.status)
        turns, self.amplitude = cache8.rotary_turns(ROT, scaling="linear", factor=4.0)
        self.turns = turns.cuda()
        self.new_rows = torch.zeros(R, REC.row_bytes, dtype=torch.uint8, device="cuda")
        self.slots = torch.zeros(R, TOP_K, dtype=torch.int32, device="cuda")
        self.out = torch.zeros(R, 1, HEADS, REC.v_dim, dtype=torch.bfloat16, device="cuda")
        self.worst = 0.0

    def resident_rows(self, layer):
        return self.pool.store[layer].view(-1, REC.row_bytes)

    def prefill(self, request):
        """The prompt's records of every layer into the host pool, and its first pages into HBM."""
        r = torch.tensor([request], dtype=torch.int32, device="cuda")
        zero = torch.zeros(1, dtype=torch.int32, device="cuda")
        held = RESIDENT * PAGE - PAGE // 2     # the last page is part-filled
        self.pool.grow(r, torch.full_like(r, RESIDENT))
        rows = torch.zeros(PROMPT, REC.row_bytes, dtype=torch.uint8, device="cuda")
        for l in range(LAYERS):
            k = (self.prompt @ self.w_k[l]).view(PROMPT, 1, REC.k_dim)
            kw = dict(reqs=r, max_len=PROMPT, turns=self.turns, rot_offset=REC.k_dim - ROT,
                      amplitude=self.amplitude, status=self.status)
            cache8.pack(REC, k, None, rows, self.scales[l], zero, **kw)
            # the pages hold the same bytes: whole blocks of the same tokens have the same scales
            cache8.pack(REC, k, None, self.resident_rows(l), self.scales[l], zero,
                        blocks=self.pool.tables, page_tokens=PAGE, **kw)
            self.mem.host_view(l)[request, :PROMPT] = rows.cpu().numpy()
            self.index[l, request, :PROMPT] = (self.prompt @ self.w_i[l]).float()
        # The part-filled page is not looked up by its second half: those rows come from the host pool.
        self.held = held

    def fork(self, src, dst):
        """Request dst continues from src's prompt: resident pages shared, host rows copied."""
        i32 = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")   # noqa: E731
        self.pool.fork(i32(src), i32(dst), i32(self.held))
        for l in range(LAYERS):
            host = self.mem.host_view(l)
            host[dst, :PROMPT] = host[src, :PROMPT]
        self.scales[:, dst] = self.scales[:, src]
        self.index[:, dst] = self.index[:, src]

    def tables(self):
        """The resident table with the part-filled page left out (RESOLVE takes whole blocks)."""
        t = self.pool.tables.clone()
        t[:, RESIDENT - 1:] = -1
        return t

    def step(self, x, position, table, check=False):
        """One token of every request through all layers; x [R][DIM] is replaced."""
        pos = torch.full((R,), position, dtype=torch.int32, device="cuda")
        before = pos - 1 if position > PROMPT else torch.full_like(pos, -1)
        for l in range(LAYERS):
            x_n = torch.nn.functional.rms_norm(x, (DIM,))
            q = (x_n @ self.w_q[l]).view(R, HEADS, REC.k_dim)
            k = (x_n @ self.w_k[l]).view(R, 1, REC.k_dim)
            cache8.rotate(q, pos, self.turns, offset=REC.k_dim - ROT, amplitude=self.amplitude)
            cache8.pack(REC, k, None, self.new_rows, self.scales[l], pos, turns=self.turns,
                        rot_offset=REC.k_dim - ROT, amplitude=self.amplitude, status=self.status)
            key = x_n @ self.w_i[l]
            self.index[l, :, position] = key.float()
            score = torch.einsum("rd,rpd->rp", key.float(), self.index[l, :, :position + 1])
            score[:, position] = float("inf")                                   # the token itself
            sel = score.topk(TOP_K, dim=1).indices.to(torch.int32)
            self.hs.resolve_resident(l, sel, self.slots, table, PAGE, newest=pos, prev_pos=before,
                                     new_rows=self.new_rows)
            cache8.attend(REC, q.view(R, 1, HEADS, REC.k_dim), sel, self.slots, self.mem.hot[l],
                          self.scales[l], self.out, resident=self.resident_rows(l), status=self.status)
            if check:
                self.worst = max(self.worst, self.error(l, q, sel, position))
            x = x + self.out.view(R, -1) @ self.w_o[l]
        return x

    def error(self, layer, q, sel, position):
        """The largest error of ``out`` against 64 bits from the host pool's rows, over its bound: the
        output's rounding and 2^-7 of what the probabilities weigh."""
        torch.cuda.synchronize()
        host, sel = self.mem.host_view(layer), sel.cpu().numpy()
        worst = 0.0
        for r in range(R - 1):
            rows = host[r][sel[r]].copy()
            rows[sel[r] == position] = self.new_rows[r].cpu().numpy()
            k = torch.from_numpy(rows).view(torch.float8_e4m3fn).double().numpy()
            s = self.scales[layer, r, :, 0].double().cpu().numpy()
            k = k * s[sel[r] // REC.block_tokens][:, None]
            logits = q[r].double().cpu().numpy() @ k.T * REC.k_dim ** -0.5
            p = np.exp(logits - logits.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            v = k[:, :REC.v_dim]
            want, bound = p @ v, 2.0 ** -7 * (p @ np.abs(v))
            got = self.out[r, 0].double().cpu().numpy()
            worst = max(worst, (np.abs(got - want) / (bound + 2.0 ** -8 * np.abs(want))).max())
        return worst


def run(steps=8, check=False, seed=0):
    """Returns (worst error over its bound, milliseconds a step, the model)."""
    m = Model(steps, seed)
    m.prefill(0)
    m.fork(0, 1)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    x = torch.randn(R, DIM, device="cuda", generator=g).bfloat16()
    table = m.tables()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for t in range(steps):
        if t == 1:
            start.record()
        x = m.step(x, PROMPT + t, table, check)
    end.record()
    torch.cuda.synchronize()
    ms = start.elapsed_time(end) / max(1, steps - 1) if steps > 1 else 0.0
    # the first request is done; its pages that the other shares stay
    m.pool.free(torch.tensor([0], dtype=torch.int32, device="cuda"))
    m.pool.compact()
    flags, _ = m.hs.status()
    if flags or int(m.status):
        raise RuntimeError(f"device-side errors: resolve {flags:#x}, operators {int(m.status):#x}")
    return m.worst, ms, m


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--check", action="store_true", help="compare every output with 64 bits")
    o = ap.parse_args()
    worst, ms, m = run(o.steps, o.check)
    used = int((m.pool.refs > 0).sum())
    print(f"{o.steps} steps of {R - 1} requests and {LAYERS} layers, {ms:.2f} ms a step"
          + (f", worst error {worst:.2f} of its bound" if o.check else "")
          + f"; {used} resident pages in use after one request left")
    m.hs.close()
    m.mem.close()


if __name__ == "__main__":
    main()
