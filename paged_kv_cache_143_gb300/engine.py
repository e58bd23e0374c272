"""Multi-step serving loop over the native scheduler and the device calls.

Each step: the native scheduler (pa_sched_step) decides the batch; the host
packs what the device needs into one pinned buffer and sends it with one
copy; then, on the stream,
  pa_apply_staged_writes  on the per-slot stored-token counts (slots whose
                          count the device does not hold: admissions,
                          resumed or forked requests) and on the block table
                          (the step's diffs, then the gather by idx_mapping),
  pa_copy_blocks          the step's copy-on-write pairs,
  pa_prepare_inputs       query_start_loc, seq_lens, positions, slot mapping,
  pa_write_kv             the step's new K/V,
  pa_forward              attention for every entry,
  pa_gather_rows          the output row of each entry's last token,
and those rows are read back into one of two pinned host buffers.

[MRV2 "재설계 1"] persistent slots and idx_mapping; [MRV2 "재설계 2"] the
host never modifies a buffer the device may still be reading: two pinned
staging buffers alternate, each reused only after the copy that read it has
completed; [MRV2 "재설계 3"] only diffs go to the device table; [MRV2
"재설계 4"] the inputs are prepared on the device.

There is no model: the caller provides the step's Q/K/V rows (token t of the
batch is row t) and the sampled tokens.

LatentEngine runs the same loop over a latent cache: pa_copy_latent_blocks,
pa_write_latent (which turns the rotary keys by the positions that
pa_prepare_inputs made) and, for the queries, pa_rope and pa_latent_forward
take the places of the calls on keys and values. SparseEngine runs it with
attention to a part of each context: pa_update_block_bounds, pa_score_blocks,
pa_select_blocks and pa_sparse_forward in the place of pa_forward.
"""
from typing import Optional

import numpy as np
import torch

from . import pa


class Engine:
    def __init__(self, sched: "pa.Scheduler", pool: "pa.KVPool", num_q_heads: int, max_reqs: int,
                 max_blocks: int, max_tokens: int, scale: float, max_splits: int = 32,
                 device=None):
        self.sched, self.pool = sched, pool
        self.B, self.Hq, self.D = pool.block_size, num_q_heads, self._out_dim(pool)
        self.max_reqs, self.max_blocks, self.max_tokens = max_reqs, max_blocks, max_tokens
        self.scale = scale
        dev = torch.device("cuda") if device is None else torch.device(device)
        self.dev = dev
        i32 = dict(dtype=torch.int32, device=dev)
        self.table = torch.full((max_reqs, max_blocks), -1, **i32)
        self.gathered = torch.full((max_reqs, max_blocks), -1, **i32)
        self.num_computed = torch.zeros((max_reqs, 1), **i32)
        self.qsl = torch.zeros(max_reqs + 1, **i32)
        self.seq = torch.zeros(max_reqs, **i32)
        self.pos = torch.zeros(max_tokens, **i32)
        self.slots = torch.zeros(max_tokens, dtype=torch.int64, device=dev)
        # staging: the largest step payload (ints)
        self.cap = 6 * max_reqs + 2 * max_reqs * max_blocks + 4 * max_reqs + 16
        self.host = [torch.zeros(self.cap, dtype=torch.int32).pin_memory() for _ in range(2)]
        self.host_np = [h.numpy() for h in self.host]
        self.done = [torch.cuda.Event(), torch.cuda.Event()]
        self.used = [False, False]
        self.dstage = torch.zeros(self.cap, **i32)
        n = self._workspace_bytes(max_splits)
        self.ws = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
        self.mirror = np.full(max_reqs, -1, np.int64)  # stored-token count the device holds
        # each entry's last output row: gathered on the device, read back into
        # one of two pinned buffers (a step's rows stay valid through the next step)
        self.last_dev = torch.empty((max_reqs, num_q_heads, self.D), dtype=torch.bfloat16,
                                    device=dev)
        self.last_host = [torch.empty((max_reqs, num_q_heads, self.D),
                                      dtype=torch.bfloat16).pin_memory() for _ in range(2)]
        self.last_turn = 0
        self.last_out = None
        self.turn = 0
        self.steps = 0
        self.h2d_bytes = 0
        self.d2h_bytes = 0

    # what a cache of another kind does otherwise
    @staticmethod
    def _out_dim(pool) -> int:
        return pool.head_dim

    def _workspace_bytes(self, max_splits: int) -> int:
        return pa.forward_workspace_size(self.max_reqs, self.Hq, self.D, max_splits)

    def _copy_blocks(self, src: torch.Tensor, dst: torch.Tensor, s) -> None:
        pa.copy_blocks(self.pool, src, dst, stream=s)

    def _store(self, k: torch.Tensor, v: torch.Tensor, T: int, s) -> None:
        pa.write_kv(self.pool, k[:T], v[:T], self.slots[:T], stream=s)

    def _attend(self, q: torch.Tensor, out: torch.Tensor, b: "pa.SchedBatch", R: int, T: int,
                s) -> None:
        pa.forward(q[:T], out[:T], self.qsl[:R + 1], self.seq[:R], b.query_start_loc, b.seq_lens,
                   self.gathered[:R], self.pool, self.scale, 1, workspace=self.ws, stream=s)

    def step(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
             stream=None) -> "pa.SchedBatch":
        """Runs one step; q/k/v/out hold at least the step's tokens as rows.
        Returns the scheduled batch; the output rows of each entry's last
        token are in `last_out` (host, pinned) once the step's stream has
        reached the end of the step (the next `step` or `sync` waits); they
        stay valid through the next step (two buffers alternate)."""
        b = self.sched.step()
        R, T = b.num_reqs, b.num_tokens
        if T > self.max_tokens or R > self.max_reqs:
            raise ValueError("batch larger than the engine's buffers")
        s = torch.cuda.current_stream() if stream is None else stream
        # slots whose stored-token count the device does not hold
        start = (b.seq_lens - b.num_scheduled).astype(np.int64)
        stale = np.nonzero(self.mirror[b.idx_mapping] != start)[0]
        W, C, S = b.diff_rows.size, b.copy_src.size, stale.size
        NV = int(b.diff_val_offsets[-1])
        parts = [b.idx_mapping, b.num_scheduled, b.diff_rows, b.diff_starts, b.diff_val_offsets,
                 b.diff_vals, b.idx_mapping[stale], np.zeros(S, np.int32),
                 np.arange(S + 1, dtype=np.int32), start[stale].astype(np.int32), b.copy_src,
                 b.copy_dst, (b.query_start_loc[1:] - 1).astype(np.int32)]
        total = sum(p.size for p in parts)
        if total > self.cap:
            raise ValueError("step payload larger than the staging buffer")
        i = self.turn
        if self.used[i]:
            self.done[i].synchronize()  # the copy that last read this buffer is over
        h = self.host_np[i]
        offs = [0]
        for p in parts:
            h[offs[-1]:offs[-1] + p.size] = p
            offs.append(offs[-1] + p.size)
        with torch.cuda.stream(s):
            self.dstage[:total].copy_(self.host[i][:total], non_blocking=True)
            self.done[i].record(s)
            self.used[i] = True
            self.turn ^= 1
            d = [self.dstage[offs[j]:offs[j + 1]] for j in range(len(parts))]
            idx, cnt = d[0], d[1]
            if S:
                pa.apply_staged_writes(self.num_computed, d[6], d[7], d[8], d[9],
                                       idx[:0], self.gathered[:0], stream=s)
            pa.apply_staged_writes(self.table, d[2], d[3], d[4], d[5], idx,
                                   self.gathered[:R], stream=s)
            if C:
                self._copy_blocks(d[10], d[11], s)
            pa.prepare_inputs(self.num_computed, self.table, self.B, self.pool.num_blocks, idx,
                              cnt, self.qsl[:R + 1], self.seq[:R], self.pos[:T],
                              self.slots[:T], stream=s)
            self._store(k, v, T, s)
            self._attend(q, out, b, R, T, s)
            host = self.last_host[self.last_turn][:R]
            if R:
                pa.gather_rows(out, d[12], self.last_dev[:R], stream=s)
                host.copy_(self.last_dev[:R], non_blocking=True)
            self.last_out = host
            self.last_turn ^= 1
        self.mirror[b.idx_mapping] = b.seq_lens
        self.h2d_bytes += 4 * total
        self.d2h_bytes += host.numel() * host.element_size()
        self.steps += 1
        self.stream = s
        return b

    def sync(self) -> None:
        self.stream.synchronize()


class LatentEngine(Engine):
    """The serving loop over a latent cache (pa.LatentPool): step(q, latent,
    k_rope, out) with q [T][Hq][L + 64] (the absorbed query, then its rotary
    part), latent [T][L], k_rope [T][64] and out [T][Hq][L].

    With inv_freq (and interleaved, factor, as pa.rope takes them) the rotary
    parts come unturned: the keys' are turned as they are stored, the queries'
    in place in q. Without, the caller has turned both."""

    def __init__(self, sched: "pa.Scheduler", pool: "pa.LatentPool", num_q_heads: int,
                 max_reqs: int, max_blocks: int, max_tokens: int, scale: float,
                 inv_freq: Optional[torch.Tensor] = None, interleaved: bool = False,
                 factor: float = 1.0, device=None):
        super().__init__(sched, pool, num_q_heads, max_reqs, max_blocks, max_tokens, scale,
                         device=device)
        self.inv_freq = None if inv_freq is None else inv_freq.to(self.dev)
        self.interleaved, self.factor = interleaved, factor

    @staticmethod
    def _out_dim(pool) -> int:
        return pool.latent_dim

    def _workspace_bytes(self, max_splits: int) -> int:
        return pa.latent_workspace_size(self.Hq, self.D)

    def _copy_blocks(self, src: torch.Tensor, dst: torch.Tensor, s) -> None:
        pa.copy_latent_blocks(self.pool, src, dst, stream=s)

    def _store(self, latent: torch.Tensor, k_rope: torch.Tensor, T: int, s) -> None:
        turn = {} if self.inv_freq is None else dict(
            positions=self.pos[:T], inv_freq=self.inv_freq, interleaved=self.interleaved,
            factor=self.factor)
        pa.write_latent(self.pool, latent[:T], k_rope[:T], self.slots[:T], stream=s, **turn)

    def _attend(self, q: torch.Tensor, out: torch.Tensor, b: "pa.SchedBatch", R: int, T: int,
                s) -> None:
        if self.inv_freq is not None:
            part = q[:T, :, self.D:]
            pa.rope(part, part, self.pos[:T], self.inv_freq, interleaved=self.interleaved,
                    factor=self.factor, stream=s)
        pa.latent_forward(q[:T], out[:T], self.qsl[:R + 1], self.seq[:R], b.query_start_loc,
                          b.seq_lens, self.gathered[:R], self.pool, self.scale, 1,
                          workspace=self.ws, stream=s)


class SparseEngine(Engine):
    """The serving loop with attention to a part of each context: every token's
    heads attend to `num_selected` blocks of their kv head, chosen by the bounds
    of the blocks' keys (pa_score_blocks) with the first `first` and the newest
    `last` among them. Contexts of no more blocks than that are attended to
    whole, as Engine does (a token at a time: long chunks on short contexts are
    Engine's work). Keeps the scores of max_tokens tokens for all of max_blocks:
    4 * max_tokens * num_kv_heads * max_blocks bytes."""

    def __init__(self, sched: "pa.Scheduler", pool: "pa.KVPool", num_q_heads: int, max_reqs: int,
                 max_blocks: int, max_tokens: int, scale: float, num_selected: int,
                 first: int = 1, last: int = 2, device=None):
        super().__init__(sched, pool, num_q_heads, max_reqs, max_blocks, max_tokens, scale,
                         device=device)
        if first < 0 or last < 0 or not 1 <= num_selected >= first + last:
            raise ValueError("num_selected must be positive and hold the first and last blocks")
        self.first, self.last = first, last
        H = pool.num_kv_heads
        self.bounds = torch.zeros((pool.num_blocks, H, 2, pool.head_dim), dtype=torch.bfloat16,
                                  device=self.dev)
        self.scores = torch.empty((max_tokens, H, max_blocks), dtype=torch.float32,
                                  device=self.dev)
        self.selected = torch.empty((max_tokens, H, num_selected), dtype=torch.int32,
                                    device=self.dev)

    def _workspace_bytes(self, max_splits: int) -> int:
        return 0

    def _attend(self, q: torch.Tensor, out: torch.Tensor, b: "pa.SchedBatch", R: int, T: int,
                s) -> None:
        qsl, seq, tab = self.qsl[:R + 1], self.seq[:R], self.gathered[:R]
        # a block that was copied on write is written to in the same step, so the bounds of
        # every block that a request reads are those of its keys
        pa.update_block_bounds(self.pool, self.bounds, tab, seq, query_start_loc=qsl,
                               num_tokens=T, stream=s)
        pa.score_blocks(q[:T], self.bounds, self.scores[:T], qsl, seq, tab, self.pool, stream=s)
        pa.select_blocks(self.scores[:T], self.selected[:T], qsl, seq, self.B, first=self.first,
                         last=self.last, stream=s)
        pa.sparse_forward(q[:T], out[:T], qsl, seq, tab, self.selected[:T], self.pool, self.scale,
                          stream=s)
