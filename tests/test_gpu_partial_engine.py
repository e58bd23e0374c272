"""The calls that attend to a part of a cache together, as a serving program uses
them: the serving loop with selected blocks, and decodes whose cache is cut down
by the attention that its tokens received, both against 64-bit replays."""
import numpy as np
import pytest
import torch

from oracle import oracle as O
from paged_kv_cache_143_gb300 import pa
from paged_kv_cache_143_gb300.engine import SparseEngine
from tests import partial_reference as ref
from tests.helpers import bits
from tests.test_gpu_partial_attention import check
from tests.test_gpu_partial_select import i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_sparse_engine_steps(cuda_device, fp8):
    """Prompts in chunks, decodes, shared prefixes, forks with copy-on-write. Bounds
    are exact; what was selected is what the 64-bit scores select, up to scores
    closer than fp32 tells apart; attention is that of the selected blocks."""
    dev, Hq, Hkv, D, B, NB, K = cuda_device, 4, 2, 64, 16, 160, 4
    max_reqs, max_blocks, max_tokens = 10, 24, 160
    rng = np.random.default_rng(41)
    gen = torch.Generator(device=dev)
    gen.manual_seed(41)
    if fp8:
        half = lambda: torch.full((NB, Hkv, B, D), 0x7F, dtype=torch.uint8, device=dev)
        scales = (1 / 64.0, 1 / 32.0)
    else:
        half = lambda: torch.full((NB, Hkv, B, D), float("nan"), dtype=torch.bfloat16, device=dev)
        scales = (1.0, 1.0)
    pool = pa.KVPool(half(), half(), *scales)
    opool = O.Pool(bits(pool.k).copy(), bits(pool.v).copy(), B, O.FP8_E4M3 if fp8 else O.BF16, *scales)
    sched = pa.Scheduler(NB, B, max_reqs, max_blocks, token_budget=128, chunk_cap=64,
                         prefix_caching=True)
    eng = SparseEngine(sched, pool, Hq, max_reqs, max_blocks, max_tokens, D ** -0.5, K, first=1,
                       last=1)
    common = rng.integers(0, 1000, size=2 * B + 5).tolist()
    rid, forked, left_out = 0, set(), 0
    for step in range(30):
        if step < 12 and rng.random() < 0.7:
            p = (common if rng.random() < 0.5 else []) + rng.integers(
                0, 1000, size=int(rng.integers(1, 130))).tolist()
            sched.add_request(rid, p, int(rng.integers(2, 25)))
            rid += 1
        q, out = (torch.randn((max_tokens, Hq, D), generator=gen, device=dev).bfloat16()
                  for _ in range(2))
        k, v = (torch.randn((max_tokens, Hkv, D), generator=gen, device=dev).bfloat16()
                for _ in range(2))
        was = out.clone()
        b = eng.step(q, k, v, out)
        eng.sync()
        assert pa.get_error() == pa.PA_OK
        R, T = b.num_reqs, b.num_tokens
        if R == 0:
            sched.commit([])
            continue
        O.copy_blocks(opool, b.copy_src, b.copy_dst)
        O.write_kv(opool, bits(k[:T]), bits(v[:T]), b.slot_mapping)
        assert np.array_equal(bits(pool.k), opool.k) and np.array_equal(bits(pool.v), opool.v)
        table = [sched.table(int(r)) for r in b.req_ids]
        qsl, seqs = b.query_start_loc.tolist(), b.seq_lens.tolist()
        kk, vv, qq = ref.cells(pool.k), ref.cells(pool.v), ref.f64(q[:T])
        bnd = ref.f64(eng.bounds)
        # every block that a request reads, whichever step made its bounds
        assert np.array_equal(bnd, ref.bounds(kk, table, None, seqs, B, bnd.copy()))
        s64, tol = ref.scores(qq, bnd, table, qsl, seqs, B, Hq // Hkv, scales[0],
                              np.zeros((T, Hkv, max_blocks)))
        sel = eng.selected[:T].cpu().numpy()
        for r, t, p in ref.rows_of(qsl, seqs):
            n = p // B + 1
            for h in range(Hkv):
                mine = sel[t, h][sel[t, h] >= 0]
                assert len(mine) == min(n, K) and (np.diff(mine) > 0).all()
                others = np.setdiff1d(np.arange(n), mine)
                left_out += len(others)
                if len(others):
                    assert 0 in mine and n - 1 in mine
                    chosen = np.setdiff1d(mine, [0, n - 1])
                    e = 2 * tol[t, h, :n].max()
                    assert s64[t, h, chosen].min() >= s64[t, h, others].max() - e
        check(ref.f64(out[:T]), *ref.sparse(qq, kk, vv, table, sel, qsl, seqs, B, Hq // Hkv,
                                            D ** -0.5, scales[0], scales[1], fp8))
        assert torch.equal(out[T:], was[T:])
        sched.commit(rng.integers(0, 1000, size=R).tolist())
        if step in (9, 14):
            for r in b.req_ids[:2].tolist():
                if r not in forked and sched.stats()["running"] < max_reqs:
                    try:
                        sched.fork(r, 1000 + rid, 6)
                        forked.add(r)
                        rid += 1
                    except pa.PaError:
                        pass
    st = sched.stats()
    assert left_out > 500 and st["prefix_hit_tokens"] > 0 and forked


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_decodes_with_an_evicted_cache(cuda_device, fp8):
    """Prompts, then decodes. Each step attends to what is stored and adds up what
    each token received; a request whose cache is full is cut down in place, its
    bounds made anew, and goes on, attending to selected blocks. The replay keeps
    each request's stored tokens as lists."""
    dev, Hq, Hkv, D, B = cuda_device, 8, 2, 128, 16
    rng = np.random.default_rng(43)
    R, full, keep = 3, 96, 40
    blocks = R * (full // B)
    shape = (blocks, Hkv, B, D)
    pool = pa.KVPool(*(torch.zeros(shape, dtype=torch.uint8 if fp8 else torch.bfloat16, device=dev)
                       for _ in range(2)), *((1 / 32.0, 1 / 32.0) if fp8 else (1.0, 1.0)))
    table = rng.permutation(blocks).reshape(R, -1)
    dtab = i32(table, dev)
    idx = [2, 0, 3]
    mass = torch.full((4, full), float("nan"), device=dev)
    bnd = torch.zeros((blocks, Hkv, 2, D), dtype=torch.bfloat16, device=dev)
    scale = D ** -0.5
    stored = [[] for _ in range(R)]       # (key, value) rows of each request, as the pool has them
    got = [np.zeros(0) for _ in range(R)]  # what each has received, in 64 bits
    off = [np.zeros(0) for _ in range(R)]  # and by how much the kernels may differ
    lens, cut = [70, 33, 90], 0

    def step(new):
        nonlocal lens
        qsl = np.cumsum([0] + new).astype(np.int32)
        seqs = np.array(lens, np.int32)
        T = int(qsl[-1])
        q = torch.from_numpy(rng.standard_normal((T, Hq, D)) * 1.5).to(dev).bfloat16()
        k, v = (torch.from_numpy(rng.standard_normal((T, Hkv, D))).to(dev).bfloat16()
                for _ in range(2))
        slots = [int(table[r, p // B]) * B + p % B for r, _, p in ref.rows_of(qsl, seqs)]
        pa.write_kv(pool, k, v, torch.tensor(slots, dtype=torch.int64, device=dev))
        dq, ds = i32(qsl, dev), i32(seqs, dev)
        pa.update_block_bounds(pool, bnd, dtab, ds, query_start_loc=dq, num_tokens=T)
        scores = torch.zeros((T, Hkv, full // B), device=dev)
        sel = torch.zeros((T, Hkv, 3), dtype=torch.int32, device=dev)
        out, part = torch.zeros_like(q), torch.zeros_like(q)
        pa.score_blocks(q, bnd, scores, dq, ds, dtab, pool)
        pa.select_blocks(scores, sel, dq, ds, B, first=1, last=1)
        pa.sparse_forward(q, part, dq, ds, dtab, sel, pool, scale)
        pa.forward(q, out, dq, ds, qsl, seqs, dtab, pool, scale)
        ws = torch.empty(pa.attention_mass_workspace_size(qsl, seqs, Hq, Hkv, 8),
                         dtype=torch.uint8, device=dev)
        pa.attention_mass(q, mass, mass, dq, ds, qsl, seqs, dtab, pool, scale,
                          idx_mapping=i32(idx, dev), decay=0.9, window=8, workspace=ws)
        assert pa.get_error() == pa.PA_OK
        kk, vv, qq = ref.cells(pool.k), ref.cells(pool.v), ref.f64(q)
        for r, _, p in ref.rows_of(qsl, seqs):
            stored[r].append((kk[table[r, p // B], :, p % B].copy(),
                              vv[table[r, p // B], :, p % B].copy()))
        # the pool holds the stored tokens, in order
        for r in range(R):
            assert len(stored[r]) == lens[r]
            for x, i in ((kk, 0), (vv, 1)):
                rows = np.concatenate([x[b].transpose(1, 0, 2) for b in table[r]])[:lens[r]]
                assert np.array_equal(rows, np.stack([s[i] for s in stored[r]]))
        everything = np.tile(np.arange(full // B), (T, Hkv, 1))
        for o, lists in ((out, everything), (part, sel.cpu().numpy())):
            check(ref.f64(o), *ref.sparse(qq, kk, vv, table, lists, qsl, seqs, B, Hq // Hkv, scale,
                                          pool.k_scale, pool.v_scale, fp8))
        want, tol = ref.mass(qq, kk, np.zeros((R, full)), range(R), table, qsl, seqs, B,
                             Hq // Hkv, scale, pool.k_scale, 0.0, 8, np.zeros((R, full)), fp8)
        m = mass.cpu().numpy()
        for r in range(R):
            n, was = lens[r], lens[r] - new[r]
            if new[r]:
                d = np.float64(np.float32(0.9))
                got[r] = want[r, :n] + np.concatenate((d * got[r], np.zeros(n - was)))
                off[r] = tol[r, :n] + np.concatenate((off[r], np.zeros(n - was))) \
                    + 2.0 ** -22 * got[r]
            assert (np.abs(m[idx[r], :n] - got[r]) <= off[r]).all()

    step(list(lens))
    for turn in range(150):
        new = [int(rng.random() < 0.9) for _ in range(R)]
        if max(new) == 0:
            continue
        lens = [a + b for a, b in zip(lens, new)]
        step(new)
        if max(lens) == full:  # all requests at once: those below `keep` stay as they are
            kept = torch.zeros((R, keep), dtype=torch.int32, device=dev)
            kept_lens = torch.zeros(R, dtype=torch.int32, device=dev)
            before = mass.cpu().numpy()
            pa.select_tokens(mass, kept, kept_lens, i32(lens, dev), idx_mapping=i32(idx, dev),
                             first=2, last=8)
            pa.compact_cache(pool, dtab, dtab, kept, kept_lens, mass_in=mass, mass_out=mass,
                             idx_mapping=i32(idx, dev))
            pa.update_block_bounds(pool, bnd, dtab, kept_lens)
            assert pa.get_error() == pa.PA_OK
            for r in range(R):
                mine = ref.pick(before[idx[r]], lens[r], 2, 8, keep)
                assert np.array_equal(kept[r].cpu().numpy(), mine)
                mine = mine[mine >= 0]
                cut += lens[r] - len(mine)
                stored[r] = [stored[r][i] for i in mine]
                got[r], off[r] = got[r][mine], off[r][mine]
            lens = kept_lens.tolist()
            assert np.array_equal(ref.f64(bnd), ref.bounds(ref.cells(pool.k), table, None, lens, B,
                                                           ref.f64(bnd)))
    assert cut > 100
