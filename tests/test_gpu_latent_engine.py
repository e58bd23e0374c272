"""The latent operators together, as a serving program uses them: the serving
loop over a latent cache against a 64-bit replay of every request's own
history, and a chunk's attention taken in both forms."""
import numpy as np
import pytest
import torch

from paged_kv_cache_143_gb300 import pa
from paged_kv_cache_143_gb300.engine import LatentEngine
from tests import latent_reference as ref

pytestmark = pytest.mark.gpu


def i32(a, dev):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=dev)


@pytest.mark.parametrize("fp8,interleaved", [(False, True), (True, False)], ids=["bf16", "e4m3"])
def test_latent_engine_steps(cuda_device, fp8, interleaved):
    """Prompts in chunks, decodes, shared prefixes, forks with copy-on-write
    and preemption. The rows of a token are a function of its request's tokens
    up to it, as a model's are, so a replay from the tokens alone says what
    every cell must hold."""
    dev, H, L, B, NB = cuda_device, 6, 256, 16, 96
    max_reqs, max_blocks, max_tokens = 12, 24, 200
    rng = np.random.default_rng(21)
    pool = ref.new_pool(pa, NB, B, L, fp8, dev)
    sched = pa.Scheduler(NB, B, max_reqs, max_blocks, token_budget=160, chunk_cap=64,
                         prefix_caching=True)
    freq, factor = pa.rope_frequencies(64, scaling="by_parts", stretch=2.0)
    scale = 192 ** -0.5
    eng = LatentEngine(sched, pool, H, max_reqs, max_blocks, max_tokens, scale, inv_freq=freq,
                       interleaved=interleaved, factor=factor)
    memo = {}

    def rows(prefix):
        """(query, latent, rotary key) of the last token of a token sequence."""
        key = hash(tuple(prefix))
        if key not in memo:
            g = np.random.default_rng(key & 0xFFFFFFFF)
            memo[key] = [torch.from_numpy(g.standard_normal(s)).bfloat16()
                         for s in ((H, L + 64), (L,), (64,))]
        return memo[key]

    tokens, rid, forked, checked = {}, 0, set(), 0
    common = rng.integers(0, 1000, 2 * B + 7).tolist()
    for step in range(36):
        if step < 14 and rng.random() < 0.7:
            p = (common if rng.random() < 0.5 else []) + rng.integers(
                0, 1000, int(rng.integers(1, 90))).tolist()
            sched.add_request(rid, p, int(rng.integers(2, 30)))
            tokens[rid] = p
            rid += 1
        # the engine schedules inside step(), and its rows depend on what it
        # schedules: the batch's rows are filled in by the hook below
        q = torch.zeros((max_tokens, H, L + 64), dtype=torch.bfloat16, device=dev)
        c = torch.zeros((max_tokens, L), dtype=torch.bfloat16, device=dev)
        kr = torch.zeros((max_tokens, 64), dtype=torch.bfloat16, device=dev)
        out = torch.full((max_tokens, H, L), 7.0, dtype=torch.bfloat16, device=dev)
        real = sched.step

        def scheduled():
            b = real()
            for i, r in enumerate(b.req_ids.tolist()):
                a, n, end = b.query_start_loc[i], b.num_scheduled[i], b.seq_lens[i]
                for t in range(n):
                    x = rows(tokens[r][:end - n + t + 1])
                    for dst, src in zip((q, c, kr), x):
                        dst[a + t] = src.to(dev)
            return b

        sched.step = scheduled
        b = eng.step(q, c, kr, out)
        sched.step = real
        eng.sync()
        assert pa.get_error() == pa.PA_OK
        R, T = b.num_reqs, b.num_tokens
        assert (out[T:] == 7).all()
        for i, r in enumerate(b.req_ids.tolist()):
            n, end = int(b.num_scheduled[i]), int(b.seq_lens[i])
            hist = [rows(tokens[r][:t + 1]) for t in range(end)]
            lat = np.stack([ref.f64(x[1]) for x in hist])
            if fp8:
                lat, s = ref.quantise(lat)
            krr = np.stack([ref.f64(x[2]) for x in hist])[:, None]
            pos = np.arange(end)
            k64 = ref.turn(krr, pos, freq.numpy(), interleaved, factor)[:, 0]
            qq = np.stack([ref.f64(x[0]) for x in hist[end - n:]])
            qt = qq.copy()
            qt[..., L:] = ref.turn(qq[..., L:], pos[end - n:], freq.numpy(), interleaved, factor)
            want, p = ref.absorbed(qt, lat, k64, scale)
            # the turned halves are rounded to bf16 (half a step each, and the turn's
            # fp32 work): a score is off by that of q and of k in 64 products
            d = ref.BF16_HALF * 1.01
            s_err = scale * 2 * d * np.einsum("thd,nd->thn", np.abs(qt[..., L:]),
                                              np.abs(k64)).max(-1)[..., None]
            s_mag = scale * np.einsum("thd,nd->thn", np.abs(qt), np.abs(
                np.concatenate((lat, k64), -1))).max(-1)[..., None]
            size = np.einsum("thn,nl->thl", p, np.abs(lat))
            tol = size * (ref.BF16_HALF + 2 * s_err + 2 * 2.0 ** -16 * s_mag) \
                + ref.BF16_HALF * np.abs(want) + 1e-6
            a = int(b.query_start_loc[i])
            err = np.abs(ref.f64(out[a:a + n]) - want)
            assert (err <= tol).all(), (step, r, (err / tol).max())
            assert torch.equal(eng.last_out[i].view(torch.int16),
                               out[a + n - 1].cpu().view(torch.int16))
            checked += n
        # what was generated so far, then the step's samples
        sampled = rng.integers(0, 1000, R).tolist()
        for i, r in enumerate(b.req_ids.tolist()):
            if int(b.seq_lens[i]) == len(tokens[r]):
                tokens[r] = tokens[r] + [sampled[i]]
        sched.commit(sampled)
        if step in (9, 15):
            for r in b.req_ids[:2].tolist():
                if r not in forked and sched.stats()["running"] < max_reqs:
                    try:
                        sched.fork(r, 1000 + rid, 6)
                        tokens[1000 + rid] = list(tokens[r])
                        forked.add(r)
                        rid += 1
                    except pa.PaError:
                        pass
    st = sched.stats()
    assert checked > 500 and st["prefix_hit_tokens"] > 0 and forked


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_both_forms_of_a_chunk_agree(cuda_device, fp8):
    """A chunk behind a cached context: stored, then attended to straight on
    the cache, and through rows read back and expanded with the layer's
    matrices. Both against the 64-bit layer on the cells' own values."""
    dev, H, L, B = cuda_device, 4, 512, 32
    rng = np.random.default_rng(31)
    past, chunk = [150, 0, 64], [60, 130, 1]
    seqs = [a + b for a, b in zip(past, chunk)]
    tab, blocks = ref.tables(rng, seqs, B)
    pool = ref.new_pool(pa, blocks, B, L, fp8, dev)
    freq = pa.rope_frequencies(64, device=dev)[0]

    def rand(*shape, m=1.0):
        return torch.from_numpy(rng.standard_normal(shape) * m).to(dev).bfloat16()

    n = sum(seqs)
    c, kr = rand(n, L), rand(n, 64)
    pos = torch.cat([torch.arange(s) for s in seqs]).int().to(dev)
    slots = torch.from_numpy(np.concatenate(
        [ref.slots_of(tab, r, s, B) for r, s in enumerate(seqs)])).to(dev)
    pa.write_latent(pool, c, kr, slots, positions=pos, inv_freq=freq, interleaved=True)
    wk, wv = rand(H, 128, L, m=L ** -0.5), rand(H, 128, L, m=L ** -0.5)
    T = sum(chunk)
    qsl = np.cumsum([0] + chunk).astype(np.int32)
    ksl = np.cumsum([0] + seqs).astype(np.int32)
    q = rand(T, H, 192)
    qpos = torch.cat([torch.arange(s - k, s) for s, k in zip(seqs, chunk)]).int().to(dev)
    pa.rope(q[..., 128:], q[..., 128:], qpos, freq, interleaved=True)
    scale = 192 ** -0.5

    # expanded: the context's rows read back, one product for keys and values
    lat = torch.empty(n, L, dtype=torch.bfloat16, device=dev)
    rot = torch.empty(n, 64, dtype=torch.bfloat16, device=dev)
    pa.read_latent(pool, i32(tab, dev), i32(ksl, dev), lat, rot)
    w = torch.cat((wk, wv), 1).reshape(H * 256, L)
    kv = (lat @ w.T).view(n, H, 256)
    exp = torch.empty(T, H, 128, dtype=torch.bfloat16, device=dev)
    pa.latent_prefill(q, kv[..., :128], rot, kv[..., 128:], exp, i32(qsl, dev), i32(ksl, dev), qsl,
                      ksl, scale)
    # absorbed: W_k into the query, W_v behind the output
    qa = torch.empty(T, H, L + 64, dtype=torch.bfloat16, device=dev)
    qa[..., :L] = torch.einsum("thd,hdl->thl", q[..., :128].float(), wk.float())
    qa[..., L:] = q[..., 128:]
    o = torch.empty(T, H, L, dtype=torch.bfloat16, device=dev)
    ws = torch.empty(pa.latent_workspace_size(H, L), dtype=torch.uint8, device=dev)
    pa.latent_forward(qa, o, i32(qsl, dev), i32(seqs, dev), qsl, np.array(seqs, np.int32),
                      i32(tab, dev), pool, scale, workspace=ws)
    absd = torch.einsum("thl,hdl->thd", o.float(), wv.float())
    assert pa.get_error() == pa.PA_OK

    cells, rots = ref.pool_rows(pool)
    d = ref.BF16_HALF
    for r, s in enumerate(seqs):
        at = ref.slots_of(tab, r, s, B)
        a, b = qsl[r], qsl[r + 1]
        k64 = np.einsum("hdl,nl->nhd", ref.f64(wk), cells[at])
        v64 = np.einsum("hdl,nl->nhd", ref.f64(wv), cells[at])
        q64 = ref.f64(q[a:b])
        want, p = ref.expanded(q64, k64, rots[at], v64, scale)
        # expanded: k and v rounded to bf16 (and their products' fp32 sums), then
        # the attention's own roundings; absorbed: the query rounded, then those
        # of the output over 512 products with W_v
        ks = scale * np.einsum("thd,nhd->thn", np.abs(q64[..., :128]), np.abs(k64)).max(-1)
        size = np.einsum("thn,nhd->thd", p, np.abs(v64))
        tol = size * (3 * d + 2 * 1.1 * d * ks[..., None]) + d * np.abs(want) + 1e-3
        err = np.abs(ref.f64(exp[a:b]) - want)
        assert (err <= tol).all(), (r, (err / tol).max())
        qn = np.einsum("thd,hdl->thl", q64[..., :128], ref.f64(wk))
        qs = scale * np.einsum("thl,nl->thn", np.abs(qn), np.abs(cells[at])).max(-1)
        osize = np.einsum("thn,nl->thl", p, np.abs(cells[at]))
        osize = np.einsum("thl,hdl->thd", osize, np.abs(ref.f64(wv)))
        tol = osize * (2 * d + 2 * 1.1 * d * qs[..., None]) + 1e-3
        err = np.abs(ref.f64(absd[a:b]) - want)
        assert (err <= tol).all(), (r, (err / tol).max())
        # and the two agree far closer than the bounds on either
        gap = np.abs(ref.f64(absd[a:b]) - ref.f64(exp[a:b]))
        assert gap.max() < 0.03 * np.abs(want).max() + 0.01
