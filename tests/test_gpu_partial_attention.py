"""GPU tests of attention over listed blocks, attention mass and cache
compaction against 64-bit definitions."""
import numpy as np
import pytest
import torch

from paged_kv_cache_143_gb300 import pa
from tests import partial_reference as ref
from tests.test_gpu_partial_select import BATCHES, batch, i32, make_pool

pytestmark = pytest.mark.gpu


def stale(pool, table, seqs, B, fp8):
    """NaN in the cells past each request's tokens."""
    for r, n in enumerate(seqs):
        if n % B:
            for x in (pool.k, pool.v):
                x[int(table[r, n // B]), :, n % B:] = 0x7F if fp8 else float("nan")


def lists(rng, qsl, seqs, Hkv, B, k, N):
    """A list for each (token, kv head): some of the visible blocks in any order,
    with holes, now and then a block past the token."""
    out = np.full((int(qsl[-1]), Hkv, k), -1)
    for r, t, p in ref.rows_of(qsl, seqs):
        for h in range(Hkv):
            n = p // B + 1
            some = rng.permutation(n)[: rng.integers(1, k + 1)]
            at = rng.permutation(k)[: len(some)]
            out[t, h, at] = some
            free = np.nonzero(out[t, h] < 0)[0]
            if len(free) and n < N and rng.random() < 0.3:
                out[t, h, free[0]] = n  # not visible yet
    return out


def attend(dev, rng, seqs, new, Hq, Hkv, D, B, k, fp8, selected=None, spoil=None, extra_rows=0):
    table, qsl, blocks = batch(rng, seqs, new, B, dev, wide=1)
    pool = make_pool(rng, blocks, Hkv, B, D, fp8, dev)
    stale(pool, table, seqs, B, fp8)
    if selected is None:
        selected = lists(rng, qsl, seqs, Hkv, B, k, table.shape[1])
    T = int(qsl[-1]) + extra_rows
    sel = np.full((T, Hkv, k), 0)
    sel[: int(qsl[-1])] = selected
    q = torch.from_numpy(rng.standard_normal((T, Hq, D)) * 1.5).to(dev).bfloat16()
    if spoil:
        spoil(q, pool, table, sel)
    out = torch.full_like(q, 7.0)
    pa.sparse_forward(q, out, i32(qsl, dev), i32(seqs, dev), i32(table, dev), i32(sel, dev), pool,
                      D ** -0.5)
    want, tol = ref.sparse(ref.f64(q), ref.cells(pool.k), ref.cells(pool.v), table, sel, qsl, seqs,
                           B, Hq // Hkv, D ** -0.5, pool.k_scale, pool.v_scale, fp8)
    assert (out[int(qsl[-1]):] == 7).all()
    n = int(qsl[-1])
    return ref.f64(out)[:n], want[:n], tol[:n]


def check(got, want, tol):
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert (np.abs(got - want)[fine] <= tol[fine]).all(), np.nanmax((np.abs(got - want) - tol)[fine])


SHAPES = [  # Hq, Hkv, D, B, k
    (1, 1, 64, 16, 1), (8, 8, 128, 16, 5), (4, 2, 128, 32, 3), (6, 2, 64, 64, 4),
    (8, 1, 128, 16, 9), (10, 2, 128, 16, 40), (16, 1, 64, 32, 7), (9, 1, 128, 64, 2),
    (34, 2, 128, 16, 8), (40, 1, 64, 16, 130), (28, 4, 128, 16, 17),
]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("case", range(len(BATCHES)))
def test_sparse(cuda_device, case, shape, fp8):
    Hq, Hkv, D, B, k = shape
    rng = np.random.default_rng(case + Hq + D)
    check(*attend(cuda_device, rng, *BATCHES[case], Hq, Hkv, D, B, k, fp8, extra_rows=case % 3))
    assert pa.get_error() == pa.PA_OK


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_sparse_long_lists(cuda_device, fp8):
    """Few tokens with long lists, which clusters share, and many tokens."""
    rng = np.random.default_rng(5)
    check(*attend(cuda_device, rng, [5000], [1], 8, 1, 128, 16, 300, fp8))
    check(*attend(cuda_device, rng, [2500, 900], [1, 3], 4, 2, 64, 16, 64, fp8))
    check(*attend(cuda_device, rng, [900, 40], [400, 30], 8, 4, 64, 32, 6, fp8))


def test_sparse_rows_that_see_nothing(cuda_device):
    rng = np.random.default_rng(6)
    for k in (4, 200):  # one CTA a list, and a cluster
        sel = np.full((3, 1, k), -1)
        sel[1, 0, 2] = 5      # a block past the token
        sel[2, 0, k - 1] = 0
        got, want, tol = attend(cuda_device, rng, [40, 33], [2, 1], 4, 1, 64, 16, k, False,
                                selected=sel[:3])
        assert (got[:2] == 0).all() and (got[2] != 0).any()
        check(got, want, tol)


def test_sparse_block_named_twice(cuda_device):
    """Twice the weight, as the definition's sum has it."""
    rng = np.random.default_rng(7)
    sel = np.array([[[0, 2, 0, 2, 1, -1, 2]]])
    check(*attend(cuda_device, rng, [45], [1], 2, 1, 128, 16, 7, False, selected=sel))


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_sparse_numbers_that_are_not_finite(cuda_device, fp8):
    """NaN in a query, a key or a value reaches the rows that see it; scores of -inf
    weigh nothing; a row of nothing else is NaN."""
    def spoil(q, pool, table, sel):
        bad = 0x7F if fp8 else float("nan")
        q[0, 1, 3] = float("nan")
        pool.k[int(table[1, 0]), 0, 2, 5] = bad       # block 0 of request 1
        pool.v[int(table[2, 1]), 0, 1, 6] = bad       # block 1 of request 2
        if not fp8:  # a key at -inf for queries that are positive there
            q[4:, :, 9] = 1.0
            pool.k[int(table[3, 0]), 0, :, 9] = float("-inf")

    rng = np.random.default_rng(8)
    sel = np.array([[[0, 1, -1]], [[0, 1, -1]], [[1, -1, -1]], [[0, 1, -1]], [[0, 1, -1]],
                    [[0, -1, -1]], [[1, -1, -1]]])
    got, want, tol = attend(cuda_device, rng, [20, 30, 40, 30, 25, 20], [1, 2, 1, 2, 0, 1], 2, 1,
                            128, 16, 3, fp8, selected=sel, spoil=spoil)
    assert np.isnan(want).any() and np.isfinite(want).any()
    check(got, want, tol)


def test_sparse_refuses_what_leaves_the_buffers(cuda_device):
    dev = cuda_device
    rng = np.random.default_rng(13)
    pool = make_pool(rng, 5, 1, 16, 64, False, dev)
    q = torch.from_numpy(rng.standard_normal((2, 2, 64))).to(dev).bfloat16()
    ok = [[[0, 1]], [[0, 1]]]
    for table, seqs, qsl, sel in [([[0, 5], [2, 3]], [20, 20], [0, 1, 2], ok),
                                  ([[-1, 1], [2, 3]], [20, 20], [0, 1, 2], ok),
                                  ([[0, 1], [2, 3]], [33, 20], [0, 1, 2], ok),
                                  ([[0, 1], [2, 3]], [20, 20], [0, 1, 2], [[[0, 2]], [[0, 1]]]),
                                  ([[0, 1], [2, 3]], [20, 20], [0, 1, 2], [[[-2, 1]], [[0, 1]]])]:
        out = torch.full_like(q, 7.0)
        pa.sparse_forward(q, out, i32(qsl, dev), i32(seqs, dev), i32(table, dev), i32(sel, dev),
                          pool, 0.125)
        assert pa.get_error() == pa.PA_ERR_DEVICE_BOUNDS
        want, tol = ref.sparse(ref.f64(q), ref.cells(pool.k), ref.cells(pool.v), table, np.array(ok),
                               [1, 1, 2], [20, 20], 16, 2, 0.125, 1.0, 1.0, False)
        check(ref.f64(out)[1], want[1], tol[1])


# ----------------------------------------------------------------------- mass

def run_mass(dev, rng, seqs, new, Hq, Hkv, D, B, fp8, window=0, decay=0.75, in_place=False,
             spoil=None, idx=True, scale=None, extra=0):
    table, qsl, blocks = batch(rng, seqs, new, B, dev, wide=1)
    pool = make_pool(rng, blocks, Hkv, B, D, fp8, dev)
    stale(pool, table, seqs, B, fp8)
    T = int(qsl[-1])
    q = torch.from_numpy(rng.standard_normal((T, Hq, D)) * 1.5).to(dev).bfloat16()
    if spoil:
        spoil(q, pool, table)
    R = len(seqs)
    rows = rng.permutation(R + 2)[:R] if idx else np.arange(R)
    places = max(seqs) + 3
    old = torch.from_numpy(rng.random((R + 2, places)).astype(np.float32)).to(dev)
    for r, n in enumerate(seqs):  # what held the row before may have left anything there
        old[int(rows[r]), n - new[r]:] = float("nan")
    out = old.clone() if in_place else torch.full_like(old, 7.0)
    qh, sh = np.array(qsl, np.int32), np.array(seqs, np.int32)
    ws = torch.empty(pa.attention_mass_workspace_size(qh, sh, Hq, Hkv, window) + extra,
                     dtype=torch.uint8, device=dev)
    ws.fill_(0xFF)
    scale = D ** -0.5 if scale is None else scale
    pa.attention_mass(q, out if in_place else old, out, i32(qsl, dev), i32(seqs, dev), qh, sh,
                      i32(table, dev), pool, scale, idx_mapping=i32(rows, dev) if idx else None,
                      decay=decay, window=window, workspace=ws)
    before = ref.f64(old)
    want, tol = ref.mass(ref.f64(q), ref.cells(pool.k), before, rows, table, qsl, seqs, B,
                         Hq // Hkv, scale, pool.k_scale, decay, window,
                         before.copy() if in_place else np.full(before.shape, 7.0), fp8)
    return ref.f64(out), want, tol


MASS_SHAPES = [  # Hq, Hkv, D, B, window
    (1, 1, 64, 16, 0), (8, 8, 128, 16, 0), (4, 2, 128, 32, 1), (6, 2, 64, 64, 3),
    (8, 1, 128, 16, 2), (10, 2, 128, 16, 16), (16, 1, 64, 32, 1), (17, 1, 128, 64, 5),
    (40, 2, 128, 16, 64), (28, 4, 64, 16, 0),
]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("shape", MASS_SHAPES, ids=str)
@pytest.mark.parametrize("case", range(len(BATCHES)))
def test_mass(cuda_device, case, shape, fp8):
    Hq, Hkv, D, B, window = shape
    rng = np.random.default_rng(case + Hq + D)
    check(*run_mass(cuda_device, rng, *BATCHES[case], Hq, Hkv, D, B, fp8, window,
                    in_place=bool(case & 1), idx=case % 3 != 0))
    assert pa.get_error() == pa.PA_OK


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
def test_mass_long(cuda_device, D, fp8):
    """Several splits and parts, row tiles that end inside a query's heads, decodes
    beside chunks, one negative scale."""
    rng = np.random.default_rng(15)
    check(*run_mass(cuda_device, rng, [2600, 1030, 700], [1, 2, 90], 6, 2, D, 16, fp8))
    check(*run_mass(cuda_device, rng, [1500, 300], [150, 1], 7, 1, D, 64, fp8, window=100))
    check(*run_mass(cuda_device, rng, [1100, 130], [1, 40], 5, 1, D, 32, fp8, scale=-0.1))
    assert pa.get_error() == pa.PA_OK


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
def test_mass_of_many_chunks(cuda_device, D, fp8):
    """More row tiles than SMs, several of them in the run of one CTA, some cut by its
    end, and decodes between them."""
    rng = np.random.default_rng(24)
    seqs = [int(x) for x in rng.integers(40, 400, 50)]
    new = [int(x) for x in rng.integers(20, 41, 50)]
    new[7] = new[20] = 1
    new[31] = 0
    check(*run_mass(cuda_device, rng, seqs, new, 12, 2, D, 16, fp8, window=30))
    assert pa.get_error() == pa.PA_OK


def test_mass_on_two_streams(cuda_device):
    """Two calls at once, each with a workspace and a mass of its own."""
    dev, B, Hkv, Hq, D = cuda_device, 16, 2, 8, 128
    rng = np.random.default_rng(25)
    jobs = []
    for seqs, new in (([3000, 2000], [40, 64]), ([2500, 1800, 900], [1, 50, 2])):
        table, qsl, blocks = batch(rng, seqs, new, B, dev)
        pool = make_pool(rng, blocks, Hkv, B, D, False, dev)
        q = torch.from_numpy(rng.standard_normal((int(qsl[-1]), Hq, D))).to(dev).bfloat16()
        old = torch.rand((len(seqs), max(seqs)), device=dev)
        qh, sh = np.array(qsl, np.int32), np.array(seqs, np.int32)
        ws = torch.empty(pa.attention_mass_workspace_size(qh, sh, Hq, Hkv), dtype=torch.uint8,
                         device=dev)
        jobs.append((q, old, torch.zeros_like(old), i32(qsl, dev), i32(seqs, dev), qh, sh,
                     i32(table, dev), pool, ws, table))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(3):
        for s, (q, old, out, dq, ds, qh, sh, tab, pool, ws, _) in zip(streams, jobs):
            pa.attention_mass(q, old, out, dq, ds, qh, sh, tab, pool, 0.1, workspace=ws, stream=s)
    torch.cuda.synchronize()
    assert pa.get_error() == pa.PA_OK
    for q, old, out, dq, ds, qh, sh, tab, pool, ws, table in jobs:
        check(ref.f64(out), *ref.mass(ref.f64(q), ref.cells(pool.k), ref.f64(old), range(len(sh)),
                                      table, qh.tolist(), sh.tolist(), B, Hq // Hkv, 0.1, 1.0, 1.0,
                                      0, np.zeros(old.shape), False))


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("new", [3, 40], ids=["streamed", "tiles"])
def test_mass_numbers_that_are_not_finite(cuda_device, new, fp8):
    """A row that meets a NaN gives NaN to every key that it sees, and to no other
    (the keys after it); a key that scores -inf receives nothing."""
    def spoil(q, pool, table):
        bad = 0x7F if fp8 else float("nan")
        q[1, 1, 3] = float("nan")
        q[2 * new + 1, 0, 4] = float("inf")
        if not fp8:
            q[new:2 * new, :, 9] = 1.0
            pool.k[int(table[1, 0]), 0, 5, 9] = float("-inf")
        pool.k[int(table[3, 3]), 0, 2, 5] = bad  # token 50 of request 3

    rng = np.random.default_rng(16)
    seqs = [60, 60, 60, 64 if new == 40 else 51]
    got, want, tol = run_mass(cuda_device, rng, seqs, [new] * 4, 2, 1, 64, 16, fp8, spoil=spoil)
    assert np.isnan(want).any() and np.isfinite(want).any()
    check(got, want, tol)


def test_mass_refuses_what_leaves_the_buffers(cuda_device):
    """Device lengths above the mirrors', bad blocks and rows: flagged; requests that
    stay within are right, and nothing else is written."""
    dev, B, Hkv, Hq, D = cuda_device, 16, 1, 2, 64
    rng = np.random.default_rng(17)
    pool = make_pool(rng, 20, Hkv, B, D, False, dev)
    table = rng.permutation(20)[:16].reshape(2, 8)
    for new in (1, 30):
        qsl, seqs = np.array([0, new, 2 * new], np.int32), np.array([40, 50], np.int32)
        q = torch.from_numpy(rng.standard_normal((2 * new, Hq, D))).to(dev).bfloat16()
        ws = torch.empty(pa.attention_mass_workspace_size(qsl, seqs, Hq, Hkv), dtype=torch.uint8,
                         device=dev)
        old = torch.rand((2, 120), device=dev)

        def run(dev_qsl=qsl, dev_seqs=seqs, dev_table=table, idx=None):
            out = torch.full_like(old, 7.0)
            pa.attention_mass(q, old, out, i32(dev_qsl, dev), i32(dev_seqs, dev), qsl, seqs,
                              i32(dev_table, dev), pool, 0.125, workspace=ws,
                              idx_mapping=None if idx is None else i32(idx, dev))
            return ref.f64(out), pa.get_error()

        want, tol = ref.mass(ref.f64(q), ref.cells(pool.k), ref.f64(old), [0, 1], table, qsl, seqs,
                             B, Hq, 0.125, 1.0, 1.0, 0, np.full((2, 120), 7.0), False)
        got, status = run()
        assert status == pa.PA_OK
        check(got, want, tol)
        bad_block = table.copy()
        bad_block[0, 1] = 20
        for kw in (dict(dev_seqs=[2000, 50]), dict(dev_seqs=[129, 50]), dict(dev_seqs=[-5, 50]),
                   dict(dev_seqs=[new - 1, 50]), dict(dev_table=bad_block), dict(idx=[2, 1]),
                   dict(idx=[-1, 1]), dict(dev_qsl=[-1, new, 2 * new])):
            got, status = run(**kw)
            assert status == pa.PA_ERR_DEVICE_BOUNDS, kw
            check(got[1], want[1], tol[1])
            if "dev_table" not in kw:
                assert (got[0] == 7).all(), kw


# ----------------------------------------------------------------- compaction

@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("D,B,Hkv", [(128, 16, 2), (64, 32, 1), (128, 64, 8), (64, 16, 5)])
def test_compact(cuda_device, D, B, Hkv, in_place, fp8):
    dev = cuda_device
    rng = np.random.default_rng(D + B + Hkv)
    seqs = [1, 700, 64, 1500, 33, 0, 2000]
    k = 1200
    kept = np.full((len(seqs), k), -1)
    lens = [1, 300, 64, 1190, 1, 0, 600]
    for r, (n, m) in enumerate(zip(seqs, lens)):
        kept[r, :m] = np.sort(rng.permutation(n)[:m])
    kept[6, :600] = np.arange(1400, 2000)
    table, _, blocks = batch(rng, seqs, seqs, B, dev)
    pool = make_pool(rng, blocks + len(seqs) * (-(-k // B)), Hkv, B, D, fp8, dev)
    if in_place:
        dst = table
    else:
        dst = blocks + rng.permutation(len(seqs) * (-(-k // B))).reshape(len(seqs), -1)
    rows = rng.permutation(len(seqs) + 1)[: len(seqs)]
    mass = torch.rand((len(seqs) + 1, 2000), device=dev)
    mass_out = mass if in_place else torch.full_like(mass, 7.0)
    want_m, was = mass_out.cpu().numpy().copy(), mass.cpu().numpy().copy()
    want = [x.cpu().view(torch.int16 if x.dtype == torch.bfloat16 else torch.uint8).numpy().copy()
            for x in (pool.k, pool.v)]
    for w in want:
        start = w.copy()
        for r, m in enumerate(lens):
            for i in range(m):
                a, b = kept[r, i], i
                w[dst[r][b // B], :, b % B] = start[table[r][a // B], :, a % B]
    for r, m in enumerate(lens):
        want_m[rows[r], :m] = was[rows[r], kept[r, :m]]
    pa.compact_cache(pool, i32(table, dev), i32(dst, dev), i32(kept, dev), i32(lens, dev),
                     mass_in=mass, mass_out=mass_out, idx_mapping=i32(rows, dev))
    assert pa.get_error() == pa.PA_OK
    for x, w in zip((pool.k, pool.v), want):
        assert np.array_equal(x.cpu().view(torch.int16 if not fp8 else torch.uint8).numpy(), w)
    assert np.array_equal(mass_out.cpu().numpy(), want_m)


def test_compact_refuses_what_leaves_the_buffers(cuda_device):
    dev, B = cuda_device, 16
    rng = np.random.default_rng(19)
    for kept, lens, src, dst in [
            ([[0, 32], [3, 9]], [2, 2], [[0, 1], [2, 3]], [[4], [5]]),
            ([[0, -1], [3, 9]], [2, 2], [[0, 1], [2, 3]], [[4], [5]]),
            ([[0, 17], [3, 9]], [3, 2], [[0, 1], [2, 3]], [[4], [5]]),
            ([[0, 17], [3, 9]], [-1, 2], [[0, 1], [2, 3]], [[4], [5]]),
            ([[0, 17], [3, 9]], [2, 2], [[0, 6], [2, 3]], [[4], [5]]),
            ([[0, 17], [3, 9]], [2, 2], [[0, 1], [2, 3]], [[-1], [5]])]:
        pool = make_pool(rng, 6, 1, B, 64, False, dev)
        was = pool.k.clone()
        mass = torch.rand((2, 40), device=dev)
        out = torch.full_like(mass, 7.0)
        pa.compact_cache(pool, i32(src, dev), i32(dst, dev), i32(kept, dev), i32(lens, dev),
                         mass_in=mass, mass_out=out)
        assert pa.get_error() == pa.PA_ERR_DEVICE_BOUNDS
        assert torch.equal(pool.k[5, 0, 0], was[2, 0, 3]) and torch.equal(pool.k[5, 0, 1], was[2, 0, 9])
        assert torch.equal(pool.k[:4], was[:4])
        assert torch.equal(out[1, :2], mass[1, [3, 9]]) and (out[:, 2:] == 7).all()


# ------------------------------------------------------ far places, other streams

def test_places_past_32_bits(cuda_device):
    """Blocks whose elements lie past 2^32 in the pool."""
    dev, B, Hkv, D, Hq = cuda_device, 64, 8, 128, 8
    blocks = (1 << 32) // (Hkv * B * D) + 20
    pool = pa.KVPool(*(torch.empty((blocks, Hkv, B, D), dtype=torch.bfloat16, device=dev)
                       for _ in range(2)))
    rng = np.random.default_rng(20)
    used = [blocks - 1, 0, blocks - 2, blocks - 7]
    near = {b: i for i, b in enumerate(used)}
    for x in (pool.k, pool.v):
        for b in used:
            x[b] = torch.from_numpy(rng.standard_normal((Hkv, B, D))).to(dev).bfloat16()
    small = [torch.stack([x[b] for b in used]) for x in (pool.k, pool.v)]
    table, seqs, qsl = [used[:3]], [150], [0, 1]
    q = torch.from_numpy(rng.standard_normal((1, Hq, D))).to(dev).bfloat16()
    bnd = torch.zeros((blocks, Hkv, 2, D), dtype=torch.bfloat16, device=dev)
    t, sq, qs = i32(table, dev), i32(seqs, dev), i32(qsl, dev)
    pa.update_block_bounds(pool, bnd, t, sq)
    scores = torch.zeros((1, Hkv, 3), device=dev)
    pa.score_blocks(q, bnd, scores, qs, sq, t, pool)
    sel = i32(np.tile([0, 2, 1], (1, Hkv, 1)), dev)
    out = torch.zeros_like(q)
    pa.sparse_forward(q, out, qs, sq, t, sel, pool, D ** -0.5)
    old = torch.zeros((1, 150), device=dev)
    mass = torch.zeros_like(old)
    ws = torch.empty(pa.attention_mass_workspace_size(qsl, seqs, Hq, Hkv), dtype=torch.uint8,
                     device=dev)
    pa.attention_mass(q, old, mass, qs, sq, qsl, seqs, t, pool, D ** -0.5, workspace=ws)
    q3 = q.expand(20, Hq, D).contiguous()
    mass3 = torch.zeros_like(old)
    ws3 = torch.empty(pa.attention_mass_workspace_size([0, 20], seqs, Hq, Hkv), dtype=torch.uint8,
                      device=dev)
    pa.attention_mass(q3, old, mass3, i32([0, 20], dev), sq, [0, 20], seqs, t, pool, D ** -0.5,
                      workspace=ws3)
    kept = np.arange(0, 150, 3)[None]
    pa.compact_cache(pool, t, i32([[used[3]]], dev), i32(kept, dev), i32([50], dev))
    assert pa.get_error() == pa.PA_OK
    k, v = (ref.f64(x) for x in small)
    tab = [[near[b] for b in used[:3]]]
    b64 = ref.bounds(k, tab, None, seqs, B, np.zeros((4, Hkv, 2, D)))
    assert np.array_equal(ref.f64(bnd[used]), b64)
    want, tol = ref.scores(ref.f64(q), b64, tab, qsl, seqs, B, 1, 1.0, np.zeros((1, Hkv, 3)))
    check(scores.cpu().numpy(), want, tol)
    check(ref.f64(out), *ref.sparse(ref.f64(q), k, v, tab, sel.cpu().numpy(), qsl, seqs, B, 1,
                                    D ** -0.5, 1.0, 1.0, False))
    for got, x, n in ((mass, q, 1), (mass3, q3, 20)):
        check(ref.f64(got), *ref.mass(ref.f64(x), k, np.zeros((1, 150)), [0], tab, [0, n], seqs, B,
                                      1, D ** -0.5, 1.0, 1.0, 0, np.zeros((1, 150)), False))
    moved = torch.cat([small[0][near[b]] for b in used[:3]], dim=1)[:, ::3][:, :50]
    assert torch.equal(pool.k[used[3]][:, :50], moved)


def test_captured_calls_follow_the_device(cuda_device):
    """All calls captured once on a side stream and replayed on lengths, tables and
    values that have changed in place."""
    dev, B, Hkv, Hq, D, k = cuda_device, 16, 2, 8, 128, 6
    rng = np.random.default_rng(23)
    cap, R, blocks = 40, 3, 60
    pool = make_pool(rng, blocks, Hkv, B, D, False, dev)
    qsl_cap, seq_cap = [0, 1, 2, 32], [200, 220, 240]
    table = i32(np.zeros((R, 15)), dev)
    qsl, seqs = i32(qsl_cap, dev), i32(seq_cap, dev)
    q = torch.zeros((cap, Hq, D), dtype=torch.bfloat16, device=dev)
    bnd = torch.zeros((blocks, Hkv, 2, D), dtype=torch.bfloat16, device=dev)
    scores = torch.zeros((cap, Hkv, 15), device=dev)
    sel = torch.zeros((cap, Hkv, k), dtype=torch.int32, device=dev)
    out = torch.zeros_like(q)
    old, mass = torch.rand((R, 240), device=dev), torch.zeros((R, 240), device=dev)
    kept = torch.zeros((R, 50), dtype=torch.int32, device=dev)
    lens = torch.zeros(R, dtype=torch.int32, device=dev)
    qh, sh = np.array([0, 1, 2, cap], np.int32), np.array(seq_cap, np.int32)
    ws = torch.empty(pa.attention_mass_workspace_size(qh, sh, Hq, Hkv), dtype=torch.uint8,
                     device=dev)

    def calls():
        pa.update_block_bounds(pool, bnd, table, seqs, query_start_loc=qsl, num_tokens=cap)
        pa.score_blocks(q, bnd, scores, qsl, seqs, table, pool)
        pa.select_blocks(scores, sel, qsl, seqs, B)
        pa.sparse_forward(q, out, qsl, seqs, table, sel, pool, D ** -0.5)
        pa.attention_mass(q, old, mass, qsl, seqs, qh, sh, table, pool, D ** -0.5, workspace=ws)
        pa.select_tokens(mass, kept, lens, seqs, first=2, last=8)

    table.copy_(i32(rng.permutation(45).reshape(R, 15), dev))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        calls()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        calls()
    for seq, new in (([200, 220, 240], [1, 1, 30]), ([17, 160, 33], [1, 1, 33]),
                     ([1, 0, 90], [1, 0, 20])):
        t = rng.permutation(45).reshape(R, 15)
        qs = np.cumsum([0] + new)
        table.copy_(i32(t, dev))
        seqs.copy_(i32(seq, dev))
        qsl.copy_(i32(qs, dev))
        q.copy_(torch.from_numpy(rng.standard_normal((cap, Hq, D))).to(dev).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        assert pa.get_error() == pa.PA_OK
        n = int(qs[-1])
        kk, vv, qq = ref.cells(pool.k), ref.cells(pool.v), ref.f64(q)
        want, tol = ref.scores(qq, ref.bounds(kk, t, qs, seq, B, ref.f64(bnd)), t, qs, seq, B, 4,
                               1.0, ref.f64(scores))
        check(ref.f64(scores)[:n], want[:n], tol[:n])
        got_sel = sel.cpu().numpy()
        for r, row, p in ref.rows_of(qs, seq):
            for h in range(Hkv):
                assert np.array_equal(got_sel[row, h], ref.pick(
                    scores[row, h].cpu().numpy(), p // B + 1, 1, 2, k))
        want, tol = ref.sparse(qq, kk, vv, t, got_sel, qs, seq, B, 4, D ** -0.5, 1.0, 1.0, False)
        check(ref.f64(out)[:n], want[:n], tol[:n])
        was = ref.f64(mass)
        check(was, *ref.mass(qq, kk, ref.f64(old), [0, 1, 2], t, qs, seq, B, 4, D ** -0.5, 1.0, 1.0,
                             0, was.copy(), False))
        for r in range(R):
            assert np.array_equal(kept[r].cpu().numpy(),
                                  ref.pick(mass[r].cpu().numpy(), seq[r], 2, 8, 50))


MASS_FORMS = [  # new tokens and lengths of a batch; Hq, Hkv
    ([1, 9, 40, 3, 0, 100], [300, 40, 150, 3, 20, 260], 4, 2),  # 2, 18, 80, 6, 200 rows a kv head
    ([9, 20, 1, 21], [1100, 20, 700, 130], 6, 2),               # 27, 60, 3, 63: streamed in parts of 16
    ([16, 1, 11], [16, 2100, 300], 4, 1),                       # 64, 4, 44
    ([8] * 20, list(range(60, 160, 5)), 64, 8),                 # 64 rows each, too much to stream
    ([17, 40], [500, 90], 8, 2),                                # none to stream
]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("case", range(len(MASS_FORMS)))
def test_mass_forms(cuda_device, case, fp8):
    new, seqs, Hq, Hkv = MASS_FORMS[case]
    rng = np.random.default_rng(600 + case)
    check(*run_mass(cuda_device, rng, seqs, new, Hq, Hkv, 128 if case % 2 else 64, 16, fp8))


@pytest.mark.parametrize("new,less", [
    ([20, 1, 30, 12], [1, 1, 30, 2]), ([12, 1, 15], [2, 0, 15]), ([20, 30], [1, 2]),
    ([20, 30, 1], [3, 0, 1]), ([20, 30, 1], [0, 18, 0]), ([40, 1, 30, 12], [1, 1, 30, 2]),
    ([40, 50], [1, 2]), ([40, 1, 3], [4, 0, 3])], ids=str)
def test_mass_device_lengths_below_the_mirrors(cuda_device, new, less):
    """Whatever form the mirrors planned for a request, fewer rows and tokens of it are
    summed right."""
    dev, B, Hkv, Hq, D = cuda_device, 16, 2, 8, 64
    rng = np.random.default_rng(31)
    R = len(new)
    seqs = [int(n) for n in rng.integers(200, 400, size=R)]
    fewer = [int(rng.integers(max(less[r], 1), seqs[r])) for r in range(R)]
    table, qsl, blocks = batch(rng, seqs, new, B, dev, wide=1)
    pool = make_pool(rng, blocks, Hkv, B, D, False, dev)
    q = torch.from_numpy(rng.standard_normal((int(qsl[-1]), Hq, D))).to(dev).bfloat16()
    qh, sh = np.array(qsl, np.int32), np.array(seqs, np.int32)
    dev_qsl = np.concatenate([[0], np.cumsum(less)])
    old = torch.rand((R, 420), device=dev)
    ws = torch.empty(pa.attention_mass_workspace_size(qh, sh, Hq, Hkv), dtype=torch.uint8, device=dev)
    out = torch.full_like(old, 7.0)
    pa.attention_mass(q, old, out, i32(dev_qsl, dev), i32(fewer, dev), qh, sh, i32(table, dev), pool,
                      0.125, workspace=ws)
    assert pa.get_error() == pa.PA_OK
    want, tol = ref.mass(ref.f64(q), ref.cells(pool.k), ref.f64(old), list(range(R)), table,
                         dev_qsl.tolist(), fewer, B, Hq // Hkv, 0.125, 1.0, 1.0, 0,
                         np.full((R, 420), 7.0), False)
    check(ref.f64(out), want, tol)


@pytest.mark.parametrize("most", [1, 3])
def test_sparse_of_many_requests(cuda_device, most):
    rng = np.random.default_rng(90 + most)
    new = rng.integers(0, most + 1, size=300)
    seqs = (new + rng.integers(0, 60, size=300)).tolist()
    check(*attend(cuda_device, rng, seqs, new.tolist(), 4, 1, 64, 16, 3, False))
