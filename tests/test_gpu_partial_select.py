"""GPU tests of block bounds, block scores and the selection of blocks and
tokens against 64-bit definitions; what is selected, and bounds, are compared
exactly."""
import numpy as np
import pytest
import torch

from paged_kv_cache_143_gb300 import pa
from tests import partial_reference as ref

pytestmark = pytest.mark.gpu


def i32(a, dev):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=dev)


def make_pool(rng, blocks, Hkv, B, D, fp8, dev, fill=None):
    """Random keys and values; `fill` NaN in every cell instead."""
    if fill is not None:
        shape = (blocks, Hkv, B, D)
        if fp8:
            k, v = (torch.full(shape, 0x7F, dtype=torch.uint8, device=dev) for _ in range(2))
        else:
            k, v = (torch.full(shape, float("nan"), dtype=torch.bfloat16, device=dev)
                    for _ in range(2))
        return pa.KVPool(k, v, 0.5 if fp8 else 1.0, 0.25 if fp8 else 1.0)
    k, v = (torch.from_numpy(rng.standard_normal((blocks, Hkv, B, D))).to(dev).bfloat16()
            for _ in range(2))
    if fp8:
        k, v = ((x.float() * 20).to(torch.float8_e4m3fn).view(torch.uint8) for x in (k, v))
        return pa.KVPool(k, v, 1 / 20.0, 1 / 16.0)
    return pa.KVPool(k, v)


def batch(rng, seqs, q_lens, B, dev, spare=3, wide=0):
    """Block tables over shuffled blocks (-1 past a request's own), start array."""
    need = [-(-n // B) for n in seqs]
    order = rng.permutation(sum(need) + spare)
    table = np.full((len(seqs), max(need + [1]) + wide), -1)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n]
        at += n
    return table, np.cumsum([0] + list(q_lens)), sum(need) + spare


BATCHES = [  # (stored tokens, new tokens) of the requests
    ([1], [1]), ([17, 1, 64, 33], [1, 1, 1, 1]), ([130, 0, 5, 257], [130, 0, 0, 100]),
    ([64, 48, 49, 1], [16, 17, 2, 1]), ([300], [1]), ([16] * 40, [1] * 40),
]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("D,B,Hkv", [(128, 16, 2), (64, 32, 1), (128, 64, 3), (64, 16, 5),
                                     (128, 32, 8), (64, 64, 2)])
@pytest.mark.parametrize("case", range(len(BATCHES)))
def test_bounds(cuda_device, case, D, B, Hkv, fp8):
    dev = cuda_device
    rng = np.random.default_rng(100 * case + D + B)
    seqs, new = BATCHES[case]
    table, qsl, blocks = batch(rng, seqs, new, B, dev)
    pool = make_pool(rng, blocks, Hkv, B, D, fp8, dev)
    for r, n in enumerate(seqs):  # cells past a request's tokens hold NaN
        if n % B:
            for x in (pool.k, pool.v):
                x[int(table[r, n // B]), :, n % B:] = 0x7F if fp8 else float("nan")
    bnd = torch.full((blocks, Hkv, 2, D), 7.0, dtype=torch.bfloat16, device=dev)
    pa.update_block_bounds(pool, bnd, i32(table, dev), i32(seqs, dev),
                           query_start_loc=i32(qsl, dev), num_tokens=int(qsl[-1]) + 5)
    assert pa.get_error() == pa.PA_OK
    k = ref.cells(pool.k)
    want = ref.bounds(k, table, qsl, seqs, B, np.full((blocks, Hkv, 2, D), 7.0))
    assert np.array_equal(ref.f64(bnd), want)
    # all blocks
    pa.update_block_bounds(pool, bnd, i32(table, dev), i32(seqs, dev))
    assert pa.get_error() == pa.PA_OK
    assert np.array_equal(ref.f64(bnd), ref.bounds(k, table, None, seqs, B, want))


def test_bounds_of_keys_that_are_not_finite(cuda_device):
    dev, B, D = cuda_device, 16, 64
    rng = np.random.default_rng(3)
    pool = make_pool(rng, 3, 1, B, D, False, dev)
    pool.k[1, 0, 3, 5] = float("nan")
    pool.k[1, 0, 4, 6] = float("inf")
    pool.k[1, 0, 5, 7] = float("-inf")
    bnd = torch.zeros((3, 1, 2, D), dtype=torch.bfloat16, device=dev)
    pa.update_block_bounds(pool, bnd, i32([[1, 2]], dev), i32([20], dev))
    want = ref.bounds(ref.cells(pool.k), [[1, 2]], None, [20], B, np.zeros((3, 1, 2, D)))
    assert np.isnan(want[1, 0, :, 5]).all() and np.isfinite(want[1, 0, :, 6:8]).all()
    assert np.array_equal(ref.f64(bnd), want, equal_nan=True)


def test_bounds_refuse_what_leaves_the_pool(cuda_device):
    """A bad block, a length past the table, a start array past num_tokens: flagged,
    and the other requests' bounds are right."""
    dev, B, D, Hkv = cuda_device, 16, 128, 2
    rng = np.random.default_rng(4)
    pool = make_pool(rng, 6, Hkv, B, D, False, dev)
    k = ref.cells(pool.k)

    def run(table, seqs, qsl, n):
        bnd = torch.full((6, Hkv, 2, D), 7.0, dtype=torch.bfloat16, device=dev)
        pa.update_block_bounds(pool, bnd, i32(table, dev), i32(seqs, dev),
                               query_start_loc=None if qsl is None else i32(qsl, dev),
                               num_tokens=n)
        return ref.f64(bnd), pa.get_error()

    blank = lambda: np.full((6, Hkv, 2, D), 7.0)
    for table, seqs, qsl, n, good in [
            ([[0, 6], [2, 3]], [20, 20], [0, 20, 40], 40, [0, 2, 3]),
            ([[-1, 1], [2, 3]], [20, 20], None, None, [1, 2, 3]),
            ([[0, 1], [2, 3]], [33, 20], [0, 1, 2], 2, [3]),
            ([[0, 1], [2, 3]], [-1, 20], None, None, [2, 3]),
            ([[0, 1], [2, 3]], [20, 20], [0, 20, 50], 40, [0, 1])]:
        got, status = run(table, seqs, qsl, n)
        assert status == pa.PA_ERR_DEVICE_BOUNDS
        want = blank()
        for r in range(2):
            for i in range(2):
                if table[r][i] in good:
                    x = k[table[r][i]][:, : min(B, 20 - i * B)]
                    want[table[r][i], :, 0], want[table[r][i], :, 1] = x.min(1), x.max(1)
        assert np.array_equal(got, want), (table, seqs)


SCORE_SHAPES = [  # Hq, Hkv, D, B
    (1, 1, 64, 16), (8, 8, 128, 16), (4, 2, 128, 32), (6, 2, 64, 64), (8, 2, 128, 16),
    (10, 2, 128, 16), (16, 2, 64, 32), (9, 1, 128, 64), (32, 2, 128, 16), (20, 1, 64, 16),
    (64, 1, 128, 32), (28, 4, 128, 16),
]


def run_scores(dev, rng, seqs, new, Hq, Hkv, D, B, fp8, spoil=None, extra_rows=0):
    table, qsl, blocks = batch(rng, seqs, new, B, dev, wide=2)
    pool = make_pool(rng, blocks, Hkv, B, D, fp8, dev, fill=True)
    raw = np.sort(rng.standard_normal((blocks, Hkv, 2, D)) * (20 if fp8 else 1), axis=2)
    bnd = torch.from_numpy(raw).to(dev).bfloat16()
    T = int(qsl[-1]) + extra_rows
    q = torch.from_numpy(rng.standard_normal((T, Hq, D))).to(dev).bfloat16()
    if spoil:
        spoil(q, bnd, table)
    out = torch.full((T, Hkv, table.shape[1]), 7.0, device=dev)
    pa.score_blocks(q, bnd, out, i32(qsl, dev), i32(seqs, dev), i32(table, dev), pool)
    want, tol = ref.scores(ref.f64(q), ref.f64(bnd), table, qsl, seqs, B, Hq // Hkv,
                           pool.k_scale, np.full(out.shape, 7.0))
    return out.cpu().numpy().astype(np.float64), want, tol


@pytest.mark.parametrize("shape", SCORE_SHAPES, ids=str)
@pytest.mark.parametrize("case", range(len(BATCHES)))
def test_scores(cuda_device, case, shape):
    Hq, Hkv, D, B = shape
    rng = np.random.default_rng(case + Hq + D)
    got, want, tol = run_scores(cuda_device, rng, *BATCHES[case], Hq, Hkv, D, B, bool(case & 1),
                                extra_rows=case % 3)
    assert pa.get_error() == pa.PA_OK
    assert (np.abs(got - want) <= tol).all()


def test_scores_long(cuda_device):
    rng = np.random.default_rng(9)
    got, want, tol = run_scores(cuda_device, rng, [9000, 700, 4111], [1, 90, 3], 8, 2, 128, 16,
                                False)
    assert (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (4, 1), (16, 1), (20, 1)])
def test_scores_of_chunks_among_empty_requests(cuda_device, Hq, Hkv):
    """No more tokens than requests, most of them in one request."""
    rng = np.random.default_rng(14)
    new = [0, 11, 0, 0, 0, 0, 1, 0, 0, 0, 0, 0, 3]
    seqs = [30, 200, 0, 5, 64, 0, 70, 1, 0, 16, 2, 0, 40]
    got, want, tol = run_scores(cuda_device, rng, seqs, new, Hq, Hkv, 64, 16, False)
    assert pa.get_error() == pa.PA_OK
    assert (np.abs(got - want) <= tol).all()


def test_scores_that_are_not_finite(cuda_device):
    """NaN of a query or a bound reaches what it takes part in; bounds are finite by
    construction, so an infinite query times a zero bound is the only other NaN."""
    def spoil(q, bnd, table):
        q[2, 3, 7] = float("nan")     # token 2: head 3 is of kv head 1
        q[4, 0, 9] = float("inf")
        bnd[table[1, 0], 0, 1, 4] = float("nan")
        q[5] = 0

    rng = np.random.default_rng(10)
    got, want, tol = run_scores(cuda_device, rng, [40, 20, 70], [3, 2, 4], 4, 2, 64, 16, False,
                                spoil=spoil)
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.isnan(want).any()
    assert np.array_equal(got[~fine], want[~fine], equal_nan=True) and np.isinf(want).any()
    assert (np.abs(got[fine] - want[fine]) <= tol[fine]).all()


def test_scores_refuse_what_leaves_the_buffers(cuda_device):
    dev = cuda_device
    rng = np.random.default_rng(12)
    pool = make_pool(rng, 5, 1, 16, 64, False, dev)
    bnd = torch.from_numpy(rng.standard_normal((5, 1, 2, 64))).to(dev).bfloat16()
    q = torch.from_numpy(rng.standard_normal((2, 2, 64))).to(dev).bfloat16()
    for table, seqs, qsl in [([[0, 5], [2, 3]], [20, 20], [0, 1, 2]),
                             ([[0, 1], [2, 3]], [33, 20], [0, 1, 2]),
                             ([[0, 1], [2, 3]], [0, 20], [0, 1, 2]),
                             ([[0, 1], [2, 3]], [20, 20], [-1, 1, 2])]:
        out = torch.full((2, 1, 2), 7.0, device=dev)
        pa.score_blocks(q, bnd, out, i32(qsl, dev), i32(seqs, dev), i32(table, dev), pool)
        assert pa.get_error() == pa.PA_ERR_DEVICE_BOUNDS
        want, tol = ref.scores(ref.f64(q), ref.f64(bnd), table, [1, 1, 2], [20, 20], 16, 2, 1.0,
                               np.full((2, 1, 2), 7.0))
        got = out.cpu().numpy()
        assert (np.abs(got - want) <= tol)[1].all()


# ------------------------------------------------------------------ selection

def spoiled(rng, shape, kind):
    if kind == "plain":
        return rng.standard_normal(shape).astype(np.float32)
    if kind == "ties":
        return rng.integers(-2, 3, shape).astype(np.float32) * np.float32(0.0 if shape[-1] < 3 else 1)
    if kind == "zeros":
        return np.where(rng.random(shape) < 0.5, 0.0, -0.0).astype(np.float32)
    x = rng.standard_normal(shape).astype(np.float32)
    x[rng.random(shape) < 0.2] = np.nan
    x[rng.random(shape) < 0.2] = np.inf
    x[rng.random(shape) < 0.2] = -np.inf
    x[rng.random(shape) < 0.1] = np.float32(-3.4028235e38)
    return x


@pytest.mark.parametrize("kind", ["plain", "ties", "zeros", "special"])
@pytest.mark.parametrize("first,last,k", [(0, 0, 1), (1, 2, 5), (3, 0, 3), (0, 4, 40), (2, 30, 129)])
def test_select_blocks(cuda_device, first, last, k, kind):
    dev, B, H = cuda_device, 16, 3
    rng = np.random.default_rng(k + first)
    seqs, new = [1, 700, 16, 17, 2000, 333, 0], [1, 3, 1, 2, 40, 1, 0]
    qsl = np.cumsum([0] + new)
    N = 127
    x = spoiled(rng, (int(qsl[-1]) + 1, H, N), kind)
    out = torch.full((x.shape[0], H, k), 9, dtype=torch.int32, device=dev)
    pa.select_blocks(torch.from_numpy(x).to(dev), out, i32(qsl, dev), i32(seqs, dev), B,
                     first=first, last=last)
    assert pa.get_error() == pa.PA_OK
    got = out.cpu().numpy()
    assert (got[-1] == 9).all()  # a row behind the last sequence
    for r, t, p in ref.rows_of(qsl, seqs):
        for h in range(H):
            want = ref.pick(x[t, h], p // B + 1, first, last, k)
            assert np.array_equal(got[t, h], want), (t, h)


@pytest.mark.parametrize("kind", ["plain", "ties", "special"])
def test_select_blocks_of_long_contexts(cuda_device, kind):
    """Rows that several CTAs share, and rows past what they hold at once."""
    dev, B, H, k = cuda_device, 16, 2, 70
    rng = np.random.default_rng(31)
    for N in (5000, 40000):
        seqs, new = [N * B, 17, N * B // 2], [2, 1, 1]
        qsl = np.cumsum([0] + new)
        x = spoiled(rng, (4, H, N), kind)
        out = torch.full((4, H, k), 9, dtype=torch.int32, device=dev)
        pa.select_blocks(torch.from_numpy(x).to(dev), out, i32(qsl, dev), i32(seqs, dev), B,
                         first=2, last=3)
        assert pa.get_error() == pa.PA_OK
        for r, t, p in ref.rows_of(qsl, seqs):
            for h in range(H):
                assert np.array_equal(out[t, h].cpu().numpy(),
                                      ref.pick(x[t, h], p // B + 1, 2, 3, k)), (N, t, h)


@pytest.mark.parametrize("places", [7, 1000, 1024, 1025, 4096, 4097, 20000, 32768, 32769, 70001])
@pytest.mark.parametrize("kind", ["plain", "ties", "special"])
def test_select_tokens(cuda_device, places, kind):
    dev = cuda_device
    rng = np.random.default_rng(places)
    seqs = [places, places - 1, max(1, places // 3), 0, 1, min(places, 33)]
    idx = rng.permutation(len(seqs) + 2)[: len(seqs)]
    x = spoiled(rng, (len(seqs) + 2, places), kind)
    for first, last, k in [(0, 0, 1), (2, 3, max(5, places // 4)), (4, 16, 20), (0, 0, places)]:
        kept = torch.full((len(seqs), k), 9, dtype=torch.int32, device=dev)
        lens = torch.full((len(seqs),), 9, dtype=torch.int32, device=dev)
        pa.select_tokens(torch.from_numpy(x).to(dev), kept, lens, i32(seqs, dev),
                         idx_mapping=i32(idx, dev), first=first, last=last)
        assert pa.get_error() == pa.PA_OK
        assert lens.tolist() == [min(n, k) for n in seqs]
        got = kept.cpu().numpy()
        for r, n in enumerate(seqs):
            assert np.array_equal(got[r], ref.pick(x[idx[r]], n, first, last, k)), (r, k)


def test_select_refuses_what_leaves_the_buffers(cuda_device):
    dev = cuda_device
    x = torch.randn((3, 50), device=dev)
    for seqs, idx in [([51, 20], None), ([-1, 20], None), ([30, 20], [3, 1]), ([30, 20], [-1, 1])]:
        kept = torch.full((2, 5), 9, dtype=torch.int32, device=dev)
        lens = torch.full((2,), 9, dtype=torch.int32, device=dev)
        pa.select_tokens(x, kept, lens, i32(seqs, dev), first=0, last=0,
                         idx_mapping=None if idx is None else i32(idx, dev))
        assert pa.get_error() == pa.PA_ERR_DEVICE_BOUNDS
        assert np.array_equal(kept[1].cpu().numpy(), ref.pick(x[1].cpu().numpy(), 20, 0, 0, 5))
        assert (kept[0] == 9).all() and lens.tolist() == [9, 5]
    s = torch.randn((2, 1, 3), device=dev)
    out = torch.full((2, 1, 2), 9, dtype=torch.int32, device=dev)
    pa.select_blocks(s, out, i32([0, 1, 2], dev), i32([49, 20], dev), 16, first=0, last=0)
    assert pa.get_error() == pa.PA_ERR_DEVICE_BOUNDS
    assert (out[0] == 9).all()
    assert np.array_equal(out[1, 0].cpu().numpy(), ref.pick(s[1, 0].cpu().numpy(), 2, 0, 0, 2))


@pytest.mark.parametrize("R,most", [(33, 1), (1100, 1), (1100, 3), (2100, 1)])
def test_rows_of_many_requests(cuda_device, R, most):
    """More requests than a warp's lanes, and than their square: which request a row or a
    unit of work belongs to."""
    dev, B, Hkv = cuda_device, 16, 1
    rng = np.random.default_rng(R + most)
    new = rng.integers(0, most + 1, size=R)
    seqs = (new + rng.integers(0, 70, size=R)).tolist()
    got, want, tol = run_scores(dev, rng, seqs, new.tolist(), 4, Hkv, 64, B, False)
    assert pa.get_error() == pa.PA_OK
    assert (np.abs(got - want) <= tol).all()
    qsl = np.cumsum([0] + new.tolist())
    x = rng.standard_normal((int(qsl[-1]) + 2, Hkv, 5)).astype(np.float32)
    selected = torch.full((x.shape[0], Hkv, 3), 7, dtype=torch.int32, device=dev)
    pa.select_blocks(torch.from_numpy(x).to(dev), selected, i32(qsl, dev), i32(seqs, dev), B,
                     first=0, last=1)
    out = np.full((x.shape[0], Hkv, 3), 7)
    for r, t, p in ref.rows_of(qsl.tolist(), seqs):
        out[t, 0] = ref.pick(x[t, 0], p // B + 1, 0, 1, 3)
    assert pa.get_error() == pa.PA_OK
    assert np.array_equal(selected.cpu().numpy(), out)
