"""GPU tests of the calls on a part of a cache at their edges: what is left after
values cancel, device lengths above the mirrors, many heads, bad block ids."""
import numpy as np
import pytest
import torch

from paged_kv_cache_143_gb300 import pa
from tests import partial_reference as ref
from tests.test_gpu_partial_attention import check
from tests.test_gpu_partial_select import batch, i32, make_pool

pytestmark = pytest.mark.gpu


def code(x, fp8):
    """The nearest bf16, or E4M3 code."""
    x = torch.as_tensor(x)
    return x.float().to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else x.bfloat16()


def cancelling(dev, rng, Hkv, g, D, fp8, k):
    """One token on 40 keys: eight whose weights fall by about e^2 from one to the next, the
    others' below e^-100. In every dim the values of the eight are chosen one after the other
    to cancel what stands, so that of weights of about 1 hardly anything is left."""
    B, n, scale = 16, 40, 1.0
    pool = make_pool(rng, 5, Hkv, B, D, fp8, dev)
    unit, unit_v = pool.k_scale, pool.v_scale
    q = torch.zeros((1, Hkv * g, D), device=dev)
    q[..., 0] = 8.0
    table = np.array([[3, 0, 4]])
    for h in range(Hkv):
        s = np.full(n, -17.0)
        order = rng.permutation(n)[:8]
        s[order] = -(2.1 * np.arange(8) + rng.random(8) * 0.5) / 8
        ks = code(s / unit, fp8)
        cells = [(int(table[0, i // B]), i % B) for i in range(n)]
        for i, (b, o) in enumerate(cells):
            pool.k[b, h, o, 0] = ks[i].to(dev)
        x = 8.0 * unit * ref.cells(ks.reshape(1, -1))[0]
        w = np.exp(x - x.max())
        w /= w.sum()
        rest = np.array([w[i] for i in range(n) if i not in order])
        assert rest.max() < np.exp(-100.0)
        left = np.zeros(D)
        for j, i in enumerate(order):
            v = (rng.random(D) + 0.5 if j == 0 else -left / w[i]) / unit_v
            c = code(v, fp8)
            b, o = cells[i]
            pool.v[b, h, o] = c.to(dev)
            left += w[i] * ref.cells(c.reshape(1, -1))[0] * unit_v
    sel = np.full((1, Hkv, k), -1)
    sel[0, :, rng.permutation(k)[:3]] = np.array([0, 1, 2])[:, None]
    out = torch.zeros((1, Hkv * g, D), dtype=torch.bfloat16, device=dev)
    q = q.bfloat16()
    pa.sparse_forward(q, out, i32([0, 1], dev), i32([n], dev), i32(table, dev), i32(sel, dev), pool,
                      scale)
    assert pa.get_error() == pa.PA_OK
    K, V = ref.cells(pool.k), ref.cells(pool.v)
    want, _ = ref.sparse(ref.f64(q), K, V, table, sel, [0, 1], [n], B, g, scale, unit, unit_v, fp8)
    # A score is one product: its factor (three roundings), the product and the difference to the
    # reference, each half a step of at most 25 in units of log 2, for the weight and for the sum.
    # A weight is off by 2^-15 (f16: 2^-22) in the second product, by 2^-20 from exp2 and sums;
    # the output is rounded to bf16.
    rel = 2 * 5 * 25 * 2.0 ** -24 * np.log(2) + 2.0 ** -20 + 2.0 ** (-22 if fp8 else -15)
    tol = np.zeros(want.shape)
    for h in range(Hkv):
        Kh = ref.context(K, table[0], n, B, h) * unit
        Vh = np.abs(ref.context(V, table[0], n, B, h)) * unit_v
        x = scale * Kh @ ref.f64(q)[0, h * g]
        w = np.exp(x - x.max())
        tol[0, h * g:(h + 1) * g] = (w / w.sum()) @ Vh * rel
    assert (np.abs(want) < 2.0 ** -10).all()
    check(ref.f64(out), want, tol + 2.0 ** -8 * (np.abs(want) + tol))


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("g", [1, 4, 12])
@pytest.mark.parametrize("k", [3, 200], ids=["one CTA", "cluster"])
def test_sparse_where_values_cancel(cuda_device, k, g, D, fp8):
    """Weights enter the second product with more bits than a 16-bit number has."""
    cancelling(cuda_device, np.random.default_rng(g + D + k), 8, g, D, fp8, k)


def test_sparse_infinite_values(cuda_device):
    """An infinite value that a row sees gives an infinity of its sign, whatever bits of the
    weight the second product takes one by one; two of different signs give NaN."""
    dev, B, D = cuda_device, 16, 64
    rng = np.random.default_rng(3)
    pool = make_pool(rng, 4, 1, B, D, False, dev)
    pool.v[1, 0, 3, 5] = float("inf")
    pool.v[1, 0, 7, 6] = float("-inf")
    pool.v[2, 0, 0, 7] = float("inf")
    pool.v[2, 0, 1, 7] = float("-inf")
    pool.v[2, 0, 9, 8] = float("inf")  # behind the token
    q = torch.from_numpy(rng.standard_normal((1, 4, D))).to(dev).bfloat16()
    q[0, 3] = 0  # equal weights, powers of two: nothing is left of them
    sel = np.array([[[1, 0]]])
    out = torch.zeros_like(q)
    pa.sparse_forward(q, out, i32([0, 1], dev), i32([24], dev), i32([[1, 2]], dev), i32(sel, dev),
                      pool, 0.125)
    assert pa.get_error() == pa.PA_OK
    want, tol = ref.sparse(ref.f64(q), ref.cells(pool.k), ref.cells(pool.v), [[1, 2]], sel, [0, 1],
                           [24], B, 4, 0.125, 1.0, 1.0, False)
    got = ref.f64(out)
    assert (got[0, :, 5] == np.inf).all() and (got[0, :, 6] == -np.inf).all()
    assert np.isnan(got[0, :, 7]).all() and np.isfinite(got[0, :, 8]).all()
    rest = [d for d in range(D) if d not in (5, 6)]
    check(got[..., rest], want[..., rest], tol[..., rest])


# ------------------------------------------------- device lengths above the mirrors

def mass_of(dev, rng, new, seqs, dev_new, dev_seqs, Hq, Hkv, D, B, fp8=False, window=0):
    """One call planned for (new, seqs) on the device's lengths; what it wrote, and what it has
    to write: nothing for the requests that are above their mirrors."""
    R, most = len(new), [max(a, b) for a, b in zip(seqs, dev_seqs)]
    table, _, blocks = batch(rng, most, most, B, dev)
    pool = make_pool(rng, blocks, Hkv, B, D, fp8, dev)
    qsl, dq = (np.cumsum([0] + list(x)).astype(np.int32) for x in (new, dev_new))
    T = int(qsl[-1])
    assert int(dq[-1]) <= T
    q = torch.from_numpy(rng.standard_normal((T, Hq, D))).to(dev).bfloat16()
    old = torch.rand((R, max(most) + 2), device=dev)
    out = torch.full_like(old, 7.0)
    sh = np.array(seqs, np.int32)
    ws = torch.empty(pa.attention_mass_workspace_size(qsl, sh, Hq, Hkv, window), dtype=torch.uint8,
                     device=dev)
    ws.fill_(0xFF)
    pa.attention_mass(q, old, out, i32(dq, dev), i32(dev_seqs, dev), qsl, sh, i32(table, dev), pool,
                      0.125, workspace=ws, window=window)
    above = [bool(a and (a > b or c > d)) for a, b, c, d in zip(dev_new, new, dev_seqs, seqs)]
    assert pa.get_error() == (pa.PA_ERR_DEVICE_BOUNDS if any(above) else pa.PA_OK)
    blank = np.full(old.shape, 7.0)
    want, tol = ref.mass(ref.f64(q), ref.cells(pool.k), ref.f64(old), range(R), table, dq.tolist(),
                         dev_seqs, B, Hq // Hkv, 0.125, pool.k_scale, 1.0, window, blank.copy(), fp8)
    want[above] = 7.0
    return ref.f64(out), want, tol


@pytest.mark.parametrize("new,seqs,dev_new,dev_seqs", [
    # a little more of one request where the other left room: none of it is written
    ([1, 1], [900, 900], [1, 1], [1000, 500]),
    ([40, 40], [900, 900], [40, 40], [1000, 500]),
    ([40, 1], [500, 900], [40, 1], [510, 900]),
    # an earlier request's excess takes nothing from those within their mirrors
    ([1, 1, 1], [300, 300, 300], [1, 1, 1], [310, 300, 300]),
    ([40, 30, 50], [300, 700, 300], [40, 30, 50], [700, 700, 300]),
    ([40, 1, 50, 2], [300, 700, 300, 90], [40, 1, 50, 2], [300, 701, 300, 90]),
    ([40, 1, 50, 2], [300, 700, 300, 90], [40, 1, 50, 2], [600, 700, 300, 90]),
    # more new tokens than the mirror's, in either form and of a request that had none
    ([1, 2, 1], [300, 300, 300], [2, 1, 1], [300, 300, 300]),
    ([30, 40, 30], [300, 300, 300], [40, 30, 30], [300, 300, 300]),
    ([0, 3, 2], [300, 300, 300], [1, 2, 2], [300, 300, 300]),
    ([0, 60, 30], [300, 300, 300], [20, 40, 30], [300, 300, 300]),
    ([1, 40, 1], [300, 300, 300], [20, 20, 1], [300, 300, 300]),
], ids=str)
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_mass_above_the_mirrors(cuda_device, new, seqs, dev_new, dev_seqs, fp8):
    """Flagged and left out request by request."""
    check(*mass_of(cuda_device, np.random.default_rng(7), new, seqs, dev_new, dev_seqs, 8, 2, 64,
                   16, fp8))


def test_mass_above_the_window(cuda_device):
    """Rows that the window cuts to the mirror's number do not make a request fit."""
    check(*mass_of(cuda_device, np.random.default_rng(8), [20, 30], [300, 300], [30, 20],
                   [300, 300], 4, 2, 64, 16, window=2))


@pytest.mark.parametrize("R", [64, 65, 480, 481, 1300, 4200])
@pytest.mark.parametrize("most", [1, 6])
def test_mass_mirrors_of_many_requests(cuda_device, R, most):
    """Mirrors that come with the launch, or by one or more of their own; every seventh request above its own."""
    rng = np.random.default_rng(R + most)
    new = rng.integers(0, most + 1, size=R).tolist()
    seqs = [int(n + s) for n, s in zip(new, rng.integers(1, 60, size=R))]
    dev_seqs = [s + (r % 7 == 3) for r, s in enumerate(seqs)]
    check(*mass_of(cuda_device, rng, new, seqs, new, dev_seqs, 4, 1, 64, 16))


@pytest.mark.parametrize("Hq,Hkv", [(752 * 16, 752), (753 * 16, 753), (768 * 16, 768), (800 * 16, 800),
                                    (4000 * 2, 4000), (12040, 12040)])
def test_mass_of_many_heads(cuda_device, Hq, Hkv):
    """Rows of all kv heads up to what the streaming form's sums hold, and past it."""
    got, want, tol = mass_of(cuda_device, np.random.default_rng(Hkv), [1], [18], [1], [18], Hq, Hkv,
                             64, 16)
    check(got, want, tol)


# ---------------------------------------------------- block ids outside the pool

@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (8, 2), (9, 1)])
@pytest.mark.parametrize("chunks", [False, True], ids=["decodes", "chunks"])
def test_scores_of_blocks_outside_the_pool(cuda_device, chunks, Hq, Hkv):
    """Such a block scores 0 in either form; every other block as it does."""
    dev, B, D, blocks = cuda_device, 16, 128, 50
    rng = np.random.default_rng(Hq)
    seqs = [700, 900, 40] if chunks else rng.integers(30000, 60000, 30).tolist()
    qsl = np.cumsum([0] + ([1, 60, 2] if chunks else [1] * 30))
    table = rng.integers(0, blocks, (len(seqs), -(-max(seqs) // B)))  # (shared: bounds alone are read)
    pool = make_pool(rng, blocks, Hkv, B, D, False, dev, fill=True)
    bnd = torch.from_numpy(np.sort(rng.standard_normal((blocks, Hkv, 2, D)), axis=2)).to(dev).bfloat16()
    q = torch.from_numpy(rng.standard_normal((int(qsl[-1]), Hq, D))).to(dev).bfloat16()
    bad = rng.random(table.shape) < 0.1
    asked = np.where(bad, rng.choice([-1, -5, blocks, blocks + 1, 2 ** 31 - 1], table.shape), table)
    out = torch.full((int(qsl[-1]), Hkv, table.shape[1]), 7.0, device=dev)
    pa.score_blocks(q, bnd, out, i32(qsl, dev), i32(seqs, dev), i32(asked, dev), pool)
    assert pa.get_error() == pa.PA_ERR_DEVICE_BOUNDS
    with_zeros = np.concatenate([ref.f64(bnd), np.zeros((1, Hkv, 2, D))])
    check(ref.f64(out), *ref.scores(ref.f64(q), with_zeros, np.where(bad, blocks, table), qsl, seqs,
                                    B, Hq // Hkv, 1.0, np.full(out.shape, 7.0)))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("new", [[1, 2, 0, 1], [40, 30, 0, 70], [50, 1, 0, 3]],
                         ids=["streamed", "tiles", "both"])
def test_mass_of_blocks_outside_the_pool(cuda_device, new, fp8, D):
    """The keys of such a block count as zeros, whichever form its request takes."""
    dev, B, Hq, Hkv = cuda_device, 16, 8, 2
    rng = np.random.default_rng(D + fp8)
    seqs = [2100, 700, 300, 200]
    table, qsl, blocks = batch(rng, seqs, new, B, dev)
    pool = make_pool(rng, blocks, Hkv, B, D, fp8, dev)
    q = torch.from_numpy(rng.standard_normal((int(qsl[-1]), Hq, D))).to(dev).bfloat16()
    bad = (rng.random(table.shape) < 0.1) & (table >= 0)
    bad[0, 0] = bad[1, 43] = bad[2, 0] = True
    asked = np.where(bad, rng.choice([-1, -5, blocks, blocks + 1, 2 ** 31 - 1], table.shape), table)
    old = torch.rand((4, 2200), device=dev)
    out = torch.full_like(old, 7.0)
    qh, sh = np.array(qsl, np.int32), np.array(seqs, np.int32)
    ws = torch.empty(pa.attention_mass_workspace_size(qh, sh, Hq, Hkv), dtype=torch.uint8, device=dev)
    pa.attention_mass(q, old, out, i32(qsl, dev), i32(seqs, dev), qh, sh, i32(asked, dev), pool, 0.125,
                      workspace=ws)
    assert pa.get_error() == pa.PA_ERR_DEVICE_BOUNDS
    keys = ref.cells(pool.k)
    check(ref.f64(out), *ref.mass(ref.f64(q), np.concatenate([keys, np.zeros_like(keys[:1])]),
                                  ref.f64(old), range(4), np.where(bad, blocks, table), qsl, seqs, B,
                                  Hq // Hkv, 0.125, pool.k_scale, 1.0, 0, np.full(old.shape, 7.0), fp8))


# ------------------------------------------------------- long contexts, captured calls

@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("new", [[1, 2, 1], [30, 40, 1]], ids=["streamed", "tiles and streamed"])
def test_mass_of_long_contexts(cuda_device, new, fp8):
    """Many splits and key tiles, row tiles cut into pieces for many CTAs."""
    seqs = [40000, 9000, 17001]
    check(*mass_of(cuda_device, np.random.default_rng(11), new, seqs, new, seqs, 6, 2, 128, 64, fp8))


@pytest.mark.parametrize("R", [6, 70])
def test_captured_mass_of_e4m3_pools(cuda_device, R):
    """A captured call keeps the mirrors that it was captured with, whatever becomes of the host
    arrays, and follows device lengths up to them; one above its own is flagged and left out."""
    dev, B, Hq, Hkv, D = cuda_device, 16, 8, 2, 64
    rng = np.random.default_rng(R)
    new = [int(x) for x in rng.choice([1, 2, 5, 20], R)]
    seqs = [int(x) for x in rng.integers(200, 400, R)]
    table, qsl, blocks = batch(rng, [n + 16 for n in seqs], new, B, dev)
    pool = make_pool(rng, blocks, Hkv, B, D, True, dev)
    tab, dq, ds = i32(table, dev), i32(qsl, dev), i32(seqs, dev)
    q = torch.zeros((int(qsl[-1]), Hq, D), dtype=torch.bfloat16, device=dev)
    old, out = torch.rand((R, 420), device=dev), torch.zeros((R, 420), device=dev)
    qh, sh = np.array(qsl, np.int32), np.array(seqs, np.int32)
    ws = torch.empty(pa.attention_mass_workspace_size(qh, sh, Hq, Hkv), dtype=torch.uint8, device=dev)

    def call():
        pa.attention_mass(q, old, out, dq, ds, qh, sh, tab, pool, 0.125, decay=0.5, workspace=ws)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        call()
    qh[:], sh[:] = 0, 0
    for turn in range(4):
        some = [int(rng.integers(0, n + 1)) for n in new] if turn else new
        lens = [int(rng.integers(max(a, 1), n + 1)) for a, n in zip(some, seqs)] if turn else list(seqs)
        above = []
        if turn == 3:
            above = [r for r in range(0, R, 5) if some[r]]
            for r in above:
                lens[r] = seqs[r] + 1 + r % 16
        qs = np.cumsum([0] + some)
        dq.copy_(i32(qs, dev))
        ds.copy_(i32(lens, dev))
        q.copy_(torch.from_numpy(rng.standard_normal(tuple(q.shape))).to(dev).bfloat16())
        ws.fill_(0xFF)
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert pa.get_error() == (pa.PA_ERR_DEVICE_BOUNDS if above else pa.PA_OK)
        want, tol = ref.mass(ref.f64(q), ref.cells(pool.k), ref.f64(old), range(R), table, qs.tolist(),
                             lens, B, Hq // Hkv, 0.125, pool.k_scale, 0.5, 0, np.full((R, 420), 7.0),
                             True)
        want[above] = 7.0
        check(ref.f64(out), want, tol)
