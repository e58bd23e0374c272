"""Attention to a part of a cache, host side (no GPU): refusals before any
launch, the workspace's size, the binding's checks, and the references' own
pins."""
import ctypes

import numpy as np
import pytest
import torch

from paged_kv_cache_143_gb300 import pa
from tests import partial_reference as ref

P = 16  # a fake, aligned device pointer: the calls return before touching it


def kv_pool(**kw):
    d = dict(k_pool=P, v_pool=P, num_blocks=4, block_size=16, num_kv_heads=2, head_dim=128,
             dtype=0, k_scale=1.0, v_scale=1.0)
    d.update(kw)
    return ctypes.byref(pa._Pool(*[d[n] for n, _ in pa._Pool._fields_]))


def host(a):
    return pa._np_addr(a)


def calls():
    """Each call with arguments that pass its host checks but for no work."""
    L = pa.lib()
    qsl, seqs = np.array([0, 1], np.int32), np.array([5], np.int32)

    def bounds(pool=None, bounds=P, qsl=P, seqs=P, tab=P, mb=1, R=1, T=1):
        return L.pa_update_block_bounds(pool or kv_pool(), bounds, qsl, seqs, tab, mb, R, T, None)

    def scores(pool=None, q=P, bounds=P, out=P, qsl=P, seqs=P, tab=P, mb=1, R=1, T=1, Hq=4):
        return L.pa_score_blocks(q, bounds, out, qsl, seqs, tab, mb, R, T, Hq, pool or kv_pool(),
                                 None)

    def sparse(pool=None, q=P, out=P, qsl=P, seqs=P, tab=P, mb=1, R=1, T=1, Hq=4, sel=P, k=2):
        return L.pa_sparse_forward(q, out, qsl, seqs, tab, mb, R, T, Hq, sel, k,
                                   pool or kv_pool(), 0.1, None)

    def mass(pool=None, q=P, a=P, b=P, stride=5, rows=1, qsl_d=P, seqs_d=P, qh=qsl, sh=seqs, tab=P,
             mb=1, R=1, T=1, Hq=4, window=0, ws=P, n=1 << 30):
        return L.pa_attention_mass(q, a, b, stride, rows, None, qsl_d, seqs_d,
                                   None if qh is None else host(qh),
                                   None if sh is None else host(sh), tab, mb, R, T, Hq,
                                   pool or kv_pool(), 0.1, 1.0, window, ws, n, None)

    def compact(pool=None, src=P, mb=1, dst=P, db=1, kept=P, k=2, lens=P, R=1, a=None, b=None,
                stride=0, rows=0):
        return L.pa_compact_cache(pool or kv_pool(), src, mb, dst, db, kept, k, lens, R, a, b,
                                  stride, rows, None, None)

    return dict(bounds=bounds, scores=scores, sparse=sparse, mass=mass, compact=compact)


@pytest.mark.parametrize("name", ["bounds", "scores", "sparse", "mass", "compact"])
@pytest.mark.parametrize("kw,status", [
    (dict(k_pool=None), pa.PA_ERR_INVALID), (dict(v_pool=24), pa.PA_ERR_INVALID),
    (dict(num_blocks=-1), pa.PA_ERR_INVALID), (dict(num_kv_heads=0), pa.PA_ERR_INVALID),
    (dict(head_dim=96), pa.PA_ERR_UNSUPPORTED), (dict(block_size=24), pa.PA_ERR_UNSUPPORTED),
    (dict(dtype=2), pa.PA_ERR_UNSUPPORTED), (dict(dtype=1, k_scale=0.0), pa.PA_ERR_INVALID)])
def test_pool_refusals(name, kw, status):
    assert calls()[name](pool=kv_pool(**kw)) == status


def test_call_refusals():
    c = calls()
    I, U = pa.PA_ERR_INVALID, pa.PA_ERR_UNSUPPORTED
    for bad in (dict(R=-1), dict(T=-1), dict(mb=-1), dict(bounds=None), dict(bounds=24),
                dict(seqs=None), dict(tab=None)):
        assert c["bounds"](**bad) == I, bad
    assert c["bounds"](R=0) == c["bounds"](T=0) == c["bounds"](mb=0) == pa.PA_OK
    for bad in (dict(R=-1), dict(T=-1), dict(mb=-1), dict(q=None), dict(q=24), dict(bounds=None),
                dict(bounds=8), dict(out=None), dict(out=18), dict(qsl=None), dict(seqs=None),
                dict(tab=None), dict(Hq=0), dict(Hq=5)):
        assert c["scores"](**bad) == I, bad
    assert c["scores"](Hq=130) == U
    assert c["scores"](T=0) == c["scores"](R=0) == c["scores"](mb=0) == pa.PA_OK
    for bad in (dict(R=-1), dict(T=-1), dict(mb=-1), dict(mb=0), dict(q=None), dict(q=24),
                dict(out=None), dict(out=8), dict(qsl=None), dict(seqs=None), dict(tab=None),
                dict(Hq=0), dict(Hq=5), dict(sel=None), dict(k=0), dict(pool=kv_pool(num_blocks=0))):
        assert c["sparse"](**bad) == I, bad
    assert c["sparse"](T=0) == c["sparse"](R=0) == pa.PA_OK
    arr = lambda *x: np.array(x, np.int32)
    for bad in (dict(R=-1), dict(T=-1), dict(mb=-1), dict(q=None), dict(q=24), dict(a=None),
                dict(b=None), dict(a=18), dict(b=17), dict(stride=-1), dict(stride=4), dict(rows=-1),
                dict(qsl_d=None), dict(seqs_d=None), dict(qh=None), dict(sh=None), dict(tab=None),
                dict(mb=0), dict(Hq=0), dict(Hq=5), dict(window=-1), dict(ws=None), dict(ws=24),
                dict(n=0), dict(qh=arr(0, 2)), dict(qh=arr(1, 1)), dict(sh=arr(0)),
                dict(sh=arr(17)), dict(pool=kv_pool(num_blocks=0))):
        assert c["mass"](**bad) == I, bad
    assert c["mass"](T=0, qh=arr(0, 0)) == c["mass"](R=0) == pa.PA_OK
    for bad in (dict(R=-1), dict(mb=-1), dict(db=-1), dict(k=-1), dict(src=None), dict(dst=None),
                dict(kept=None), dict(lens=None), dict(a=P), dict(b=P), dict(a=P, b=18),
                dict(a=P, b=P, stride=-1), dict(a=P, b=P, rows=-1)):
        assert c["compact"](**bad) == I, bad
    assert c["compact"](R=65536) == U
    assert c["compact"](R=0) == c["compact"](k=0) == pa.PA_OK


def test_selection_refusals():
    L = pa.lib()

    def blocks(x=P, qsl=P, seqs=P, R=1, T=1, H=1, mb=4, B=16, first=1, last=1, k=2, out=P):
        return L.pa_select_blocks(x, qsl, seqs, R, T, H, mb, B, first, last, k, out, None)

    def tokens(x=P, stride=4, rows=1, seqs=P, R=1, first=1, last=1, k=2, out=P, lens=P):
        return L.pa_select_tokens(x, stride, rows, None, seqs, R, first, last, k, out, lens, None)

    for bad in (dict(R=-1), dict(T=-1), dict(H=0), dict(mb=-1), dict(B=0), dict(first=-1),
                dict(last=-1), dict(k=0), dict(k=1), dict(x=None), dict(x=18), dict(qsl=None),
                dict(seqs=None), dict(out=None), dict(first=2 ** 31 - 1, last=2 ** 31 - 1)):
        assert blocks(**bad) == pa.PA_ERR_INVALID, bad
    assert blocks(T=0) == blocks(R=0) == pa.PA_OK
    assert blocks(T=2 ** 30, H=8) == pa.PA_ERR_UNSUPPORTED
    for bad in (dict(R=-1), dict(rows=-1), dict(stride=-1), dict(stride=2 ** 31), dict(first=-1),
                dict(last=-1), dict(k=0), dict(k=1), dict(x=None), dict(x=17), dict(seqs=None),
                dict(out=None), dict(lens=None)):
        assert tokens(**bad) == pa.PA_ERR_INVALID, bad
    assert tokens(R=0) == pa.PA_OK


def test_mass_workspace():
    """Room for the scores of short steps and for the tiles of long ones; 0 where the
    mirrors make no batch."""
    size = pa.attention_mass_workspace_size
    assert size([0, 1], [1000], 8, 2) >= 8 * 1008 * 4
    assert size([0, 1, 2], [1000, 500], 8, 2) > size([0, 1], [1000], 8, 2)
    rows = 64 * 8
    assert size([0, 64], [1000], 8, 2) >= rows * 128 * 2
    assert size([0, 64], [1000], 8, 2, window=4) < size([0, 64], [1000], 8, 2, window=16)
    assert size([0, 0], [1000], 8, 2) == 0
    assert size([0, 5], [4], 8, 2) == 0 and size([0, 5], [9], 7, 2) == 0
    with pytest.raises(ValueError):
        size([0, 1], [5, 6], 8, 2)


def test_binding_wants_gpu_tensors():
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    b = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    f = lambda *s: torch.zeros(s)
    pool = pa.KVPool(b(4, 2, 16, 64), b(4, 2, 16, 64))
    for call in (
            lambda: pa.update_block_bounds(pool, b(4, 2, 2, 64), i(1, 2), i(1)),
            lambda: pa.score_blocks(b(1, 4, 64), b(4, 2, 2, 64), f(1, 2, 2), i(2), i(1), i(1, 2),
                                    pool),
            lambda: pa.select_blocks(f(1, 2, 3), i(1, 2, 4), i(2), i(1), 16),
            lambda: pa.sparse_forward(b(1, 4, 64), b(1, 4, 64), i(2), i(1), i(1, 2), i(1, 2, 3),
                                      pool, 1.0),
            lambda: pa.attention_mass(b(1, 4, 64), f(1, 9), f(1, 9), i(2), i(1), [0, 1], [5],
                                      i(1, 2), pool, 1.0),
            lambda: pa.select_tokens(f(1, 9), i(1, 100), i(1), i(1)),
            lambda: pa.compact_cache(pool, i(1, 2), i(1, 2), i(1, 9), i(1))):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for call in (
            lambda: pa.update_block_bounds(pool, b(4, 2, 64), i(1, 2), i(1)),
            lambda: pa.update_block_bounds(pool, b(4, 2, 2, 64), i(2, 2), i(1)),
            lambda: pa.update_block_bounds(pool, b(4, 2, 2, 64), i(1, 2), i(1),
                                           query_start_loc=i(2)),
            lambda: pa.score_blocks(b(1, 4, 64), b(4, 2, 2, 64), f(1, 2, 3), i(2), i(1), i(1, 2),
                                    pool),
            lambda: pa.select_blocks(f(1, 2, 3), i(2, 2, 4), i(2), i(1), 16),
            lambda: pa.select_blocks(f(1, 2, 3), i(1, 2, 4), i(3), i(1), 16),
            lambda: pa.sparse_forward(b(1, 4, 64), b(1, 4, 64), i(2), i(1), i(1, 2), i(1, 1, 3),
                                      pool, 1.0),
            lambda: pa.attention_mass(b(1, 4, 64), f(1, 9), f(1, 8), i(2), i(1), [0, 1], [5],
                                      i(1, 2), pool, 1.0),
            lambda: pa.attention_mass(b(1, 4, 64), f(1, 9), f(1, 9), i(2), i(1), [0, 1], [5, 6],
                                      i(1, 2), pool, 1.0),
            lambda: pa.select_tokens(f(1, 9), i(2, 100), i(1), i(1)),
            lambda: pa.select_tokens(f(1, 9), i(2, 100), i(2), i(2)),
            lambda: pa.compact_cache(pool, i(1, 2), i(1, 2), i(1, 9), i(1), mass_in=f(1, 9)),
            lambda: pa.compact_cache(pool, i(1, 2), i(2, 2), i(1, 9), i(1))):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------- pins of the references

def test_reference_codes():
    c = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(c).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.e4m3(c), want, equal_nan=True)


def test_reference_scores_are_reached():
    """The most that the box allows: no key of the block exceeds it, and the corner
    that the signs of q choose reaches it."""
    rng = np.random.default_rng(0)
    k = rng.standard_normal((3, 2, 16, 8))
    bnd = ref.bounds(k, [[0, 2]], None, [30], 16, np.zeros((3, 2, 2, 8)))
    q = rng.standard_normal((1, 4, 8))
    s, _ = ref.scores(q, bnd, [[0, 2]], [0, 1], [30], 16, 2, 1.0, np.zeros((1, 2, 2)))
    for h in range(2):
        for i, b in enumerate((0, 2)):
            keys = k[b, h][: 16 if i == 0 else 14]
            dots = keys @ q[0, 2 * h:2 * h + 2].T
            corner = np.where(q[0, 2 * h:2 * h + 2] > 0, bnd[b, h, 1], bnd[b, h, 0])
            best = (corner * q[0, 2 * h:2 * h + 2]).sum(-1).max()
            assert dots.max() <= s[0, h, i] + 1e-12 and abs(best - s[0, h, i]) < 1e-12


def test_reference_attention_and_mass_agree_with_dense():
    """All blocks listed: causal attention by torch; the mass of every query is the
    column sum of the same weights."""
    rng = np.random.default_rng(1)
    B, n, new, D, g = 16, 37, 5, 8, 2
    k, v = rng.standard_normal((2, 4, 1, B, D))
    table, qsl = [[2, 0, 3]], [0, new]
    q = rng.standard_normal((new, g, D))
    K, V = (torch.from_numpy(ref.context(x, table[0], n, B, 0)) for x in (k, v))
    x = torch.from_numpy(q) @ K.T * 0.3                                  # [new][g][n]
    x = x.masked_fill(torch.arange(n) > (n - new + torch.arange(new))[:, None, None], -np.inf)
    w = torch.softmax(x, -1)
    out, _ = ref.sparse(q, k, v, table, np.tile([1, 2, 0], (new, 1, 1)), qsl, [n], B, g, 0.3, 1.0,
                        1.0, False)
    assert np.abs(out - (w @ V).numpy()).max() < 1e-12
    old = rng.random((1, 40))
    for window in (0, 3):
        got, _ = ref.mass(q, k, old, [0], table, qsl, [n], B, g, 0.3, 1.0, 0.5, window,
                          np.zeros((1, 40)), False)
        want = w[-(window or new):].sum((0, 1)).numpy()
        want[: n - new] += 0.5 * old[0, : n - new]
        assert np.abs(got[0, :n] - want).max() < 1e-12 and (got[0, n:] == 0).all()


def test_reference_pick():
    x = np.array([3.0, 1.0, 3.0, np.nan, 2.0, -0.0, 0.0])
    assert ref.pick(x, 7, 0, 0, 3).tolist() == [0, 2, 3]
    assert ref.pick(x, 7, 0, 0, 2).tolist() == [0, 3]
    assert ref.pick(x, 7, 2, 1, 4).tolist() == [0, 1, 3, 6]
    assert ref.pick(x, 3, 0, 0, 5).tolist() == [0, 1, 2, -1, -1]
    assert ref.pick(x[5:], 2, 0, 0, 1).tolist() == [0]


def test_lengths_at_the_end_of_int32():
    """Lists of almost 2^31 entries, which loops over them would leave, are refused."""
    U, most = pa.PA_ERR_UNSUPPORTED, 2 ** 31 - 1
    L, c = pa.lib(), calls()
    assert L.pa_select_blocks(P, P, P, 1, 1, 1, 4, 16, 1, 1, most, P, None) == U
    assert L.pa_select_tokens(P, 4, 1, None, P, 1, 1, 1, most, P, P, None) == U
    assert c["compact"](k=most) == U
    seqs = np.array([most], np.int32)
    assert c["mass"](sh=seqs, mb=2 ** 27, stride=2 ** 31) == U
    assert pa.attention_mass_workspace_size([0, 1], seqs, 4, 2) == 0
