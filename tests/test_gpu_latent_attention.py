"""GPU tests of pa_latent_forward (absorbed attention over the paged latent
cache) against the 64-bit reference on the cells' own values.

Tolerance of an output element o = sum_n p_n v_n:
  * p is rounded to bf16 before the product (half a step, relative 2^-8 by the
    count used here) while the sum of p is not: at most 2^-8 sum_n p_n |v_n|;
  * the scores are fp32 sums of bf16 products: for scores of magnitude up to
    S = scale * sum |q||k| the error is below 2^-20 S (576 terms, fp32
    accumulation), and a score error d moves o by at most 2 d sum p |v|;
  * one rounding of o to bf16: 2^-8 |o|.
On E4M3 pools, besides:
  * the latent part of q is hi + lo in E4M3 after a power of two that brings the
    row's maximum to [2^7, 2^8): at most half of E4M3's smallest step, 2^-10, off,
    so 2^-17 of the row's maximum, and a score by scale 2^-17 max|q| sum |c|;
  * the weights p_n s_n are three parts in E5M2, within 2^-9 relative (below the
    count above) or half of its smallest step, 2^-17, where the row's largest
    weight is at least 2^7: 2^-24 max_n(p_n s_n) for every key, on codes v_n / s_n.
The bound below sums these per element, from the reference's own p and v."""
import numpy as np
import pytest
import torch

from paged_kv_cache_143_gb300 import pa
from tests import latent_reference as ref

pytestmark = pytest.mark.gpu


def i32(a, dev):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=dev)


class Batch:
    """A filled cache, its tables and a step's queries. Cells past each
    request's length, and blocks of nobody, stay poisoned with NaN."""

    def __init__(self, seqs, q_lens, H, L, B, fp8, dev, seed=0, mult=1.0, causal=1, spare_rows=0):
        rng = np.random.default_rng(seed)
        self.seqs, self.q_lens, self.H, self.L, self.B = seqs, q_lens, H, L, B
        self.dev, self.causal, self.scale = dev, causal, (128 + 64) ** -0.5
        live = [s if q else 0 for s, q in zip(seqs, q_lens)]
        self.tab, blocks = ref.tables(rng, live, B)
        self.pool = ref.new_pool(pa, blocks, B, L, fp8, dev)
        n = sum(live)
        if n:
            c = torch.from_numpy(rng.standard_normal((n, L)).astype(np.float32)).to(dev).bfloat16()
            kr = torch.from_numpy(rng.standard_normal((n, 64)).astype(np.float32)).to(dev).bfloat16()
            slots = np.concatenate([ref.slots_of(self.tab, r, s, B) for r, s in enumerate(live)])
            pa.write_latent(self.pool, c, kr, torch.from_numpy(slots).to(dev))
        self.qsl = np.cumsum([0] + list(q_lens)).astype(np.int32)
        self.T = int(self.qsl[-1]) + spare_rows
        self.q = torch.from_numpy((rng.standard_normal((self.T, H, L + 64)) * mult).astype(
            np.float32)).to(dev).bfloat16()
        self.out = torch.full((self.T, H, L), 9.0, dtype=torch.bfloat16, device=dev)
        self.ws = torch.full((pa.latent_workspace_size(H, L),), 0xFF, dtype=torch.uint8, device=dev)
        self.seq_dev, self.qsl_dev, self.tab_dev = (i32(seqs, dev), i32(self.qsl, dev),
                                                    i32(self.tab, dev))

    def run(self, out=None, qsl_host=None, seq_host=None, ws=None, stream=None):
        pa.latent_forward(self.q, self.out if out is None else out, self.qsl_dev, self.seq_dev,
                          self.qsl if qsl_host is None else qsl_host,
                          np.array(self.seqs, np.int32) if seq_host is None else seq_host,
                          self.tab_dev, self.pool, self.scale, self.causal,
                          workspace=self.ws if ws is None else ws, stream=stream)
        return self.out if out is None else out

    def check(self, out=None, seqs=None, reqs=None):
        out = self.out if out is None else out
        seqs = self.seqs if seqs is None else seqs
        lat, rot = ref.pool_rows(self.pool)
        p_half = ref.BF16_HALF
        worst = 0.0
        for r in range(len(seqs)) if reqs is None else reqs:
            a, b = self.qsl[r], self.qsl[r + 1]
            if a == b:
                continue
            at = ref.slots_of(self.tab, r, seqs[r], self.B)
            q = ref.f64(self.q[a:b])
            want, p = ref.absorbed(q, lat[at], rot[at], self.scale, self.causal)
            size = np.einsum("thn,nl->thl", p, np.abs(lat[at]))
            k = np.concatenate((lat[at], rot[at]), -1)
            s_mag = self.scale * np.einsum("thd,nd->thn", np.abs(q), np.abs(k)).max(-1)[..., None]
            s_err = 2.0 ** -20 * s_mag
            floor = 0.0
            if self.pool.scales is not None:
                s = ref.f64(self.pool.scales).reshape(-1)[at]
                q_max = np.abs(q[..., :self.L]).max(-1)[..., None]
                s_err = s_err + self.scale * 2.0 ** -17 * q_max * np.abs(lat[at]).sum(-1).max()
                seen = (p > 0).astype(np.float64)
                floor = 2.0 ** -24 * (p * s).max(-1)[..., None] * np.einsum(
                    "thn,nl->thl", seen, np.abs(lat[at]) / s[:, None])
            tol = size * (p_half + 2 * s_err) + floor + p_half * np.abs(want) + 1e-30
            got = ref.f64(out[a:b])
            assert np.isfinite(got).all()
            err = np.abs(got - want)
            assert (err <= tol).all(), (r, err.max(), (err / tol).max())
            worst = max(worst, (err / tol).max())
        return worst


SHAPES = [  # seq_lens, q_lens, H, L, B
    ([1], [1], 1, 512, 16),
    ([1, 63, 64, 65, 127, 128, 129], [1] * 7, 16, 512, 16),
    ([200, 7, 1000], [1, 1, 1], 5, 256, 32),
    ([333, 64, 2049], [1, 1, 1], 32, 512, 64),
    ([90, 400], [1, 1], 40, 512, 16),
    ([511, 3000], [1, 1], 128, 512, 64),
    ([700, 65], [1, 1], 128, 256, 16),
    ([130, 77, 300], [1, 4, 2], 16, 512, 32),      # drafted tokens among decodes
    ([50, 64, 65], [50, 64, 33], 3, 512, 16),      # whole prompts and a chunk
    ([900], [130], 24, 256, 64),                   # many row tiles
    ([40, 10, 70], [1, 0, 1], 4, 512, 16),         # an empty request
    ([5000], [1], 20, 256, 16),                    # one request cut over every CTA
    ([12000, 1, 1, 12000], [1, 1, 1, 3], 64, 512, 64),
    ([17] * 400, [1] * 400, 16, 256, 16),          # more requests than threads
    ([64] * 152 + [1], [1] * 153, 8, 512, 32),
    ([64] * 450, [1] * 450, 40, 256, 64),          # pieces of one tile each
    ([70, 1, 130, 200, 64] * 50, [1, 1, 2, 1, 1] * 50, 24, 256, 32),
]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_shapes(cuda_device, case, fp8):
    seqs, q_lens, H, L, B = SHAPES[case]
    b = Batch(seqs, q_lens, H, L, B, fp8, cuda_device, seed=case)
    b.run()
    assert pa.get_error() == pa.PA_OK
    b.check()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("mult", [0.0, 0.05, 6.0])
def test_flat_and_peaked_scores(cuda_device, mult, fp8):
    """Equal weights, nearly equal ones, and rows that one key owns (the
    reference maximum moves and O is rescaled)."""
    b = Batch([3000, 70, 640], [1, 1, 5], 16, 512, 16, fp8, cuda_device, seed=3, mult=mult)
    b.run()
    assert pa.get_error() == pa.PA_OK
    b.check()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_rising_scores_rescale_every_tile(cuda_device, fp8):
    """Keys that grow along the context: the maximum rises tile after tile."""
    dev = cuda_device
    b = Batch([1500], [2], 24, 256, 16, fp8, dev, seed=4)
    n = 1500
    ramp = torch.linspace(0, 60, n, device=dev)[:, None]
    one = torch.ones(1, 64, device=dev)
    rng = np.random.default_rng(8)
    c = torch.from_numpy(rng.standard_normal((n, 256)).astype(np.float32)).to(dev).bfloat16()
    slots = torch.from_numpy(ref.slots_of(b.tab, 0, n, 16)).to(dev)
    pa.write_latent(b.pool, c, (ramp * one).bfloat16(), slots)
    b.q[..., 256:] = 0.25
    b.run()
    assert pa.get_error() == pa.PA_OK
    b.check()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_one_large_weight_beside_many_small_ones(cuda_device, fp8):
    """A first key that holds a third of the weight, and 20000 others, each
    2^-13 of it and less, that hold the rest."""
    dev = cuda_device
    n = 20000
    b = Batch([n], [1], 16, 512, 16, fp8, dev, seed=14)
    rng = np.random.default_rng(15)
    c = torch.from_numpy(rng.standard_normal((n, 512)).astype(np.float32)).to(dev).bfloat16()
    rope = torch.zeros(n, 64, device=dev)
    rope[0] = 1.0
    pa.write_latent(b.pool, c, rope.bfloat16(), torch.from_numpy(ref.slots_of(b.tab, 0, n, 16)).to(dev))
    b.q.mul_(0.02)
    b.q[..., 512:] = float(np.log(n / 2.0) / 64 / b.scale)
    b.run()
    assert pa.get_error() == pa.PA_OK
    b.check()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_not_causal(cuda_device, fp8):
    b = Batch([100, 64, 7], [30, 1, 7], 6, 512, 16, fp8, cuda_device, seed=5, causal=0)
    b.run()
    assert pa.get_error() == pa.PA_OK
    b.check()


def test_rows_past_the_last_sequence_stay(cuda_device):
    """A padded batch: query_start_loc ends before the rows do (the device
    array; the host mirror sizes the launch for all rows)."""
    dev = cuda_device
    b = Batch([100, 40], [1, 3], 16, 512, 16, False, dev, seed=6, spare_rows=5)
    host = b.qsl.copy()
    host[-1] = b.T  # as planned for a larger step
    b.run(qsl_host=host, seq_host=np.array([100, 64], np.int32))
    assert pa.get_error() == pa.PA_OK
    b.check()
    assert (b.out[4:] == 9).all()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_deterministic_and_independent_of_placement(cuda_device, fp8):
    dev = cuda_device
    b = Batch([777, 2000, 33], [1, 2, 1], 20, 512, 32, fp8, dev, seed=7)
    first = b.run().clone()
    again = b.run(out=torch.empty_like(first))
    assert torch.equal(first.view(torch.int16), again.view(torch.int16))
    perm = torch.from_numpy(np.random.default_rng(1).permutation(b.pool.num_blocks)).to(dev)

    def moved(t):
        if t is None:
            return None
        u = torch.empty_like(t)
        u[perm] = t
        return u

    b.pool = pa.LatentPool(moved(b.pool.latent), moved(b.pool.rope), moved(b.pool.scales))
    b.tab_dev = torch.where(b.tab_dev >= 0, perm[b.tab_dev.clamp(min=0).long()].int(), b.tab_dev)
    third = b.run(out=torch.empty_like(first))
    assert torch.equal(first.view(torch.int16), third.view(torch.int16))
    assert pa.get_error() == pa.PA_OK


def test_captured_call_follows_the_device_lengths(cuda_device):
    """One captured call replayed while the contexts grow (the cache holds the
    longer contexts from the start; the lengths on the device change)."""
    dev = cuda_device
    seqs = [900, 130, 64, 2000]
    b = Batch(seqs, [1] * 4, 16, 512, 16, False, dev, seed=9)
    b.seq_dev.copy_(i32([10, 130, 1, 65], dev))
    b.run(seq_host=np.array([10, 130, 1, 65], np.int32))  # warm: attributes, module
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        b.run(seq_host=np.array([10, 130, 1, 65], np.int32))
    for lens in ([10, 130, 1, 65], [11, 64, 2, 66], [900, 129, 63, 1999], seqs):
        b.seq_dev.copy_(i32(lens, dev))
        b.out.fill_(9.0)
        g.replay()
        torch.cuda.synchronize()
        assert pa.get_error() == pa.PA_OK
        b.check(seqs=lens)


def test_two_streams_with_workspaces_of_their_own(cuda_device):
    dev = cuda_device
    batches = [Batch([3000 + i, 500], [1, 1], 16, 512, 16, False, dev, seed=20 + i)
               for i in range(2)]
    streams = [torch.cuda.Stream() for _ in batches]
    torch.cuda.synchronize()
    for _ in range(10):
        for b, s in zip(batches, streams):
            b.run(stream=s)
    torch.cuda.synchronize()
    for b in batches:
        b.check()
    assert pa.get_error() == pa.PA_OK


def test_cells_past_32_bits_of_bytes(cuda_device):
    """A cache whose request lies more than 2^32 bytes into the pool."""
    dev = cuda_device
    b = Batch([200], [1], 16, 512, 64, False, dev, seed=11)
    far = (1 << 32) // (64 * 512 * 2) + 5
    latent = torch.zeros(far + b.pool.num_blocks, 64, 512, dtype=torch.bfloat16, device=dev)
    rope = torch.zeros(far + b.pool.num_blocks, 64, 64, dtype=torch.bfloat16, device=dev)
    latent[far:], rope[far:] = b.pool.latent, b.pool.rope
    near = b.run().clone()
    b.pool = pa.LatentPool(latent, rope)
    b.tab_dev = torch.where(b.tab_dev >= 0, b.tab_dev + far, b.tab_dev)
    assert torch.equal(b.run(out=torch.empty_like(near)).view(torch.int16), near.view(torch.int16))
    assert pa.get_error() == pa.PA_OK


def test_bad_blocks_and_lengths_are_flagged(cuda_device):
    dev = cuda_device
    b = Batch([100, 40, 64], [1, 1, 2], 16, 256, 16, False, dev, seed=12)
    good = b.run().clone()
    assert pa.get_error() == pa.PA_OK
    tab = b.tab_dev.clone()
    for bad in (b.pool.num_blocks, -1, 1 << 30, -(1 << 31)):
        b.tab_dev = tab.clone()
        b.tab_dev[1, 0] = bad
        b.run()
        assert pa.get_error() == pa.PA_ERR_DEVICE_BOUNDS
    b.tab_dev = tab
    host = np.array(b.seqs, np.int32)
    for r, n in ((0, 10 ** 6), (2, 1), (1, 0), (1, -5)):  # past the table; q_len > seq_len
        b.seq_dev = i32(b.seqs, dev)
        b.seq_dev[r] = n
        b.out.fill_(9.0)
        b.run(seq_host=host)
        assert pa.get_error() == pa.PA_ERR_DEVICE_BOUNDS
        for o in range(3):  # the others are right, the bad one is left alone
            a, e = b.qsl[o], b.qsl[o + 1]
            if o != r:
                b.check(reqs=[o])
            else:
                assert (b.out[a:e] == 9).all()
    b.seq_dev = i32(b.seqs, dev)
    for q in ([0, 1, 2, 5], [-1, 1, 2, 4], [0, 3, 2, 4]):  # rows that leave q
        b.qsl_dev = i32(q, dev)
        b.run()
        assert pa.get_error() == pa.PA_ERR_DEVICE_BOUNDS
    b.qsl_dev = i32(b.qsl, dev)
    assert torch.equal(b.run().view(torch.int16), good.view(torch.int16))
    assert pa.get_error() == pa.PA_OK


@pytest.mark.parametrize("L", [256, 512])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_rows_that_are_not_numbers(cuda_device, fp8, L):
    """A NaN or an infinity in a query makes its own row NaN, whether the row's
    keys are cut over CTAs or not, and no other row changes."""
    b = Batch([5000, 200, 40], [1, 3, 1], 20, L, 16, fp8, cuda_device, seed=21)
    clean = b.run().clone()
    bad = {(0, 3): (5, float("nan")), (1, 7): (L - 1, float("inf")),
           (2, 0): (L + 3, float("nan")), (3, 19): (0, float("nan")),
           (4, 19): (L + 63, float("-inf")), (0, 11): (17, float("-inf"))}
    for (t, h), (d, value) in bad.items():
        b.q[t, h, d] = value
    got = b.run()
    assert pa.get_error() == pa.PA_OK
    for t in range(b.T):
        for h in range(b.H):
            if (t, h) in bad:
                assert torch.isnan(got[t, h]).all(), (t, h)
            else:
                assert torch.equal(got[t, h], clean[t, h]), (t, h)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_a_key_of_infinite_score(cuda_device, fp8):
    """An infinity in a key's rotary part: rows that it scores +inf are NaN, to
    rows that it scores -inf it weighs nothing."""
    b = Batch([3000, 90], [1, 1], 24, 512, 32, fp8, cuda_device, seed=22)
    for r, key in ((0, 1234), (1, 50)):
        slot = int(ref.slots_of(b.tab, r, b.seqs[r], b.B)[key])
        b.pool.rope.view(-1, 64)[slot, 9] = float("inf")
    got = b.run()
    assert pa.get_error() == pa.PA_OK
    up = b.q[:, :, 512 + 9] > 0
    assert torch.isnan(got).all(-1)[up].all()
    assert torch.isfinite(got)[~up].all()


@pytest.mark.parametrize("H,L", [(20, 256), (3, 512), (64, 512)])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_later_tokens_that_are_not_numbers(cuda_device, fp8, H, L):
    """A NaN or an infinity in a chunk's later cells leaves the rows that do not
    see them as they are; rows that see a NaN are NaN."""
    b = Batch([700, 40, 130], [9, 5, 130], H, L, 16, fp8, cuda_device, seed=23)
    clean = b.run().clone()
    first = {}                        # request -> first bad position
    for r, keys in ((0, (697, 699)), (1, (38,)), (2, (64, 65, 100))):
        first[r] = min(keys)
        for i, key in enumerate(keys):
            slot = int(ref.slots_of(b.tab, r, b.seqs[r], b.B)[key])
            cell = b.pool.latent.view(-1, L)[slot]
            if fp8:
                cell[7 + 40 * i] = 0x7F
            else:
                cell[7 + 40 * i] = float("nan") if i != 1 else float("inf")
    got = b.run()
    assert pa.get_error() == pa.PA_OK
    for r in range(3):
        a, n = int(b.qsl[r]), b.q_lens[r]
        hide = first[r] - (b.seqs[r] - n)        # rows before this one do not see it
        assert 0 < hide < n
        assert torch.equal(got[a:a + hide].view(torch.int16), clean[a:a + hide].view(torch.int16))
        assert torch.isnan(got[a + hide:a + n]).any(-1).all()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_starts_that_claim_more_than_32_bits_of_work(cuda_device, fp8):
    """Device starts 0, T, 0, T, ..: half of the requests claim every row, each a
    valid request by itself, and their passes together more key tiles than 32 bits
    hold. The call is flagged and writes nothing."""
    dev = cuda_device
    T, H, L, B, R, ctx = 2048, 128, 256, 64, 1024, 1 << 18
    # tiles of 64 rows and 64 keys, the rows' two by two
    assert (R // 2) * (T * H // 64 // 2) * (ctx // 64) > 2 ** 31
    pool = ref.new_pool(pa, 2, B, L, fp8, dev, poison=False)
    q = torch.zeros(T, H, L + 64, dtype=torch.bfloat16, device=dev)
    out = torch.full((T, H, L), 9.0, dtype=torch.bfloat16, device=dev)
    table = torch.zeros(R, ctx // B, dtype=torch.int32, device=dev)
    host = np.arange(R + 1, dtype=np.int32) * (T // R)
    seq = np.full(R, ctx, np.int32)
    ws = torch.empty(pa.latent_workspace_size(H, L), dtype=torch.uint8, device=dev)
    starts = i32([0, T] * (R // 2) + [0], dev)
    pa.latent_forward(q, out, starts, i32(seq, dev), host, seq, table, pool, 0.1, workspace=ws)
    assert pa.get_error() == pa.PA_ERR_DEVICE_BOUNDS
    assert (out == 9).all()


def check_with_infinite_cells(b):
    """b.out against the formula with its infinities (bf16 cells): a row is NaN where
    a visible score is NaN or +inf or all are -inf; a key of score -inf weighs 0, and
    0 times an element of it that is not finite is NaN. The rest within Batch.check's
    tolerance, from the finite cells."""
    lat, rot = ref.pool_rows(b.pool)
    for r in range(len(b.seqs)):
        at = ref.slots_of(b.tab, r, b.seqs[r], b.B)
        c, kr = lat[at], rot[at]
        k = np.concatenate((c, kr), -1)
        for j in range(b.q_lens[r]):
            t = int(b.qsl[r]) + j
            n = b.seqs[r] - b.q_lens[r] + j + 1 if b.causal else b.seqs[r]
            q = ref.f64(b.q[t])
            with np.errstate(invalid="ignore"):
                x = q @ k[:n].T * b.scale
                row_nan = np.isnan(x).any(-1) | (x == np.inf).any(-1) | (x == -np.inf).all(-1)
            good = np.isfinite(k[:n]).all(-1)
            dims = ~np.isfinite(c[:n]).all(0)          # where some visible cell is not finite
            got = ref.f64(b.out[t])
            want_nan = row_nan[:, None] | dims[None]
            np.testing.assert_array_equal(np.isnan(got), want_nan, err_msg=f"token {t}")
            p = ref.softmax_rows(np.where(np.isfinite(x) & good, x, -np.inf))
            v = np.where(good[:, None], c[:n], 0.0)
            want, size = p @ v, p @ np.abs(v)
            s_mag = b.scale * (np.abs(q)[:, :] @ np.abs(np.where(good[:, None], k[:n], 0.0)).T
                               ).max(-1, keepdims=True)
            tol = size * (ref.BF16_HALF + 2 * 2.0 ** -20 * s_mag) + ref.BF16_HALF * np.abs(want)
            err = np.abs(np.where(want_nan, 0.0, got - want))
            assert (err <= tol + 1e-30).all(), (t, (err / (tol + 1e-30)).max())


@pytest.mark.parametrize("where", ["hidden", "seen"])
@pytest.mark.parametrize("H,L,seqs,q_lens", [
    (20, 256, [700, 40, 130], [9, 5, 130]), (3, 512, [700, 40, 130], [9, 5, 130]),
    (64, 512, [300, 5000], [7, 4]), (16, 512, [20000], [3])])
def test_an_infinite_element_of_either_score(cuda_device, H, L, seqs, q_lens, where):
    """One infinite element in a cell, its scores +inf and -inf by the queries' signs:
    the same result whether the tile also holds keys that some rows hide or not."""
    b = Batch(seqs, q_lens, H, L, 16, False, cuda_device, seed=24)
    for r, n in enumerate(q_lens):
        key = b.seqs[r] - n + (n // 2 if where == "hidden" else 0) - (where == "seen")
        slot = int(ref.slots_of(b.tab, r, b.seqs[r], b.B)[key])
        b.pool.latent.view(-1, L)[slot, 130 + r] = float("inf") if r != 1 else float("-inf")
    b.run()
    assert pa.get_error() == pa.PA_OK
    check_with_infinite_cells(b)


@pytest.mark.parametrize("L", [256, 512])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_scores_of_minus_infinity_alone(cuda_device, fp8, L):
    """A row whose query holds an infinity that scores every visible key -inf is NaN,
    as the softmax of such scores is, whether its keys are cut over CTAs or not."""
    b = Batch([5000, 200, 1], [1, 3, 1], 20, L, 16, fp8, cuda_device, seed=25)
    b.pool.rope[..., 7] = b.pool.rope[..., 7].abs() + 0.01      # (NaN cells stay NaN)
    clean = b.run().clone()
    bad = ((0, 3), (1, 7), (3, 19), (4, 0))
    for t, h in bad:
        b.q[t, h, L + 7] = float("-inf")
    got = b.run()
    assert pa.get_error() == pa.PA_OK
    for t in range(b.T):
        for h in range(b.H):
            if (t, h) in bad:
                assert torch.isnan(got[t, h]).all(), (t, h)
            else:
                assert torch.equal(got[t, h], clean[t, h]), (t, h)


@pytest.mark.parametrize("seqs", [[20000], [5000, 7000], [300] * 160], ids=["one", "two", "many"])
def test_pieces_of_minus_infinity_scores(cuda_device, seqs):
    """Requests whose first half scores -inf: it weighs nothing, but an infinite
    element among it is 0 times infinity, a NaN, in its dim; cut over CTAs and joined."""
    b = Batch(seqs, [1] * len(seqs), 16, 512, 16, False, cuda_device, seed=26)
    b.q[..., 512 + 7] = -b.q[..., 512 + 7].abs() - 0.01
    for r, n in enumerate(seqs):
        slots = torch.from_numpy(ref.slots_of(b.tab, r, n // 2, b.B)).to(cuda_device)
        b.pool.rope.view(-1, 64)[slots, 7] = float("inf")
        cell = b.pool.latent.view(-1, 512)[int(slots[n // 5])]
        cell[99] = -float("inf")
        b.q[r, :, 99] = b.q[r, :, 99].abs() + 0.01
    b.run()
    assert pa.get_error() == pa.PA_OK
    check_with_infinite_cells(b)


@pytest.mark.parametrize("H,L", [(20, 256), (3, 512), (64, 512)])
def test_later_scales_that_are_not_numbers(cuda_device, H, L):
    """A NaN or an infinity as the scale of a chunk's later E4M3 cell leaves the rows
    that do not see it as they are; rows that see a NaN are NaN."""
    b = Batch([700, 40, 130], [9, 5, 130], H, L, 16, True, cuda_device, seed=27)
    clean = b.run().clone()
    first = {}
    for r, keys in ((0, (697, 699)), (1, (38,)), (2, (64, 65, 100))):
        first[r] = min(keys)
        for i, key in enumerate(keys):
            slot = int(ref.slots_of(b.tab, r, b.seqs[r], b.B)[key])
            b.pool.scales.view(-1)[slot] = float("nan") if i != 1 else float("inf")
    got = b.run()
    assert pa.get_error() == pa.PA_OK
    for r in range(3):
        a, n = int(b.qsl[r]), b.q_lens[r]
        hide = first[r] - (b.seqs[r] - n)        # rows before this one do not see it
        assert torch.equal(got[a:a + hide].view(torch.int16), clean[a:a + hide].view(torch.int16))
        assert torch.isnan(got[a + hide:a + n]).all()


@pytest.mark.parametrize("H,L", [(20, 256), (16, 512), (64, 512)])
@pytest.mark.parametrize("power", [105, -80])
def test_small_queries_on_large_cells(cuda_device, H, L, power):
    """E4M3 cells near the ends of the scales' range and queries as far the other way:
    ordinary scores, whose query parts keep their bits."""
    b = Batch([5, 9, 3, 200, 64], [1, 2, 1, 1, 4], H, L, 16, True, cuda_device, seed=28)
    rng = np.random.default_rng(29)
    for r, n in enumerate(b.seqs):
        c = torch.from_numpy(rng.standard_normal((n, L)) * 2.0 ** power).to(cuda_device).bfloat16()
        kr = torch.from_numpy(rng.standard_normal((n, 64))).to(cuda_device).bfloat16()
        pa.write_latent(b.pool, c, kr, torch.from_numpy(ref.slots_of(b.tab, r, n, b.B)).to(cuda_device))
    b.q[..., :L] *= 2.0 ** -power
    b.run()
    assert pa.get_error() == pa.PA_OK
    b.check()
