"""GPU tests of pa_latent_prefill (expanded attention) against the 64-bit
reference. The tolerance is that of the absorbed form's tests: half a bf16 step
of every softmax weight and of the output, and the fp32 scores' error."""
import numpy as np
import pytest
import torch

from paged_kv_cache_143_gb300 import pa
from tests import latent_reference as ref

pytestmark = pytest.mark.gpu

DN, DR, DV = 128, 64, 128


def i32(a, dev):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=dev)


class Chunks:
    def __init__(self, q_lens, k_lens, H, dev, seed=0, mult=1.0, causal=1, spare=0, split=True):
        rng = np.random.default_rng(seed)

        def rand(*shape, m=1.0):
            x = rng.standard_normal(shape, dtype=np.float32) * np.float32(m)
            return torch.from_numpy(x).to(dev).bfloat16()

        self.q_lens, self.k_lens, self.H, self.causal = q_lens, k_lens, H, causal
        self.qsl, self.ksl = (np.cumsum([0] + list(x)).astype(np.int32) for x in (q_lens, k_lens))
        T, Tk = int(self.qsl[-1]) + spare, int(self.ksl[-1]) + spare
        self.q = rand(T, H, DN + DR, m=mult)
        kv = rand(Tk, H, DN + DV)
        self.k, self.v = (kv[..., :DN], kv[..., DN:])
        if not split:
            self.k, self.v = self.k.contiguous(), self.v.contiguous()
        self.kr = rand(Tk, DR)
        self.scale = (DN + DR) ** -0.5
        self.out = torch.full((T, H, DV), 9.0, dtype=torch.bfloat16, device=dev)
        self.qsl_dev, self.ksl_dev = i32(self.qsl, dev), i32(self.ksl, dev)
        # the mirrors plan for every row of the buffers, the spare ones too
        self.qsl_host, self.ksl_host = self.qsl.copy(), self.ksl.copy()
        self.qsl_host[-1] += spare
        self.ksl_host[-1] += spare

    def run(self):
        pa.latent_prefill(self.q, self.k, self.kr, self.v, self.out, self.qsl_dev, self.ksl_dev,
                          self.qsl_host, self.ksl_host, self.scale, self.causal)
        return self.out

    def check(self, reqs=None, rows=None):
        for r in range(len(self.q_lens)) if reqs is None else reqs:
            a, b, c, d = self.qsl[r], self.qsl[r + 1], self.ksl[r], self.ksl[r + 1]
            if a == b:
                continue
            q = ref.f64(self.q[a:b])
            k, kr, v = ref.f64(self.k[c:d]), ref.f64(self.kr[c:d]), ref.f64(self.v[c:d])
            want, p = ref.expanded(q, k, kr, v, self.scale, self.causal)
            size = np.einsum("thn,nhd->thd", p, np.abs(v))
            s_mag = np.zeros((b - a, self.H, 1))
            if d > c:
                s_mag = self.scale * (
                    np.einsum("thd,nhd->thn", np.abs(q[..., :DN]), np.abs(k))
                    + np.einsum("thd,nd->thn", np.abs(q[..., DN:]), np.abs(kr))).max(-1)[..., None]
            tol = size * (ref.BF16_HALF + 2 * 2.0 ** -20 * s_mag) + ref.BF16_HALF * np.abs(want)
            got = ref.f64(self.out[a:b])
            assert np.isfinite(got).all()
            err = np.abs(got - want)
            assert (err <= tol + 1e-30).all(), (r, err.max(), (err / (tol + 1e-30)).max())


SHAPES = [  # q_lens, k_lens, H
    ([1], [1], 1),
    ([1, 1, 1], [1, 128, 1000], 3),
    ([127, 128, 129, 255, 256, 257], [127, 128, 129, 255, 256, 257], 2),
    ([64, 300], [64 + 500, 300 + 77], 5),
    ([5, 0, 130], [40, 9, 130], 4),
    ([700], [2100], 2),
    ([33, 520], [33, 520], 16),
    ([2] * 70, [3] * 70, 1),
    # few units, split along their keys over a cluster of CTAs
    ([5], [3000], 1),
    ([40, 3], [2000, 9000], 2),
    ([300], [5000], 1),
    ([1, 2, 130], [4000, 10, 700], 3),
    ([1500], [1450], 1),
    ([257, 1], [2300, 1100], 8),
]


@pytest.mark.parametrize("causal", [1, 0])
@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_shapes(cuda_device, case, causal):
    q, k, H = SHAPES[case]
    b = Chunks(q, k, H, cuda_device, seed=case, causal=causal)
    b.run()
    assert pa.get_error() == pa.PA_OK
    b.check()


@pytest.mark.parametrize("mult", [0.0, 8.0])
def test_flat_and_peaked_scores(cuda_device, mult):
    b = Chunks([200, 300], [900, 300], 2, cuda_device, seed=1, mult=mult)
    b.run()
    b.check()


def test_rows_without_a_visible_key_are_zero(cuda_device):
    """Fewer keys than queries: the first queries see nothing; a request
    without keys is all zeros."""
    for causal in (1, 0):
        b = Chunks([300, 40, 200], [100, 0, 200], 3, cuda_device, seed=2, causal=causal)
        b.run()
        assert pa.get_error() == pa.PA_OK
        b.check()
        assert (b.out[300:340] == 0).all()
        if causal:
            assert (b.out[:200] == 0).all()
    empty = Chunks([7], [0], 2, cuda_device, seed=2)  # no key at all
    empty.run()
    assert pa.get_error() == pa.PA_OK and (empty.out == 0).all()


def test_foreign_rows_may_hold_nan(cuda_device):
    """Keys and values of other requests, and rows past the last request,
    never reach a request's rows."""
    dev = cuda_device
    b = Chunks([90, 150, 64], [90, 150 + 33, 64], 2, dev, seed=3, spare=40)
    b.run()
    want = b.out[90:240].clone()
    nan = float("nan")
    for t in (b.k, b.v, b.kr):
        t[:90] = nan
        t[90 + 183:] = nan
    b.out.fill_(9.0)
    b.run()
    assert pa.get_error() == pa.PA_OK
    assert torch.equal(b.out[90:240].view(torch.int16), want.view(torch.int16))
    assert (b.out[304:] == 9).all()  # rows past the last sequence stay
    b.check(reqs=[1])


def test_strides(cuda_device):
    """Contiguous keys and values, heads outside tokens, a padded query row."""
    dev = cuda_device
    b = Chunks([130, 20], [200, 50], 4, dev, seed=4)
    want = b.run().clone()
    for form in ("contiguous", "heads_outside"):
        k, v, q, kr = b.k, b.v, b.q, b.kr
        if form == "contiguous":
            k, v = k.contiguous(), v.contiguous()
            q = torch.nn.functional.pad(q, (0, 8))[..., :192]
            kr = torch.nn.functional.pad(kr, (0, 16))[..., :64]
        else:
            k, v, q = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (k, v, q))
        out = torch.empty_like(want)
        pa.latent_prefill(q, k, kr, v, out, b.qsl_dev, b.ksl_dev, b.qsl, b.ksl, b.scale)
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    assert pa.get_error() == pa.PA_OK
    bad = torch.zeros(b.k.shape[0], 4, DN + 4, dtype=torch.bfloat16, device=dev)[..., :DN]
    with pytest.raises(pa.PaError):
        pa.latent_prefill(b.q, bad, b.kr, b.v, out, b.qsl_dev, b.ksl_dev, b.qsl, b.ksl, b.scale)


def test_more_units_than_the_list_holds(cuda_device):
    """1100 one-token requests: the grid walks every request."""
    n = 1100
    b = Chunks([1] * n, [2] * n, 1, cuda_device, seed=5)
    b.run()
    assert pa.get_error() == pa.PA_OK
    b.check(reqs=range(0, n, 37))


def test_deterministic(cuda_device):
    b = Chunks([400, 31], [1000, 31], 3, cuda_device, seed=6)
    first = b.run().clone()
    assert torch.equal(b.run().view(torch.int16), first.view(torch.int16))


def test_captured_and_on_another_stream(cuda_device):
    b = Chunks([140, 31], [500, 31], 3, cuda_device, seed=7)
    first = b.run().clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        b.run()
    b.out.fill_(9.0)
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(b.out.view(torch.int16), first.view(torch.int16))
    assert pa.get_error() == pa.PA_OK


def test_device_starts_that_disagree_are_flagged(cuda_device):
    dev = cuda_device
    b = Chunks([300, 40], [300, 40], 2, dev, seed=8)
    good = b.run().clone()
    assert pa.get_error() == pa.PA_OK
    for q, k in (([0, 300, 341], None), ([0, 30, 340], None), ([0, -1, 340], None),
                 (None, [0, 300, 341]), (None, [0, 400, 340]), (None, [-3, 300, 340])):
        b.qsl_dev = i32(b.qsl if q is None else q, dev)
        b.ksl_dev = i32(b.ksl if k is None else k, dev)
        b.run()
        assert pa.get_error() == pa.PA_ERR_DEVICE_BOUNDS, (q, k)
    b.qsl_dev, b.ksl_dev = i32(b.qsl, dev), i32(b.ksl, dev)
    assert torch.equal(b.run().view(torch.int16), good.view(torch.int16))
    assert pa.get_error() == pa.PA_OK


def test_rows_that_are_not_numbers(cuda_device):
    """A NaN or an infinity in a query makes its own row NaN, and no other row
    changes."""
    c = Chunks([200, 3], [500, 40], 2, cuda_device, seed=31)
    clean = c.run().clone()
    bad = {(0, 0): (5, float("nan")), (150, 1): (DN + 2, float("inf")), (202, 0): (DN, float("nan"))}
    for (t, h), (d, value) in bad.items():
        c.q[t, h, d] = value
    got = c.run()
    assert pa.get_error() == pa.PA_OK
    for t in range(203):
        for h in range(2):
            if (t, h) in bad:
                assert torch.isnan(got[t, h]).all(), (t, h)
            else:
                assert torch.equal(got[t, h], clean[t, h]), (t, h)


def test_split_units_captured_flagged_and_beside_nan(cuda_device):
    """Units that a cluster of CTAs shares: replayed from a graph, with device
    starts that disagree, and with NaN in every row of nobody."""
    dev = cuda_device
    b = Chunks([30, 70], [2500, 1300], 2, dev, seed=41, spare=50)
    first = b.run().clone()
    b.check()
    for t in (b.k, b.v, b.kr):
        t[b.ksl[-1]:] = float("nan")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        b.run()
    b.out.fill_(9.0)
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    assert pa.get_error() == pa.PA_OK
    assert torch.equal(b.out[:100].view(torch.int16), first[:100].view(torch.int16))
    assert (b.out[100:] == 9).all()
    for q, k in (([0, 30, 151], None), ([0, -1, 100], None), (None, [0, 2500, 3851]),
                 (None, [0, 3900, 3800])):
        b.qsl_dev = i32(b.qsl if q is None else q, dev)
        b.ksl_dev = i32(b.ksl if k is None else k, dev)
        b.run()
        assert pa.get_error() == pa.PA_ERR_DEVICE_BOUNDS, (q, k)


def test_later_keys_that_are_not_numbers(cuda_device):
    """NaN and infinities in a chunk's later keys and values leave the rows that do
    not see them as they are, whole units and split ones alike."""
    for q_lens, k_lens, H in (([300, 70], [420, 70], 3), ([40], [3000], 1)):
        b = Chunks(q_lens, k_lens, H, cuda_device, seed=51)
        clean = b.run().clone()
        for r, n in enumerate(q_lens):
            bad = int(b.ksl[r]) + k_lens[r] - n + n // 2     # seen from row n / 2 on
            b.k[bad, :, 3] = float("nan")
            b.v[bad, :, 5] = float("inf")
            b.kr[bad + 1, 7] = float("nan")
            b.v[bad + 1] = float("nan")
        got = b.run()
        assert pa.get_error() == pa.PA_OK
        for r, n in enumerate(q_lens):
            a = int(b.qsl[r])
            assert torch.equal(got[a:a + n // 2].view(torch.int16),
                               clean[a:a + n // 2].view(torch.int16))
            assert torch.isnan(got[a + n // 2:a + n]).all()


@pytest.mark.parametrize("form", ["query", "later_key", "next_request"])
@pytest.mark.parametrize("q_lens,k_lens,H", [([300, 70], [420, 70], 3), ([40, 30], [3000, 1500], 1)],
                         ids=["whole", "split"])
def test_a_visible_infinite_value_stays(cuda_device, q_lens, k_lens, H, form):
    """An infinite value behind a finite key makes its dimension infinite in every
    row that sees it, whatever else of the tile is no number: another row's query, a
    key that the row hides, or the next request's keys (after the tile's last)."""
    b = Chunks(q_lens, k_lens, H, cuda_device, seed=61)
    last = []                       # the first row's own key: in a tile that hides keys
    for r, n in enumerate(q_lens):
        last.append(int(b.ksl[r]) + k_lens[r] - n)
        b.v[last[r], :, 5] = float("inf")
    clean = b.run().clone()
    for r, n in enumerate(q_lens):
        a = int(b.qsl[r])
        assert (clean[a:a + n, :, 5] == float("inf")).all()
        others = [d for d in range(DV) if d != 5]
        assert torch.isfinite(clean[a:a + n][..., others]).all()
    same = torch.ones(int(b.qsl[-1]), dtype=torch.bool, device=cuda_device)
    if form == "query":
        row = int(b.qsl[0]) + 7
        b.q[row, :, 9] = float("nan")
        same[row] = False
    elif form == "later_key":
        for r, n in enumerate(q_lens):
            b.k[last[r] + n // 2, :, 3] = float("nan")       # seen from row n / 2 on
            same[int(b.qsl[r]) + n // 2:int(b.qsl[r + 1])] = False
    else:
        b.k[b.ksl[1]:] = float("nan")
        b.v[b.ksl[1]:] = float("nan")
        same[b.qsl[1]:] = False
    got = b.run()
    assert pa.get_error() == pa.PA_OK
    rows = got[:b.qsl[-1]]
    assert torch.equal(rows[same].view(torch.int16), clean[:b.qsl[-1]][same].view(torch.int16))
    assert torch.isnan(rows[~same]).all()


def test_a_cleared_value_returns_to_the_rows_that_see_it(cuda_device):
    """A key that its first rows hide, with an infinite rotary element and an
    infinite value: the rows that see it with score -inf get 0 times infinity, a NaN,
    in that dimension and nothing else from it."""
    for q_lens, k_lens, H in (([300, 70], [420, 70], 3), ([40], [3000], 1)):
        b = Chunks(q_lens, k_lens, H, cuda_device, seed=62)
        b.q[..., DN + 7] = -b.q[..., DN + 7].abs() - 0.01     # every score of the key is -inf
        clean = {}
        for bad_value in (False, True):
            for r, n in enumerate(q_lens):
                key = int(b.ksl[r]) + k_lens[r] - n + n // 2  # seen from row n / 2 on
                b.kr[key, 7] = float("inf")
                if bad_value:
                    b.v[key, :, 5] = float("inf")
            clean[bad_value] = b.run().clone()
        assert pa.get_error() == pa.PA_OK
        assert torch.isfinite(clean[False]).all()
        for r, n in enumerate(q_lens):
            a = int(b.qsl[r])
            want = clean[False][a:a + n].clone()
            want[n // 2:, :, 5] = float("nan")
            got = clean[True][a:a + n]
            assert torch.equal(torch.isnan(got), torch.isnan(want))
            assert torch.equal(got.nan_to_num(), want.nan_to_num())


@pytest.mark.parametrize("q_lens,k_lens,H", [([1, 300, 70], [1, 420, 70], 3), ([40, 2], [3000, 700], 1)],
                         ids=["whole", "split"])
def test_scores_of_minus_infinity_alone(cuda_device, q_lens, k_lens, H):
    """A row whose query holds an infinity that scores every visible key -inf is NaN,
    as the softmax of such scores is, and not zero."""
    b = Chunks(q_lens, k_lens, H, cuda_device, seed=63)
    b.kr[:, 7] = b.kr[:, 7].abs() + 0.01
    clean = b.run().clone()
    rows = [int(a) for a in b.qsl[:-1]] + [int(b.qsl[-1]) - 1]
    for t in rows:
        b.q[t, H - 1, DN + 7] = float("-inf")
    got = b.run()
    assert pa.get_error() == pa.PA_OK
    for t in range(b.qsl[-1]):
        for h in range(H):
            if t in rows and h == H - 1:
                assert torch.isnan(got[t, h]).all(), t
            else:
                assert torch.equal(got[t, h], clean[t, h]), (t, h)


def test_a_piece_of_minus_infinity_scores(cuda_device):
    """A unit that CTAs share, the first half of whose keys score -inf: they weigh
    nothing, but an infinite value among them is 0 times infinity, a NaN."""
    b = Chunks([40], [4000], 1, cuda_device, seed=64)
    b.q[..., DN + 7] = -b.q[..., DN + 7].abs() - 0.01
    b.kr[:2000, 7] = float("inf")
    clean = b.run().clone()
    assert torch.isfinite(clean).all()
    half = Chunks([40], [2000], 1, cuda_device, seed=64)     # the other half alone
    half.q, half.k, half.v, half.kr, half.out = b.q, b.k[2000:], b.v[2000:], b.kr[2000:], clean
    half.check()
    b.v[77, 0, 5] = float("inf")
    got = b.run().clone()
    assert pa.get_error() == pa.PA_OK
    assert torch.isnan(got[..., 5]).all()
    others = [d for d in range(DV) if d != 5]
    assert torch.equal(got[..., others], clean[..., others])


@pytest.mark.parametrize("q_lens,k_lens,spare", [
    ([250], [250], 9), ([507, 3], [504, 80], 9), ([30, 1], [30, 40], 700), ([5], [3000], 300)])
def test_padded_batches(cuda_device, q_lens, k_lens, spare):
    """The mirrors plan for padding rows that end in a query tile of their own: the
    batch is right, they stay as they are, and nothing is flagged."""
    b = Chunks(q_lens, k_lens, 2, cuda_device, seed=71, spare=spare)
    b.run()
    assert pa.get_error() == pa.PA_OK
    b.check()
    assert (b.out[b.qsl[-1]:] == 9).all()
