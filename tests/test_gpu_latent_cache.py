"""GPU tests of pa_rope, pa_write_latent, pa_read_latent and
pa_copy_latent_blocks against 64-bit references; what is stored as codes or
copied is compared bit for bit."""
import numpy as np
import pytest
import torch

from paged_kv_cache_143_gb300 import pa
from tests import latent_reference as ref

pytestmark = pytest.mark.gpu


def randn(rng, shape, dev, mult=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * mult).to(dev).bfloat16()


def i32(a, dev):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=dev)


def check_turn(x, out, positions, inv_freq, interleaved, factor):
    n = len(inv_freq)
    want = ref.turn(ref.f64(x), positions, inv_freq, interleaved, factor)
    err = np.abs(ref.f64(out) - want)
    tol = ref.turn_tolerance(ref.f64(x), want, n, interleaved, factor)
    assert (err[..., :2 * n] <= tol[..., :2 * n]).all(), (err - tol).max()
    assert torch.equal(out[..., 2 * n:].view(torch.int16), x[..., 2 * n:].view(torch.int16))


SHAPES = [  # T, H, D, rot
    (1, 1, 64, 64), (1, 128, 64, 64), (7, 3, 128, 64), (300, 5, 80, 32), (129, 16, 192, 64),
    (33, 1, 2, 2), (5, 4, 34, 18), (64, 2, 256, 256), (1000, 1, 64, 48), (3, 700, 16, 16),
    (17, 2, 96, 96), (200, 1, 8, 0),
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_rope_shapes(cuda_device, shape, interleaved):
    T, H, D, rot = shape
    rng = np.random.default_rng(T + H + D)
    x = randn(rng, (T, H, D), cuda_device)
    pos = rng.integers(0, 40000, T)
    freq, factor = pa.rope_frequencies(rot, scaling="by_parts", stretch=4.0) if rot else (
        torch.empty(0), 1.0)
    out = torch.full_like(x, 7.0)
    pa.rope(x, out, i32(pos, cuda_device), freq.to(cuda_device), interleaved, factor)
    check_turn(x, out, pos, freq.numpy(), interleaved, factor)
    pa.rope(x, x, i32(pos, cuda_device), freq.to(cuda_device), interleaved, factor)  # in place
    assert torch.equal(x.view(torch.int16), out.view(torch.int16))
    assert pa.get_error() == pa.PA_OK


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_far_positions(cuda_device, interleaved):
    """Every int32 position, negative ones among them: angles keep their
    accuracy where an fp32 product would be lost."""
    pos = np.array([0, 1, -1, 65535, 65536, -65536, 10 ** 6, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31],
                   np.int64)
    rng = np.random.default_rng(1)
    x = randn(rng, (len(pos), 2, 64), cuda_device)
    freq, _ = pa.rope_frequencies(64)
    out = torch.empty_like(x)
    pa.rope(x, out, i32(pos, cuda_device), freq.to(cuda_device), interleaved)
    check_turn(x, out, pos, freq.numpy(), interleaved, 1.0)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("form", ["tail", "heads_outside", "odd_stride", "odd_start", "broadcast"])
def test_rope_strides(cuda_device, form, interleaved):
    rng = np.random.default_rng(3)
    T, H, D = 21, 6, 64
    pos = rng.integers(0, 9000, T)
    freq, _ = pa.rope_frequencies(D)
    whole = torch.full((T, H, 192), 5.0, dtype=torch.bfloat16, device=cuda_device)
    src = randn(rng, (T, H, 192), cuda_device)
    x, out = src[..., 128:], whole[..., 100 - 100 % 8:][..., :D]
    if form == "heads_outside":
        x = randn(rng, (H, T, D), cuda_device).transpose(0, 1)
        whole = torch.full((H, T, D), 5.0, dtype=torch.bfloat16, device=cuda_device)
        out = whole.transpose(0, 1)
    elif form == "odd_stride":
        whole = torch.full((T, H, 67), 5.0, dtype=torch.bfloat16, device=cuda_device)
        out = whole[..., :D]
    elif form == "odd_start":
        x = src[..., 1:1 + D]
    elif form == "broadcast":
        x = randn(rng, (T, 1, D), cuda_device).expand(T, H, D)
    before = whole.clone()
    pa.rope(x, out, i32(pos, cuda_device), freq.to(cuda_device), interleaved)
    check_turn(x, out, pos, freq.numpy(), interleaved, 1.0)
    out.fill_(5.0)  # what lies between the rows was left alone
    assert torch.equal(whole, before)


def test_rope_turned_back(cuda_device):
    """The inverse is the turn by the negated positions."""
    rng = np.random.default_rng(4)
    x = randn(rng, (50, 3, 64), cuda_device)
    pos = i32(rng.integers(0, 100000, 50), cuda_device)
    freq = pa.rope_frequencies(64, device=cuda_device)[0]
    y, z = torch.empty_like(x), torch.empty_like(x)
    pa.rope(x, y, pos, freq, factor=2.0)
    pa.rope(y, z, -pos, freq, factor=0.5)
    # two roundings of values no larger than the pair's magnitude, and fp32 work
    pair = (x[..., :32].float() ** 2 + x[..., 32:].float() ** 2).sqrt().repeat(1, 1, 2)
    assert ((z.float() - x.float()).abs() <= pair * (2 * ref.BF16_HALF * 1.5 + 1e-5)).all()


def exact_turns(pos, freq):
    """pos * freq / (2 pi) in turns, within [-1/2, 1/2), by whole numbers: 1 / (2 pi) to
    2^-200, freq a multiple of 2^-149."""
    inv = 255752132986241185678408580023709873616295664310550962376831  # 2^200 / (2 pi)
    t = (int(pos) * int(float(freq) * 2.0 ** 149) * inv) % (1 << 349)
    return (t - (1 << 349) if t >> 348 else t) / 2.0 ** 349


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_angles_at_any_position(cuda_device, interleaved):
    """Angles next to a whole number of half turns, where sin is small and its bf16
    rounding with it: (1, 0) turned by theta is (cos, sin). The angle may be off by 2^-25
    of a turn, sin by 2^-22 of itself (two fp32 steps), and both are rounded to bf16."""
    rng = np.random.default_rng(6)
    freq = np.concatenate((10.0 ** rng.uniform(-8, 0, 24), 2.0 ** rng.uniform(0, 8, 6),
                           [1.0, -0.37])).astype(np.float32)
    n, per = len(freq), 40
    positions = []
    for f in freq:                      # positions next to k / 2 turns, the nearest kept
        top = 2 ** 31 - 1
        k = rng.integers(-int(top * abs(f) / np.pi) - 1, int(top * abs(f) / np.pi) + 1, 4000)
        p = np.clip(np.rint(k * np.pi / abs(float(f))), -top - 1, top).astype(np.int64)
        off = [abs((2 * exact_turns(x, f) + 0.5) % 1 - 0.5) for x in p]
        positions.append(p[np.argsort(off)[:per]])
    pos = np.concatenate(positions)
    x = torch.zeros(len(pos), 1, 2 * n, dtype=torch.bfloat16, device=cuda_device)
    x[..., 0:2 * n:2 if interleaved else 1][..., :n] = 1.0
    out = torch.empty_like(x)
    pa.rope(x, out, i32(pos, cuda_device), torch.from_numpy(freq).to(cuda_device), interleaved)
    assert pa.get_error() == pa.PA_OK
    got = ref.f64(out)[:, 0]
    small = 0
    for i, f in enumerate(freq):
        rows = range(per * i, per * i + per)
        turns = np.array([exact_turns(pos[t], f) for t in rows])
        c, s = (got[rows.start:rows.stop, j] for j in
                ((2 * i, 2 * i + 1) if interleaved else (i, n + i)))
        for value, want in ((c, np.cos(2 * np.pi * turns)), (s, np.sin(2 * np.pi * turns))):
            tol = ref.BF16_HALF * np.abs(want) * (1 + 2.0 ** -20) + 2 * np.pi * 2.0 ** -25 \
                + 2.0 ** -22 * np.abs(want)
            assert (np.abs(value - want) <= tol).all(), (f, (np.abs(value - want) / tol).max())
        small += int((np.abs(np.sin(2 * np.pi * turns)) < 2.0 ** -12).sum())
    assert small > n * per // 2         # (the test's own inputs: most angles are such)


def test_rope_more_wide_heads_than_a_grid_has_rows(cuda_device):
    """66000 heads of 8256 dims, each more than a CTA's work: one token of them."""
    rng = np.random.default_rng(7)
    H, D = 66000, 8256
    x = randn(rng, (1, 1, D), cuda_device)
    out = torch.empty(1, H, D, dtype=torch.bfloat16, device=cuda_device)
    freq = pa.rope_frequencies(64)[0]
    pa.rope(x.expand(1, H, D), out, i32([12345], cuda_device), freq.to(cuda_device))
    check_turn(x, out[:, :1], [12345], freq.numpy(), False, 1.0)
    assert torch.equal(out, out[:, :1].expand(1, H, D))
    assert pa.get_error() == pa.PA_OK


ROWS = [(1, 16, 512), (5, 32, 256), (255, 64, 512), (256, 16, 256), (1030, 32, 512)]


def write_case(T, B, L, seed, dev):
    rng = np.random.default_rng(seed)
    blocks = (T + B - 1) // B + 2
    slots = rng.permutation(blocks * B)[:T].astype(np.int64)
    mult = np.exp2(rng.integers(-12, 12, (T, 1)))
    c = torch.from_numpy(rng.standard_normal((T, L)) * mult).to(dev).bfloat16()
    kr = randn(rng, (T, ref.ROPE), dev)
    return rng, blocks, slots, c, kr


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("interleaved", [None, False, True])
@pytest.mark.parametrize("rows", ROWS, ids=str)
def test_write_latent(cuda_device, rows, interleaved, fp8):
    T, B, L = rows
    dev = cuda_device
    rng, blocks, slots, c, kr = write_case(T, B, L, T + L, dev)
    if T > 4:
        slots[3] = -1  # padding
        c[2] = 0.0
        c[4, 5:9] = torch.tensor([float("inf"), float("-inf"), float("nan"), 1e-40], device=dev)
    pool = ref.new_pool(pa, blocks, B, L, fp8, dev)
    pos = rng.integers(0, 10 ** 6, T)
    freq = pa.rope_frequencies(64)[0]
    kw = {} if interleaved is None else dict(positions=i32(pos, dev), inv_freq=freq.to(dev),
                                             interleaved=interleaved, factor=1.25)
    before = pool.latent.clone()
    pa.write_latent(pool, c, kr, torch.from_numpy(slots).to(dev), **kw)
    assert pa.get_error() == pa.PA_OK
    live = slots >= 0
    at = torch.from_numpy(slots[live]).to(dev)
    got = pool.latent.view(-1, L)[at]
    if fp8:
        want, scale = ref.quantise(ref.f64(c)[live])
        np.testing.assert_array_equal(ref.f64(pool.scales).reshape(-1)[slots[live]], scale)
        np.testing.assert_array_equal(ref.e4m3_values(got.cpu().numpy()) * scale[:, None], want)
        assert not (got == 0xFF).any()  # NaN is 0x7F
    else:
        assert torch.equal(got.view(torch.int16), c[torch.from_numpy(live).to(dev)].view(torch.int16))
    rot = pool.rope.view(-1, 64)[at]
    if interleaved is None:
        assert torch.equal(rot, kr[torch.from_numpy(live).to(dev)])
    else:
        x = ref.f64(kr)[live][:, None]
        want = ref.turn(x, pos[live], freq.numpy(), interleaved, 1.25)
        err = np.abs(ref.f64(rot)[:, None] - want)
        assert (err <= ref.turn_tolerance(x, want, 32, interleaved, 1.25)).all()
    # every other cell was left alone
    rest = np.setdiff1d(np.arange(blocks * B), slots)
    rest = torch.from_numpy(rest).to(dev)
    elt = torch.uint8 if fp8 else torch.int16
    assert torch.equal(pool.latent.view(-1, L)[rest].view(elt), before.view(-1, L)[rest].view(elt))
    assert torch.isnan(pool.rope.view(-1, 64)[rest]).all()


def test_write_latent_strided_rows(cuda_device):
    """Latent and rotary key as the two parts of one projection's output."""
    dev = cuda_device
    rng, blocks, slots, c, kr = write_case(37, 16, 512, 9, dev)
    both = torch.cat((c, kr), -1)
    a = ref.new_pool(pa, blocks, 16, 512, True, dev, poison=False)
    b = ref.new_pool(pa, blocks, 16, 512, True, dev, poison=False)
    at = torch.from_numpy(slots).to(dev)
    pa.write_latent(a, c, kr, at)
    pa.write_latent(b, both[:, :512], both[:, 512:], at)
    for x, y in ((a.latent, b.latent), (a.rope, b.rope), (a.scales, b.scales)):
        assert torch.equal(x, y)


def test_write_latent_flags_slots_past_the_pool(cuda_device):
    dev = cuda_device
    pool = ref.new_pool(pa, 2, 16, 256, False, dev, poison=False)
    c, kr = torch.ones(3, 256, device=dev).bfloat16(), torch.ones(3, 64, device=dev).bfloat16()
    pa.write_latent(pool, c, kr, torch.tensor([0, 32, 1 << 40], device=dev))
    assert pa.get_error() == pa.PA_ERR_DEVICE_BOUNDS
    assert pool.latent.sum() == 256 and pool.rope.sum() == 64


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,L", [(16, 256), (32, 512), (64, 512)])
def test_read_latent(cuda_device, B, L, fp8):
    dev = cuda_device
    rng = np.random.default_rng(B + L)
    seqs = [1, 0, 130, 64, 63, 0, 65, 300, 1]
    firsts = [0, 0, 7, 64, 0, 3, 1, 99, 0]
    tab, blocks = ref.tables(rng, [f + s for f, s in zip(firsts, seqs)], B)
    pool = ref.new_pool(pa, blocks, B, L, fp8, dev)
    for r, n in enumerate(f + s for f, s in zip(firsts, seqs)):
        if n:
            c = randn(rng, (n, L), dev, 2.0 ** rng.integers(-6, 6))
            pa.write_latent(pool, c, randn(rng, (n, 64), dev),
                            torch.from_numpy(ref.slots_of(tab, r, n, B)).to(dev))
    lat, rot = pool_values = ref.pool_rows(pool)
    start = np.cumsum([0] + seqs)
    N = start[-1] + 5  # rows past the last request stay
    out = torch.full((N, L + 8), 3.0, dtype=torch.bfloat16, device=dev)
    rout = torch.full((N, 70), 3.0, dtype=torch.bfloat16, device=dev)
    pa.read_latent(pool, i32(tab, dev), i32(start, dev), out[:, :L], rout[:, :64],
                   first=i32(firsts, dev))
    assert pa.get_error() == pa.PA_OK
    for r, (f, n) in enumerate(zip(firsts, seqs)):
        at = ref.slots_of(tab, r, f + n, B)[f:]
        np.testing.assert_array_equal(ref.f64(out[start[r]:start[r + 1], :L]), lat[at])
        np.testing.assert_array_equal(ref.f64(rout[start[r]:start[r + 1], :64]), rot[at])
    assert (out[start[-1]:] == 3).all() and (out[:, L:] == 3).all()
    assert (rout[start[-1]:] == 3).all() and (rout[:, 64:] == 3).all()
    # without `first`: from the start of each request
    pa.read_latent(pool, i32(tab, dev), i32(start, dev), out[:, :L], rout[:, :64])
    for r, n in enumerate(seqs):
        np.testing.assert_array_equal(ref.f64(out[start[r]:start[r + 1], :L]),
                                      lat[ref.slots_of(tab, r, n, B)])


def test_read_latent_flags_what_it_cannot_read(cuda_device):
    dev = cuda_device
    pool = ref.new_pool(pa, 4, 16, 256, False, dev, poison=False)
    out = torch.full((20, 256), 3.0, dtype=torch.bfloat16, device=dev)
    rout = torch.full((20, 64), 3.0, dtype=torch.bfloat16, device=dev)

    def status(tab, start, first=None):
        pa.read_latent(pool, i32(tab, dev), i32(start, dev), out, rout,
                       first=None if first is None else i32(first, dev))
        return pa.get_error()

    assert status([[0, 1]], [0, 20]) == pa.PA_OK
    assert status([[0, 4]], [0, 20]) == pa.PA_ERR_DEVICE_BOUNDS      # block past the pool
    assert status([[0, -1]], [0, 20]) == pa.PA_ERR_DEVICE_BOUNDS
    assert status([[0]], [0, 20]) == pa.PA_ERR_DEVICE_BOUNDS         # past the table
    assert status([[0, 1]], [0, 20], [20]) == pa.PA_ERR_DEVICE_BOUNDS
    assert status([[0, 1]], [0, 20], [-1]) == pa.PA_ERR_DEVICE_BOUNDS
    assert status([[0, 1]], [0, 21]) == pa.PA_ERR_DEVICE_BOUNDS      # more rows than outputs
    assert status([[0, 1]], [1, 20]) == pa.PA_ERR_DEVICE_BOUNDS
    assert status([[0, 1]], [0, 0]) == pa.PA_OK


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B", [16, 64])
def test_copy_latent_blocks(cuda_device, B, fp8):
    dev = cuda_device
    rng = np.random.default_rng(B)
    pool = ref.new_pool(pa, 9, B, 512, fp8, dev, poison=False)
    pa.write_latent(pool, randn(rng, (9 * B, 512), dev), randn(rng, (9 * B, 64), dev),
                    torch.arange(9 * B, device=dev))
    want = [t.clone() for t in (pool.latent, pool.rope)] + ([pool.scales.clone()] if fp8 else [])
    src, dst = [0, 3, 3], [8, 1, 5]
    for t in want:
        t[dst] = t[src]
    pa.copy_latent_blocks(pool, i32(src, dev), i32(dst, dev))
    assert pa.get_error() == pa.PA_OK
    for t, w in zip((pool.latent, pool.rope, pool.scales), want):
        assert torch.equal(t, w)
    pa.copy_latent_blocks(pool, i32([0, 9], dev), i32([-1, 2], dev))
    assert pa.get_error() == pa.PA_ERR_DEVICE_BOUNDS
    for t, w in zip((pool.latent, pool.rope, pool.scales), want):
        assert torch.equal(t, w)


def test_cells_past_32_bits_of_bytes(cuda_device):
    """A pool whose last cells lie more than 2^32 bytes past its start."""
    dev = cuda_device
    B, L = 64, 512
    blocks = (1 << 32) // (B * L * 2) + 3
    pool = pa.LatentPool(torch.zeros(blocks, B, L, dtype=torch.bfloat16, device=dev),
                         torch.zeros(blocks, B, 64, dtype=torch.bfloat16, device=dev))
    rng = np.random.default_rng(2)
    c, kr = randn(rng, (B, L), dev), randn(rng, (B, 64), dev)
    at = (blocks - 1) * B + torch.arange(B, device=dev)
    pa.write_latent(pool, c, kr, at)
    assert torch.equal(pool.latent[-1], c) and torch.equal(pool.rope[-1], kr)
    out, rout = torch.empty_like(c), torch.empty_like(kr)
    pa.read_latent(pool, i32([[blocks - 1]], dev), i32([0, B], dev), out, rout)
    assert torch.equal(out, c) and torch.equal(rout, kr)
    pa.copy_latent_blocks(pool, i32([blocks - 1], dev), i32([blocks - 2], dev))
    assert torch.equal(pool.latent[-2], c) and pa.get_error() == pa.PA_OK
