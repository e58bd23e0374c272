"""Plain 64-bit references of the latent path, straight from the definitions,
and seeded inputs for its tests (numpy / CPU torch; no code of the library)."""
import numpy as np
import torch

ROPE = 64
BF16_HALF = torch.finfo(torch.bfloat16).eps / 2   # largest relative rounding error of bf16
E4M3_HALF = torch.finfo(torch.float8_e4m3fn).eps / 2


def f64(t):
    return t.detach().cpu().double().numpy()


def turn(x, positions, inv_freq, interleaved, factor=1.0):
    """x [T][H][D] with its first 2 * len(inv_freq) dims turned, in 64 bits."""
    y = np.array(x, np.float64)
    n = len(inv_freq)
    ang = np.asarray(positions, np.float64)[:, None, None] * np.asarray(inv_freq, np.float64)
    c, s = np.cos(ang) * factor, np.sin(ang) * factor
    a = (slice(None), slice(None), slice(0, 2 * n, 2) if interleaved else slice(0, n))
    b = (slice(None), slice(None), slice(1, 2 * n, 2) if interleaved else slice(n, 2 * n))
    u, v = np.array(y[a]), np.array(y[b])
    y[a], y[b] = u * c - v * s, v * c + u * s
    return y


def turn_tolerance(x, y, n, interleaved, factor=1.0):
    """Half a bf16 step of the result, and the fp32 work: the angle is off by
    at most 2^-23 of a turn (2 pi 2^-23 = 7.5e-7 rad), cos, sin, products and
    the sum by a few 2^-24: under 1.5e-6 * factor * (|x| + |y|) of the pair."""
    x = np.abs(np.asarray(x, np.float64))
    pair = np.zeros_like(x)
    if interleaved:
        p = x[..., 0:2 * n:2] + x[..., 1:2 * n:2]
        pair[..., 0:2 * n:2] = pair[..., 1:2 * n:2] = p
    else:
        p = x[..., :n] + x[..., n:2 * n]
        pair[..., :n] = pair[..., n:2 * n] = p
    return BF16_HALF * np.abs(y) * 1.0001 + 1.5e-6 * factor * pair


def e4m3_round(x):
    """Nearest E4M3 value (ties to even), saturating; NaN stays NaN."""
    x = np.asarray(x, np.float64)
    _, e = np.frexp(np.where(np.isfinite(x), x, 1.0))
    step = np.exp2(np.maximum(e - 4, -9).astype(np.float64))
    with np.errstate(invalid="ignore"):
        near = np.clip(np.round(x / step) * step, -448, 448)
        return np.where(np.isinf(x), np.sign(x) * 448, near)


def token_scale(row):
    """The smallest power of two 2^e, e >= -60, with max |row| <= 448 * 2^e
    over the finite elements; 1 for a row of zeros."""
    fin = np.abs(row[np.isfinite(row)])
    m = fin.max() if fin.size else 0.0
    if m == 0:
        return 1.0
    e = -60
    while m > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def quantise(rows):
    """(values that the stored codes stand for, scales) of latent rows."""
    s = np.array([token_scale(r) for r in rows])
    return e4m3_round(rows / s[:, None]) * s[:, None], s


def e4m3_values(codes):
    """E4M3 codes (uint8) as doubles."""
    c = np.asarray(codes).astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    return np.where(c > 127, -v, v)


def new_pool(pa, blocks, B, L, fp8, dev, poison=True):
    """A pool of NaN cells (codes 0x7F, NaN scales)."""
    nan = float("nan") if poison else 0.0
    rope = torch.full((blocks, B, ROPE), nan, dtype=torch.bfloat16, device=dev)
    if fp8:
        return pa.LatentPool(torch.full((blocks, B, L), 0x7F if poison else 0, dtype=torch.uint8,
                                        device=dev),
                             rope, torch.full((blocks, B), nan, device=dev))
    return pa.LatentPool(torch.full((blocks, B, L), nan, dtype=torch.bfloat16, device=dev), rope)


def pool_rows(pool):
    """(latents, rotary parts) of every cell in 64 bits, [slots][..]."""
    rope = f64(pool.rope).reshape(-1, ROPE)
    if pool.scales is None:
        return f64(pool.latent).reshape(-1, pool.latent_dim), rope
    v = e4m3_values(pool.latent.cpu().numpy()).reshape(-1, pool.latent_dim)
    return v * f64(pool.scales).reshape(-1, 1), rope


def tables(rng, seqs, B, spare=3):
    """(block tables [R][max_blocks] with -1 past each request, num_blocks)."""
    need = [(s + B - 1) // B for s in seqs]
    order = rng.permutation(sum(need) + spare).astype(np.int32)
    tab = np.full((len(seqs), max(max(need, default=0), 1)), -1, np.int32)
    at = 0
    for r, n in enumerate(need):
        tab[r, :n] = order[at:at + n]
        at += n
    return tab, len(order)


def slots_of(tab, r, n, B):
    t = np.arange(n)
    return tab[r, t // B].astype(np.int64) * B + t % B


def softmax_rows(x):
    """Softmax along the last axis; a row of -inf gives zeros."""
    m = x.max(-1, keepdims=True, initial=-np.inf)
    p = np.exp(x - np.where(np.isfinite(m), m, 0.0))
    p[~np.isfinite(x)] = 0.0
    l = p.sum(-1, keepdims=True)
    return p / np.where(l > 0, l, 1.0)


def visible(q_len, k_len, causal):
    """[q_len][k_len]: query j of the request sees key n."""
    n = np.arange(k_len)
    if not causal:
        return np.ones((q_len, k_len), bool)
    return n[None] <= (k_len - q_len + np.arange(q_len))[:, None]


def absorbed(q, c, kr, scale, causal=1):
    """Absorbed attention of one request: q [Tq][H][L + 64], c [N][L], kr [N][64]."""
    k = np.concatenate((c, kr), -1)
    x = np.einsum("thd,nd->thn", q, k) * scale
    x = np.where(visible(q.shape[0], k.shape[0], causal)[:, None], x, -np.inf)
    p = softmax_rows(x)
    return np.einsum("thn,nl->thl", p, c), p


def expanded(q, k_nope, k_rope, v, scale, causal=1):
    """Expanded attention of one request: q [Tq][H][Dn + Dr], k_nope [N][H][Dn],
    k_rope [N][Dr], v [N][H][Dv]."""
    dn = k_nope.shape[-1]
    x = (np.einsum("thd,nhd->thn", q[..., :dn], k_nope)
         + np.einsum("thd,nd->thn", q[..., dn:], k_rope)) * scale
    x = np.where(visible(q.shape[0], k_nope.shape[0], causal)[:, None], x, -np.inf)
    p = softmax_rows(x)
    return np.einsum("thn,nhd->thd", p, v), p
