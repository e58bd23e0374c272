"""64-bit definitions of the calls that attend to a part of a cache (block
bounds, scores, selection, attention over listed blocks, attention mass,
compaction), straight from the documentation, and bounds on what fp32 kernels
may be off by. Numpy only; nothing here is shared with the kernels.

Error bounds. A product of two bf16 (or of bf16 and E4M3) numbers is exact in
fp32, so a dot product of n terms is off by n additions, each by at most one
step of the partial sum (2^-23 of it: tensor cores may cut off where a processor
rounds). A softmax weight exp(s - lse) is off by twice the largest error of a
score of its row (its own and lse's), by the rounding of score and reference to
fp32 in units of log 2 and by 2^-21 for exp2 and the sums' own rounding."""
import numpy as np
import torch


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def e4m3(codes):
    """Values of E4M3 codes (uint8), from their bits."""
    c = np.asarray(codes).astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c > 127, -v, v)


def cells(pool_half):
    """A pool's K or V [blocks][Hkv][B][D] as 64-bit values (codes unscaled)."""
    if pool_half.dtype == torch.uint8:
        return e4m3(pool_half.cpu().numpy())
    return f64(pool_half)


def rows_of(qsl, seqs):
    """(request, row, position) of every query token."""
    for r, n in enumerate(seqs):
        for j in range(qsl[r + 1] - qsl[r]):
            yield r, qsl[r] + j, n - (qsl[r + 1] - qsl[r]) + j


def context(half, table, n, B, h):
    """Rows 0 .. n-1 of a request's stored keys (or values) of head h."""
    x = np.concatenate([half[table[i], h] for i in range(-(-n // B))]) if n else half[0, h][:0]
    return x[:n]


def bounds(k, table, qsl, seqs, B, out):
    """out [blocks][Hkv][2][D] with the bounds of the blocks that hold new tokens
    (qsl None: of all blocks) made anew."""
    top = float(torch.finfo(torch.bfloat16).max)
    for r, n in enumerate(seqs):
        new = n if qsl is None else qsl[r + 1] - qsl[r]
        if new == 0:
            continue
        for i in range((n - new) // B, -(-n // B)):
            x = np.clip(k[table[r][i]][:, : min(B, n - i * B)], -top, top)
            out[table[r][i], :, 0] = x.min(1)  # (numpy's min and max keep NaN)
            out[table[r][i], :, 1] = x.max(1)
    return out


def scores(q, bnd, table, qsl, seqs, B, g, k_scale, out):
    """out [T][Hkv][N] for the visible blocks, and the bound on each error."""
    tol = np.zeros_like(out)
    D = q.shape[-1]
    for r, t, p in rows_of(qsl, seqs):
        n = p // B + 1
        b = bnd[np.asarray(table[r][:n])]                     # [n][Hkv][2][D]
        x = q[t].reshape(-1, 1, g, D)                         # [Hkv][1][g][D]
        pos, neg = np.maximum(x, 0), np.minimum(x, 0)
        lo, hi = (b[:, :, i].transpose(1, 0, 2)[:, :, None] for i in (0, 1))  # [Hkv][n][1][D]
        with np.errstate(invalid="ignore", over="ignore"):
            s = (pos * hi + neg * lo).sum(-1)                 # [Hkv][n][g]
            size = (np.abs(pos * hi) + np.abs(neg * lo)).sum(-1)
        out[t, :, :n] = s.max(-1) * k_scale
        tol[t, :, :n] = size.max(-1) * k_scale * (2 * D + 4) * 2.0 ** -23
    return out, tol


def pick(x, n, first, last, k):
    """Kept indices of x[:n], ascending, -1 behind: the first and last, then the
    greatest, the lower index of equal ones, NaN above all."""
    if n <= k:
        return np.concatenate([np.arange(n), np.full(k - n, -1)])
    forced = [i for i in range(n) if i < first or i >= n - last]
    rest = [i for i in range(n) if not (i < first or i >= n - last)]
    rest.sort(key=lambda i: (0, 0.0, i) if np.isnan(x[i]) else (1, -float(x[i]), i))
    return np.array(sorted(forced + rest[: k - len(forced)]))


def _softmax(s):
    with np.errstate(invalid="ignore"):
        e = np.exp(s - s.max()) if s.size and not np.isnan(s).any() else np.full(s.shape, np.nan)
        return e / e.sum()


def _score_error(q, k, scale, f8_tiles=False):
    """Bound on the error of any of a row's scores (natural units)."""
    D = q.shape[-1]
    with np.errstate(invalid="ignore", over="ignore"):
        size = np.abs(scale) * (np.abs(k) @ np.abs(q))
        err = size * (D + 4) * 2.0 ** -23 + size * 2.0 ** -23
        if f8_tiles:
            err = err + np.abs(scale) * np.abs(q).max() * 2.0 ** -17 * np.abs(k).sum(-1)
    return float(np.where(np.isfinite(err), err, 0).max()) if err.size else 0.0


def sparse(q, k, v, table, selected, qsl, seqs, B, g, scale, k_scale, v_scale, f8):
    """(out, bound) [T][Hq][D]: attention over the listed blocks' visible keys."""
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    p_step = 2.0 ** (-11 if f8 else -8)  # half a step of a weight in f16 or bf16
    for r, t, p in rows_of(qsl, seqs):
        for h in range(k.shape[1]):
            at = [(b, o) for b in selected[t, h] if b >= 0 for o in range(B) if b * B + o <= p]
            if not at:
                continue
            ids = np.array([table[r][b] for b, _ in at])
            off = np.array([o for _, o in at])
            K, V = k[ids, h, off] * k_scale, v[ids, h, off] * v_scale
            for j in range(h * g, (h + 1) * g):
                with np.errstate(invalid="ignore", over="ignore"):
                    w = _softmax(scale * (K @ q[t, j]))
                    out[t, j] = w @ V
                    d = 2 * _score_error(q[t, j], K, scale) + 2.0 ** -20
                    tol[t, j] = (w @ np.abs(V)) * (p_step + d) + 2.0 ** -8 * np.abs(out[t, j]) * (
                        1 + p_step + d) + (2.0 ** -24 * np.abs(V).sum(0) if f8 else 0) + 1e-38
    return out, tol


def mass(q, k, old, rows, table, qsl, seqs, B, g, scale, k_scale, decay, window, out, f8):
    """out [max_reqs][N] with the requests' rows made anew, and the bound."""
    tol = np.zeros(out.shape)
    Hkv = k.shape[1]
    for r, n in enumerate(seqs):
        new = qsl[r + 1] - qsl[r]
        if new == 0:
            continue
        w = min(new, window) if window else new
        tiles = w * g > 16
        got, err = np.zeros(n), np.zeros(n)
        adds = 48 if tiles else Hkv * w * g + 2
        for h in range(Hkv):
            K = context(k, table[r], n, B, h) * k_scale
            for j in range(w):
                sees = n - w + j + 1
                for i in range(h * g, (h + 1) * g):
                    x = q[qsl[r + 1] - w + j, i]
                    with np.errstate(invalid="ignore", over="ignore"):
                        p = _softmax(scale * (K[:sees] @ x))
                        d = 2 * _score_error(x, K[:sees], scale, f8 and tiles) + 2.0 ** -20
                    got[:sees] += p
                    err[:sees] += p * d
        before = np.zeros(n)
        before[: n - new] = np.float64(np.float32(decay)) * old[rows[r], : n - new]
        out[rows[r], :n] = got + before
        tol[rows[r], :n] = err + (adds * got + np.abs(before) * 2 + got) * 2.0 ** -23 + 1e-38
    return out, tol
