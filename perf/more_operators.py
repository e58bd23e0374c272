"""Cases for attending to a part of a long cache: blocks selected for each query by a cheap score (bounds of a block's
keys, scores from them, selection, attention over the selected blocks), and tokens evicted from the cache by the
attention that they received (weights summed, tokens kept, the cache compacted).

``run`` computes a case in elementary torch operations where ``own`` is false, and makes a user's calls of the
framework where it is true. Lengths are drawn from a case's own ``len_seed``; values from the seed of ``prepare``.
"""
import math
import random

import numpy as np
import torch

own = False


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # bounds of the blocks that one decode step wrote to: one per running request
        {"name": "bounds-decode-64", "op": "bounds", "R": 64, "lo": 100, "hi": 4096, "q_lo": 1, "q_hi": 1, "len_seed": 1,
         "Hq": 32, "Hkv": 8, "D": 128, "B": 16, "dtype": "bf16"},
        # bounds of the prompts of a few long requests, all at once
        {"name": "bounds-prompts-fp8", "op": "bounds", "R": 6, "lo": 20000, "hi": 40000, "q_lo": 15000, "q_hi": 20000,
         "len_seed": 2, "Hq": 64, "Hkv": 8, "D": 128, "B": 64, "dtype": "fp8"},
        # every block of long decodes scored
        {"name": "score-decode-32", "op": "score", "R": 32, "lo": 9000, "hi": 65000, "q_lo": 1, "q_hi": 1, "len_seed": 3,
         "Hq": 64, "Hkv": 8, "D": 128, "B": 16, "dtype": "fp8"},
        # the tokens of prompt chunks behind cached contexts, each scoring the blocks before it
        {"name": "score-chunks", "op": "score", "R": 3, "lo": 8000, "hi": 33000, "q_lo": 300, "q_hi": 1024, "len_seed": 4,
         "Hq": 32, "Hkv": 8, "D": 128, "B": 32, "dtype": "bf16"},
        # 128 of the blocks of each decode
        {"name": "select-blocks-32", "op": "select_blocks", "R": 32, "lo": 9000, "hi": 65000, "q_lo": 1, "q_hi": 1,
         "len_seed": 3, "Hkv": 8, "B": 16, "k": 128, "first": 1, "last": 4},
        # a quarter of the tokens of long requests kept, their beginning and their newest tokens among them
        {"name": "select-tokens-24", "op": "select_tokens", "R": 24, "lo": 12000, "hi": 32000, "len_seed": 5, "k": 4096,
         "first": 4, "last": 256},
        # the smallest attention: drafted tokens of two requests
        {"name": "sparse-draft-2x4", "op": "sparse", "R": 2, "lo": 3000, "hi": 9000, "q_lo": 4, "q_hi": 4, "len_seed": 6,
         "Hq": 32, "Hkv": 8, "D": 128, "B": 16, "dtype": "bf16", "k": 64},
        # a batch of long decodes
        {"name": "sparse-decode-fp8-48", "op": "sparse", "R": 48, "lo": 16000, "hi": 32768, "q_lo": 1, "q_hi": 1,
         "len_seed": 7, "Hq": 64, "Hkv": 8, "D": 128, "B": 16, "dtype": "fp8", "k": 256},
        # weights of one decode step over middling contexts
        {"name": "mass-decode-40", "op": "mass", "R": 40, "lo": 1000, "hi": 8192, "q_lo": 1, "q_hi": 1, "len_seed": 8,
         "Hq": 32, "Hkv": 8, "D": 128, "B": 16, "dtype": "bf16", "window": 0, "decay": 1.0},
        # the last 64 queries of long prompts judge the tokens before them
        {"name": "mass-window-fp8", "op": "mass", "R": 4, "lo": 14000, "hi": 32768, "q_lo": 500, "q_hi": 2048, "len_seed": 9,
         "Hq": 32, "Hkv": 8, "D": 128, "B": 64, "dtype": "fp8", "window": 64, "decay": 0.9},
        # one request's cache cut down to 512 tokens
        {"name": "compact-one", "op": "compact", "R": 1, "lo": 4000, "hi": 5000, "len_seed": 10, "Hkv": 8, "D": 128,
         "B": 16, "dtype": "bf16", "k": 512, "first": 4, "last": 64},
        # the caches of long requests cut down together
        {"name": "compact-16-fp8", "op": "compact", "R": 16, "lo": 9000, "hi": 20000, "len_seed": 11, "Hkv": 8, "D": 128,
         "B": 32, "dtype": "fp8", "k": 4096, "first": 16, "last": 512},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5))))))


def _heads(rng):
    Hkv = rng.choice([1, 2, 4, 8, 8, 8])
    return Hkv * rng.choice([1, 2, 4, 4, 5, 7, 8, 8, 16]), Hkv


def draw(rng):
    op = rng.choice(["bounds", "score", "score", "select_blocks", "select_tokens", "sparse", "sparse", "sparse", "mass",
                     "mass", "mass", "compact"])
    Hq, Hkv = _heads(rng)
    c = {"op": op, "len_seed": rng.randrange(1 << 30), "Hq": Hq, "Hkv": Hkv, "D": rng.choice([64, 128, 128]),
         "B": rng.choice([16, 32, 64]), "dtype": rng.choice(["bf16", "fp8"])}
    if op in ("select_tokens", "compact"):
        R = _log_int(rng, 1, 24)
        hi = _log_int(rng, 1, min(32000, (500000 if op == "select_tokens" else 120000) // R))
        k = _log_int(rng, 1, min(hi, 4096))
        first = rng.randint(0, min(16, k))
        return {**c, "R": R, "lo": rng.randint(1, hi), "hi": hi, "k": k, "first": first,
                "last": rng.randint(0, min(256, k - first))}
    R = _log_int(rng, 1, 64)
    q_hi = rng.choice([1, 1, 1, rng.randint(2, 8), _log_int(rng, 8, 1024)])
    if op == "bounds":
        hi = _log_int(rng, 1, 200000 // R)
    elif op in ("score", "select_blocks"):
        q_hi = min(q_hi, 1500 * 32 // (R * max(Hq, 8)) + 1)
        hi = _log_int(rng, 1, min(65000, 1200000 // R, max(1, 33000 * 1500 * 32 // (R * q_hi * Hq))))
    elif op == "sparse":
        q_hi = min(q_hi, 300 // R + 1)
        hi = _log_int(rng, 1, min(32768, 1200000 // R))
    else:
        q_hi = min(q_hi, 64 * 16 // R + 1)
        hi = _log_int(rng, 1, min(32768, 240000 // R))
        c |= {"window": rng.choice([0, 0, 1, 16, 33, 64]), "decay": rng.choice([1.0, 0.9])}
        rows = min(q_hi, c["window"] or q_hi) * Hq
        hi = min(hi, max(1, 180000000 // (R * rows)))
    q_hi = min(q_hi, hi)
    if op in ("select_blocks", "sparse"):
        most = max(1, min(256, 48 * 256 * 16 * 8 // (R * q_hi * Hkv * c["B"])))  # as many keys as in the largest listed case
        c["k"] = _log_int(rng, 1, most)
    if op == "select_blocks":
        c["first"] = rng.randint(0, min(2, c["k"]))
        c["last"] = rng.randint(0, min(8, c["k"] - c["first"]))
    q_lo = rng.randint(1, q_hi)
    return {**c, "R": R, "lo": rng.randint(q_hi, hi), "hi": hi, "q_lo": q_lo, "q_hi": q_hi}


def _lengths(case):
    """(query tokens, context lengths with them) of a case's requests."""
    rng = random.Random(case["len_seed"])
    seqs = [rng.randint(case["lo"], case["hi"]) for _ in range(case["R"])]
    qs = [min(n, rng.randint(case["q_lo"], case["q_hi"])) for n in seqs] if "q_lo" in case else [0] * case["R"]
    return qs, seqs


def _blocks(n, B):
    return -(-n // B)


def work(case):
    qs, seqs = _lengths(case)
    op, Hkv, B, D = case["op"], case.get("Hkv", 1), case.get("B", 1), case.get("D", 1)
    cell = Hkv * D * (1 if case.get("dtype") == "fp8" else 2)  # a token's keys
    if op == "bounds":
        blocks = sum(_blocks(n, B) - (n - q) // B for q, n in zip(qs, seqs))
        keys = sum(n - (n - q) // B * B for q, n in zip(qs, seqs))
        return {"bytes": keys * cell + blocks * Hkv * 2 * D * 2, "flops": keys * Hkv * D * 2}
    rows = [n - q + j + 1 for q, n in zip(qs, seqs) for j in range(q)]  # keys that each query may see
    T = len(rows)
    if op == "score":
        pairs = sum(_blocks(m, B) for m in rows)
        read = sum(_blocks(n, B) for n in seqs) * Hkv * 2 * D * 2
        return {"bytes": read + T * case["Hq"] * D * 2 + pairs * Hkv * 4, "flops": pairs * case["Hq"] * D * 4}
    if op == "select_blocks":
        cand = sum(_blocks(m, B) for m in rows) * Hkv
        return {"bytes": cand * 4 + T * Hkv * case["k"] * 4, "flops": cand}
    if op == "select_tokens":
        return {"bytes": sum(seqs) * 4 + case["R"] * case["k"] * 4, "flops": sum(seqs)}
    if op == "sparse":
        pairs = sum(min(case["k"] * B, m) for m in rows)
        held = sum(min(_blocks(n, B), q * case["k"]) * B for q, n in zip(qs, seqs))  # cells read at the least
        return {"bytes": min(pairs, held) * cell * 2 + T * case["Hq"] * D * 4 + T * Hkv * case["k"] * 4,
                "flops": pairs * case["Hq"] * D * 4}
    if op == "mass":
        w = case["window"] or max(qs)
        pairs = sum(min(q, w) * n - min(q, w) * (min(q, w) - 1) // 2 for q, n in zip(qs, seqs)) * case["Hq"]
        return {"bytes": sum(seqs) * (cell + 8) + sum(min(q, w) for q in qs) * case["Hq"] * D * 2,
                "flops": pairs * (2 * D + 4)}
    kept = sum(min(case["k"], n) for n in seqs)
    return {"bytes": kept * (4 * cell + 12), "flops": kept}


# ------------------------------------------------------------------ inputs

def _tables(g, seqs, B, dev):
    """Block tables over shuffled blocks; -1 past a request's own."""
    need = [_blocks(n, B) for n in seqs]
    order = torch.randperm(sum(need) + 3, generator=g, device=dev).int()
    ends = torch.tensor(np.cumsum([0] + need), device=dev)
    i = torch.arange(max(need), device=dev)
    at = ends[:-1, None] + i
    return torch.where(at < ends[1:, None], order[at.clamp(max=sum(need) - 1)], -1).contiguous(), sum(need) + 3


def _stored(g, blocks, case, dev, spread):
    """Keys or values of a pool: [blocks][Hkv][B][D], the tokens of a block alike as far as `spread` says, which lets a
    block be told by its bounds. E4M3 codes stand for themselves times a scale."""
    shape = (blocks, case["Hkv"], case["B"], case["D"])
    x = torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)
    x += torch.randn((blocks, case["Hkv"], 1, case["D"]), generator=g, device=dev, dtype=torch.bfloat16) * spread
    if case["dtype"] == "bf16":
        return x
    return (x * 64.0).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


SCALE_FP8 = 1.0 / 64.0


def _pick(x, k, first, last, n):
    """x [rows][N], the numbers of candidates n [rows] -> the indices of the candidates kept, ascending, [rows][k] with
    -1 behind them: all where there are no more than k, else the first and last ones and the greatest others, of equal
    ones the lower index."""
    i = torch.arange(x.shape[1], device=x.device)
    n = n[:, None]
    forced = (i < first) | (i >= n - last)
    x = x.masked_fill(forced, math.inf).masked_fill(i >= n, -math.inf)
    order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]
    order = order.masked_fill(torch.arange(order.shape[1], device=x.device) >= n, 1 << 30).sort(1).values
    out = torch.full((x.shape[0], k), -1, dtype=torch.int32, device=x.device)
    out[:, : order.shape[1]] = order.masked_fill(order == 1 << 30, -1).int()
    return out


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    qs, seqs = _lengths(case)
    R, T = len(seqs), sum(qs)
    s["seq_host"] = np.array(seqs, np.int32)
    s["seq"] = torch.from_numpy(s["seq_host"]).to(dev)
    if T:
        s["qsl_host"] = np.cumsum([0] + qs).astype(np.int32)
        s["qsl"] = torch.from_numpy(s["qsl_host"]).to(dev)
        # for the plain forms: each query's request, and the keys that it may see
        s["req"] = torch.repeat_interleave(torch.arange(R, device=dev), s["qsl"].long().diff())
        at = torch.arange(T, device=dev) - s["qsl"].long()[s["req"]]
        s["sees"] = (s["seq"].long() - s["qsl"].long().diff())[s["req"]] + at + 1
    if op in ("mass", "select_tokens", "compact"):
        # the weights that each request's tokens have received, in the rows of their slots
        s["slots"] = torch.randperm(R + 2, generator=g, device=dev)[:R].int()
        width = max(seqs) + 5
        s["mass"] = torch.exp(1.5 * torch.randn((R + 2, width), generator=g, device=dev) - 3)
        s["mass_out"] = torch.zeros_like(s["mass"])
    if op == "select_blocks":
        N = _blocks(max(seqs), case["B"])
        s["scores"] = 30 * torch.randn((T, case["Hkv"], N), generator=g, device=dev)
        s["selected"] = torch.zeros((T, case["Hkv"], case["k"]), dtype=torch.int32, device=dev)
    elif op == "select_tokens":
        s["kept"] = torch.zeros((R, case["k"]), dtype=torch.int32, device=dev)
        s["kept_lens"] = torch.zeros(R, dtype=torch.int32, device=dev)
    else:
        s["table"], blocks = _tables(g, seqs, case["B"], dev)
        s["scales"] = (1.0, 1.0) if case["dtype"] == "bf16" else (SCALE_FP8, SCALE_FP8)
    if op in ("bounds", "score"):
        bounds = torch.randn((blocks, case["Hkv"], 2, case["D"]), generator=g, device=dev, dtype=torch.bfloat16)
        bounds += 0.5 * torch.randn((blocks, case["Hkv"], 1, case["D"]), generator=g, device=dev, dtype=torch.bfloat16)
        unit = 1.0 if case["dtype"] == "bf16" else 64.0  # bounds are those of the codes
        s["bounds"] = ((bounds.sort(2).values + torch.tensor([[-1.0], [1.0]], device=dev).bfloat16()) * unit).contiguous()
    if op == "bounds":
        s["k"] = _stored(g, blocks, case, dev, 0.5)
        s["v"] = s["k"]
    if op == "score":
        s["k"] = torch.zeros((blocks, case["Hkv"], case["B"], case["D"]), device=dev,
                             dtype=torch.bfloat16 if case["dtype"] == "bf16" else torch.uint8)
        s["v"] = s["k"]
        s["scores"] = torch.full((T, case["Hkv"], s["table"].shape[1]), -math.inf, device=dev)
    if op in ("sparse", "mass"):
        s["k"], s["v"] = _stored(g, blocks, case, dev, 0.7), None
        s["v"] = _stored(g, blocks, case, dev, 0.0) if op == "sparse" else s["k"]
        s["scale"] = case["D"] ** -0.5
    if op in ("score", "sparse", "mass"):
        s["q"] = torch.randn((T, case["Hq"], case["D"]), generator=g, device=dev).bfloat16()
        s["out"] = torch.zeros_like(s["q"])
    if op == "sparse":
        # what a score of the blocks selects: neighbouring queries mostly the same blocks, the first and newest always
        B, Hkv, N = case["B"], case["Hkv"], s["table"].shape[1]
        x = torch.randn((R, Hkv, N), generator=g, device=dev)[s["req"]]
        x = x + 0.3 * torch.randn((T, Hkv, N), generator=g, device=dev)
        n = ((s["sees"] + B - 1) // B).repeat_interleave(Hkv)
        k = case["k"]
        s["selected"] = _pick(x.view(T * Hkv, N), k, min(1, k - 1), min(2, max(1, k - 1)), n).view(T, Hkv, k).contiguous()
    if op == "compact":
        # the tokens kept move into blocks of their own
        s["kept_lens"] = s["seq"].clamp(max=case["k"])
        N = int(s["seq_host"].max())
        s["kept"] = _pick(torch.randn((R, N), generator=g, device=dev), case["k"], case["first"], case["last"],
                          s["seq"].long()).contiguous()
        new = _blocks(case["k"], case["B"])
        s["k"] = _stored(g, blocks + R * new, case, dev, 0.0)
        s["v"] = _stored(g, blocks + R * new, case, dev, 0.0)
        s["new_table"] = (blocks + torch.randperm(R * new, generator=g, device=dev).int()).view(R, new).contiguous()
    if own:  # what a program that uses the framework keeps beside its tensors
        from paged_kv_cache_143_gb300 import pa

        if "k" in s:
            s["pool"] = pa.KVPool(s["k"], s["v"], *s["scales"])
        if op == "mass":
            n = pa.attention_mass_workspace_size(s["qsl_host"], s["seq_host"], case["Hq"], case["Hkv"],
                                                 window=case["window"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device=dev)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _calls(s)
    return {"bounds": _plain_bounds, "score": _plain_score, "select_blocks": _plain_select_blocks,
            "select_tokens": _plain_select_tokens, "sparse": _plain_sparse, "mass": _plain_mass,
            "compact": _plain_compact}[s["case"]["op"]](s)


def _values(x):
    """A pool's elements as what they stand for."""
    return x.view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x


def _calls(s):
    """A user's calls of the framework."""
    from paged_kv_cache_143_gb300 import pa

    case, op = s["case"], s["case"]["op"]
    if op == "bounds":
        pa.update_block_bounds(s["pool"], s["bounds"], s["table"], s["seq"], query_start_loc=s["qsl"],
                               num_tokens=int(s["qsl_host"][-1]))
        return s["bounds"]
    if op == "score":
        pa.score_blocks(s["q"], s["bounds"], s["scores"], s["qsl"], s["seq"], s["table"], s["pool"])
        return s["scores"]
    if op == "select_blocks":
        pa.select_blocks(s["scores"], s["selected"], s["qsl"], s["seq"], case["B"], first=case["first"],
                         last=case["last"])
        return s["selected"]
    if op == "select_tokens":
        pa.select_tokens(s["mass"], s["kept"], s["kept_lens"], s["seq"], idx_mapping=s["slots"], first=case["first"],
                         last=case["last"])
        return s["kept"], s["kept_lens"]
    if op == "sparse":
        pa.sparse_forward(s["q"], s["out"], s["qsl"], s["seq"], s["table"], s["selected"], s["pool"], s["scale"])
        return s["out"]
    if op == "mass":
        pa.attention_mass(s["q"], s["mass"], s["mass_out"], s["qsl"], s["seq"], s["qsl_host"], s["seq_host"], s["table"],
                          s["pool"], s["scale"], idx_mapping=s["slots"], decay=case["decay"], window=case["window"],
                          workspace=s["workspace"])
        return s["mass_out"]
    pa.compact_cache(s["pool"], s["table"], s["new_table"], s["kept"], s["kept_lens"], mass_in=s["mass"],
                     mass_out=s["mass_out"], idx_mapping=s["slots"])
    return _values(s["k"]), _values(s["v"]), s["mass_out"]


def _plain_bounds(s):
    """The least and the greatest key of each block with a new token, over the block's stored tokens."""
    B, dev = s["case"]["B"], s["seq"].device
    new, n = s["qsl"].long().diff(), s["seq"].long()
    i = torch.arange(s["table"].shape[1], device=dev)
    r, i = torch.nonzero((i >= ((n - new) // B)[:, None]) & (i * B < n[:, None]), as_tuple=True)
    ids = s["table"][r, i].long()
    live = (i[:, None] * B + torch.arange(B, device=dev) < n[r, None])[:, None, :, None]
    x = _values(s["k"][ids]).float()
    top = torch.finfo(torch.bfloat16).max
    lo, hi = x.masked_fill(~live, math.inf).amin(2), x.masked_fill(~live, -math.inf).amax(2)
    s["bounds"][ids] = torch.stack((lo, hi), 2).clamp(-top, top).bfloat16()
    return s["bounds"]


def _plain_score(s):
    case = s["case"]
    T, Hkv, D, g = s["q"].shape[0], case["Hkv"], case["D"], case["Hq"] // case["Hkv"]
    q = s["q"].float().view(T, Hkv, g, D)
    b = s["bounds"].float()[s["table"].clamp(min=0).long()]                       # [R][N][Hkv][2][D]
    q_len = int(np.diff(s["qsl_host"]).max())
    # queries padded to the longest chunk
    at = torch.arange(q_len, device=q.device)
    rows = (s["qsl"].long()[:-1, None] + at).clamp(max=T - 1)                       # [R][J]
    q = q[rows].permute(0, 2, 3, 1, 4).flatten(2, 3)                               # [R][Hkv][g J][D]
    x = q.clamp(min=0) @ b[..., 1, :].permute(0, 2, 3, 1) + q.clamp(max=0) @ b[..., 0, :].permute(0, 2, 3, 1)
    x = x.unflatten(2, (g, q_len)).amax(2).permute(0, 2, 1, 3) * s["scales"][0]    # [R][J][Hkv][N]
    j = torch.arange(T, device=q.device) - s["qsl"].long()[s["req"]]
    x = x[s["req"], j]
    hidden = torch.arange(x.shape[-1], device=q.device) * case["B"] >= s["sees"][:, None, None]
    return x.masked_fill(hidden, -math.inf)


def _plain_select_blocks(s):
    case = s["case"]
    x = s["scores"]
    n = ((s["sees"] + case["B"] - 1) // case["B"]).repeat_interleave(case["Hkv"])
    return _pick(x.flatten(0, 1), case["k"], case["first"], case["last"], n).view(s["selected"].shape)


def _plain_select_tokens(s):
    case = s["case"]
    x = s["mass"][s["slots"].long(), : int(s["seq_host"].max())]
    return _pick(x, case["k"], case["first"], case["last"], s["seq"].long()), s["seq"].clamp(max=case["k"])


def _softmax(x):
    p = torch.exp(x - x.amax(-1, keepdim=True))
    return p / p.sum(-1, keepdim=True)


def _plain_sparse(s):
    case = s["case"]
    T, Hkv, D, g, B = s["q"].shape[0], case["Hkv"], case["D"], case["Hq"] // case["Hkv"], case["B"]
    sel = s["selected"].long()                                                     # [T][Hkv][K]
    ids = s["table"].long()[s["req"][:, None, None], sel.clamp(min=0)].clamp(min=0)
    head = torch.arange(Hkv, device=sel.device)[:, None]
    k = _values(s["k"][ids, head]).float().flatten(2, 3)                           # [T][Hkv][K B][D]
    key = (sel[..., None] * B + torch.arange(B, device=sel.device)).flatten(2)
    q = s["q"].float().view(T, Hkv, g, D) * (s["scale"] * s["scales"][0])
    x = q @ k.mT
    del k
    hidden = (key < 0) | (key >= s["sees"][:, None, None])
    p = _softmax(x.masked_fill_(hidden[:, :, None], -math.inf))
    v = _values(s["v"][ids, head]).float().flatten(2, 3)
    return (p @ v * s["scales"][1]).view(T, case["Hq"], D).bfloat16()


def _plain_mass(s):
    """Requests padded to the longest, their queries to the most that count."""
    case, dev = s["case"], s["seq"].device
    R, Hkv, D, g, B = case["R"], case["Hkv"], case["D"], case["Hq"] // case["Hkv"], case["B"]
    n, new = s["seq"].long(), s["qsl"].long().diff()
    J = min(int(np.diff(s["qsl_host"]).max()), case["window"] or 1 << 30)
    back = torch.arange(J, device=dev)                                             # queries from the last one on
    counts = back < new[:, None]
    rows = (s["qsl"].long()[1:, None] - 1 - back).clamp(min=0)                     # [R][J]
    q = s["q"].float()[rows].view(R, J, Hkv, g, D).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [R][Hkv][g J][D]
    k = _values(s["k"][s["table"].clamp(min=0).long()]).float()                    # [R][N][Hkv][B][D]
    k = k.transpose(1, 2).flatten(2, 3)                                            # [R][Hkv][N B][D]
    x = (q * (s["scale"] * s["scales"][0])) @ k.mT
    del k
    key = torch.arange(x.shape[-1], device=dev)
    x = x.unflatten(2, (g, J))
    x.masked_fill_((key >= n[:, None, None] - back[:, None])[:, None, None], -math.inf)
    x -= x.amax(-1, keepdim=True)
    p = x.exp_()
    p /= p.sum(-1, keepdim=True)
    got = p.masked_fill_(~counts[:, None, None, :, None], 0).sum((1, 2, 3))        # [R][N B]
    width = min(got.shape[1], s["mass"].shape[1])
    got, key = got[:, :width], key[:width]
    old = s["mass"][s["slots"].long(), :width] * case["decay"]
    got = got + old.masked_fill(key >= (n - new)[:, None], 0)
    out = s["mass_out"]
    out[s["slots"].long(), :width] = torch.where(key < n[:, None], got, out[s["slots"].long(), :width])
    return out


def _plain_compact(s):
    B, dev = s["case"]["B"], s["seq"].device
    i = torch.arange(s["kept"].shape[1], device=dev)
    r, i = torch.nonzero(i < s["kept_lens"][:, None], as_tuple=True)
    p = s["kept"][r, i].long()
    src, dst = s["table"][r, p // B].long(), s["new_table"][r, i // B].long()
    s["k"][dst, :, i % B] = s["k"][src, :, p % B]
    s["v"][dst, :, i % B] = s["v"][src, :, p % B]
    slots = s["slots"].long()[r]
    s["mass_out"][slots, i] = s["mass"][slots, p]
    return _values(s["k"]), _values(s["v"]), s["mass_out"]


# ------------------------------------------------------------------ in 64 bits, from the definitions

def _codes64(codes):
    """E4M3 codes as doubles, from their bits."""
    c = codes.long()
    e, m = (c >> 3) & 15, c & 7
    v = torch.where(e == 0, m * 2.0 ** -9, (8 + m).double() * torch.exp2(e.double() - 10))
    return torch.where(c > 127, -v, v)


def _context64(s, which, r, ids, h):
    """Stored rows of blocks `ids` (logical) of request r for one kv head, in order."""
    x = s[which][s["table"][r, ids].long(), h].flatten(0, 1)
    x = _codes64(x) if x.dtype == torch.uint8 else x.double()
    return x * s["scales"][0 if which == "k" else 1]


def exact(case, seed):
    op = case["op"]
    if op in ("select_blocks", "select_tokens", "compact"):
        return None  # whole numbers, or values moved as they are
    s = prepare(case, seed)
    qs, seqs = _lengths(case)
    Hkv, g, B = case["Hkv"], case["Hq"] // case["Hkv"], case["B"]
    starts = [sum(qs[:r]) for r in range(len(qs))]
    if op == "bounds":
        out = s["bounds"].double()
        for r, (q, n) in enumerate(zip(qs, seqs)):
            for h in range(Hkv):
                x = s["k"][s["table"][r, : _blocks(n, B)].long(), h].flatten(0, 1)[:n]
                x = _codes64(x) if x.dtype == torch.uint8 else x.double()
                for i in range((n - q) // B, _blocks(n, B)):
                    out[s["table"][r, i].long(), h] = torch.stack(x[i * B:(i + 1) * B].aminmax(dim=0))
        return out
    if op == "score":
        out = torch.full(s["scores"].shape, -math.inf, dtype=torch.float64, device="cuda")
        for r, (a, q, n) in enumerate(zip(starts, qs, seqs)):
            for h in range(Hkv):
                low, high = s["bounds"][s["table"][r, : _blocks(n, B)].long(), h].double().unbind(1)
                mid, half = (high + low) / 2, (high - low) / 2
                x = s["q"][a:a + q, h * g:(h + 1) * g].double()
                x = (x @ mid.T + x.abs() @ half.T).amax(1) * s["scales"][0]        # the most that the box allows
                m = n - q + 1 + torch.arange(q, device="cuda")
                seen = torch.arange(x.shape[1], device="cuda") * B < m[:, None]
                out[a:a + q, h, : x.shape[1]] = torch.where(seen, x, -math.inf)
        return out
    if op == "sparse":
        if sum(qs) * Hkv > 4000:
            return None
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        sel = s["selected"].cpu()
        for r, (a, q, n) in enumerate(zip(starts, qs, seqs)):
            for j in range(q):
                m = n - q + j + 1
                for h in range(Hkv):
                    ids = sel[a + j, h][sel[a + j, h] >= 0].long().cuda()
                    key = (ids[:, None] * B + torch.arange(B, device="cuda")).flatten()
                    see = key < m
                    k, v = _context64(s, "k", r, ids, h)[see], _context64(s, "v", r, ids, h)[see]
                    x = s["q"][a + j, h * g:(h + 1) * g].double() @ k.T * s["scale"]
                    out[a + j, h * g:(h + 1) * g] = torch.exp(torch.log_softmax(x, -1)) @ v
        return out
    out = s["mass_out"].double()
    for r, (a, q, n) in enumerate(zip(starts, qs, seqs)):
        w = min(q, case["window"] or q)
        got = torch.zeros(n, dtype=torch.float64, device="cuda")
        hidden = torch.arange(n, device="cuda") > (n - w + torch.arange(w, device="cuda"))[:, None]
        for h in range(Hkv):
            k = _context64(s, "k", r, torch.arange(_blocks(n, B), device="cuda"), h)[:n]
            for i in range(h * g, (h + 1) * g):
                x = s["q"][a + q - w:a + q, i].double() @ k.T * s["scale"]
                got += torch.exp(torch.log_softmax(x.masked_fill(hidden, -math.inf), -1)).sum(0)
        slot = int(s["slots"][r])
        got[: n - q] += case["decay"] * s["mass"][slot, : n - q].double()
        out[slot, :n] = got
    return out
