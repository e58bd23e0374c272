"""Cases for the latent-attention path: rotary positions, the latent cache (written, quantised, read back), attention
over it in the absorbed form (the query moved into the latent space, straight on the paged cache) and in the expanded
form (keys and values of every head made from the latents).

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
        # rotary positions of one decode step's queries, cut from the up-projected heads and placed beside the
        # absorbed part: one row per running request
        {"name": "rope-decode-256", "op": "rope", "T": 256, "H": 64, "D": 64, "rot": 64, "interleaved": True,
         "in_width": 192, "out_width": 576, "max_pos": 32768, "stretch": 1.0},
        # the queries of a full token budget of prefill chunks; half of each head turned, context stretched
        {"name": "rope-chunk-8192-partial", "op": "rope", "T": 8192, "H": 32, "D": 128, "rot": 64,
         "interleaved": False, "in_width": 128, "out_width": 128, "max_pos": 131072, "stretch": 8.0},
        # one decode step's new rows into a bf16 cache
        {"name": "store-decode-bf16-256", "op": "store", "T": 256, "L": 512, "B": 16, "dtype": "bf16",
         "spare": 2048, "interleaved": True, "max_pos": 32768},
        # a prefill budget quantised into an E4M3 cache, and those rows read back for the expanded form
        {"name": "store-fetch-fp8-8192", "op": "store", "T": 8192, "L": 512, "B": 64, "dtype": "fp8",
         "spare": 100, "interleaved": True, "max_pos": 131072},
        # the cached contexts of a few long requests read back and widened, ragged
        {"name": "fetch-fp8-long", "op": "fetch", "R": 5, "lo": 9000, "hi": 40000, "len_seed": 3, "L": 512, "B": 32,
         "dtype": "fp8"},
        # the smallest attention calls: a handful of short chats
        {"name": "absorbed-tiny", "op": "absorbed", "R": 4, "lo": 17, "hi": 200, "q_len": 1, "len_seed": 1, "H": 16,
         "L": 512, "B": 16, "dtype": "bf16"},
        # an ordinary decode batch
        {"name": "absorbed-decode-160", "op": "absorbed", "R": 160, "lo": 128, "hi": 2048, "q_len": 1, "len_seed": 2,
         "H": 32, "L": 512, "B": 32, "dtype": "bf16"},
        # a decode batch of a wide layer, every head on one GPU
        {"name": "absorbed-wide-64", "op": "absorbed", "R": 64, "lo": 1000, "hi": 8192, "q_len": 1, "len_seed": 4,
         "H": 128, "L": 512, "B": 64, "dtype": "bf16"},
        # long contexts in an E4M3 cache
        {"name": "absorbed-long-fp8-12", "op": "absorbed", "R": 12, "lo": 20000, "hi": 65000, "q_len": 1,
         "len_seed": 5, "H": 64, "L": 512, "B": 64, "dtype": "fp8"},
        # drafted tokens checked four at a time, an odd head count, a narrower latent
        {"name": "absorbed-draft-24", "op": "absorbed", "R": 24, "lo": 100, "hi": 6000, "q_len": 4, "len_seed": 6,
         "H": 20, "L": 256, "B": 16, "dtype": "bf16"},
        # short prompts prefilled together, ragged
        {"name": "expanded-short", "op": "expanded", "R": 6, "q_lo": 30, "q_hi": 500, "past_hi": 300, "len_seed": 7,
         "H": 16},
        # long chunks behind cached contexts
        {"name": "expanded-long", "op": "expanded", "R": 4, "q_lo": 1900, "q_hi": 4096, "past_hi": 16000,
         "len_seed": 8, "H": 24},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5))))))


def draw(rng):
    op = rng.choice(["rope", "store", "fetch", "absorbed", "absorbed", "absorbed", "expanded", "expanded"])
    if op == "rope":
        D, rot = rng.choice([(64, 64), (64, 32), (96, 96), (128, 128), (128, 64), (80, 32), (192, 64)])
        in_width = D + rng.choice([0, 128])
        H = _log_int(rng, 1, 128)
        return {"op": op, "T": _log_int(rng, 1, max(1, 8192 * 32 * 128 // (H * D))), "H": H, "D": D, "rot": rot,
                "interleaved": rng.random() < 0.5, "in_width": in_width, "out_width": D + rng.choice([0, 256, 512]),
                "max_pos": _log_int(rng, 1, 1 << 20), "stretch": rng.choice([1.0, 4.0, 16.0])}
    if op == "store":
        return {"op": op, "T": _log_int(rng, 1, 8192), "L": rng.choice([256, 512]), "B": rng.choice([16, 32, 64]),
                "dtype": rng.choice(["bf16", "fp8"]), "spare": rng.randint(0, 3000), "interleaved": rng.random() < 0.5,
                "max_pos": _log_int(rng, 1, 1 << 20)}
    if op == "fetch":
        R = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, 100000 // R)
        return {"op": op, "R": R, "lo": rng.randint(1, hi), "hi": hi, "len_seed": rng.randrange(1 << 30),
                "L": rng.choice([256, 512]), "B": rng.choice([16, 32, 64]), "dtype": rng.choice(["bf16", "fp8"])}
    if op == "absorbed":
        R = _log_int(rng, 1, 192)
        q_len = rng.choice([1, 1, 1, 1, 2, 3, 5, 8])
        H = rng.choice([1, 5, 8, 16, 20, 32, 40, 64, 96, 128, 128])
        H = min(H, 512 // q_len)
        # keys x (query rows read with them) stays below the largest listed case's
        most = 500000 * 64 // max(64, q_len * H)
        hi = max(q_len, _log_int(rng, q_len, max(q_len, min(65000, most // R))))
        return {"op": op, "R": R, "lo": rng.randint(q_len, hi), "hi": hi, "q_len": q_len,
                "len_seed": rng.randrange(1 << 30), "H": H, "L": rng.choice([256, 512, 512]),
                "B": rng.choice([16, 32, 64]), "dtype": rng.choice(["bf16", "fp8"])}
    R = _log_int(rng, 1, 8)
    q_hi = _log_int(rng, 1, 4000 * 2 // (R + 1))
    return {"op": op, "R": R, "q_lo": rng.randint(1, q_hi), "q_hi": q_hi,
            "past_hi": rng.choice([0, _log_int(rng, 1, 16000 * 2 // (R + 1))]), "len_seed": rng.randrange(1 << 30),
            "H": _log_int(rng, 1, 24)}


def _lengths(case):
    """Context lengths (fetch, absorbed) or (query, context) lengths (expanded) of a case's requests."""
    rng = random.Random(case["len_seed"])
    if case["op"] == "expanded":
        q = [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(case["R"])]
        return q, [n + rng.randint(0, case["past_hi"]) for n in q]
    return [rng.randint(case["lo"], case["hi"]) for _ in range(case["R"])]


def work(case):
    op = case["op"]
    if op == "rope":
        n = case["T"] * case["H"]
        return {"bytes": n * case["D"] * 4 + case["T"] * 4, "flops": n * case["rot"] * 3}
    cell = {"bf16": 2, "fp8": 1}.get(case.get("dtype"), 2)
    if op in ("store", "fetch"):
        rows = case["T"] if op == "store" else sum(_lengths(case))
        wide = rows * (case["L"] + ROPE) * 2
        held = rows * (case["L"] * cell + ROPE * 2 + (4 if cell == 1 else 0))
        if op == "fetch":
            return {"bytes": held + wide, "flops": rows * case["L"]}
        both = 2 if cell == 1 else 1  # quantised rows are read back
        return {"bytes": both * (held + wide) + rows * 12, "flops": rows * (case["L"] + ROPE * 3)}
    if op == "absorbed":
        L, q, H = case["L"], case["q_len"], case["H"]
        seqs = _lengths(case)
        pairs = sum(q * s - q * (q - 1) // 2 for s in seqs) * H
        cache = sum(seqs) * (L * cell + ROPE * 2 + (4 if cell == 1 else 0))
        return {"bytes": cache + case["R"] * q * H * (2 * L + ROPE) * 2, "flops": pairs * 2 * (2 * L + ROPE)}
    qs, ks = _lengths(case)
    pairs = sum(q * k - q * (q - 1) // 2 for q, k in zip(qs, ks)) * case["H"]
    H = case["H"]
    size = sum(qs) * H * (NOPE + ROPE + WIDE_V) + sum(ks) * (H * (NOPE + WIDE_V) + ROPE)
    return {"bytes": size * 2, "flops": pairs * 2 * (NOPE + ROPE + WIDE_V)}


# ------------------------------------------------------------------ inputs

ROPE, NOPE, WIDE_V = 64, 128, 128  # rotary part of a key; the other part and the value of an expanded head


def _frequencies(rot, stretch, dev):
    """Inverse frequencies of the rotary pairs; a stretched context divides the slow ones and keeps the fast ones,
    with a linear ramp between."""
    i = torch.arange(rot // 2, dtype=torch.float64, device=dev)
    f = 10000.0 ** (-2.0 * i / rot)
    if stretch != 1.0:
        turns = 4096 * f / (2 * math.pi)  # turns over the context seen in training
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        f = f * keep + f / stretch * (1 - keep)
    return f.float()


def _bf16(g, shape, dev, mult=1.0):
    return (torch.randn(shape, generator=g, device=dev) * mult).bfloat16()


def _cache(g, blocks, case, dev):
    """A cache whose every cell is written: bf16 rows, or E4M3 codes with a power-of-two scale for each row."""
    B, L = case["B"], case["L"]
    rope = _bf16(g, (blocks, B, ROPE), dev)
    latent = _bf16(g, (blocks, B, L), dev)
    if case["dtype"] == "bf16":
        return latent, rope, None
    scales = torch.exp2(torch.randint(-7, -4, (blocks, B), generator=g, device=dev).float())
    codes = (latent.float() / scales[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), rope, scales


def _tables(g, seqs, B, dev):
    """Block tables over shuffled blocks; -1 past a request's own."""
    need = [(s + B - 1) // B for s in seqs]
    total = sum(need) + 3
    order = torch.randperm(total, generator=g, device=dev).int()
    tab = torch.full((len(seqs), max(need)), -1, dtype=torch.int32, device=dev)
    at = 0
    for r, n in enumerate(need):
        tab[r, :n] = order[at:at + n]
        at += n
    return tab, total


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    if op == "rope":
        T, H, D = case["T"], case["H"], case["D"]
        x = _bf16(g, (T, H, case["in_width"]), dev)
        out = torch.zeros((T, H, case["out_width"]), dtype=torch.bfloat16, device=dev)
        s["x"], s["out"] = x[..., case["in_width"] - D:], out[..., case["out_width"] - D:]
        s["positions"] = torch.randint(0, case["max_pos"], (T,), generator=g, device=dev, dtype=torch.int32)
        s["inv_freq"] = _frequencies(case["rot"], case["stretch"], dev)
        s["factor"] = 1.0 + 0.1 * math.log(case["stretch"])
    elif op == "store":
        T, L, B = case["T"], case["L"], case["B"]
        blocks = (T + case["spare"] + B - 1) // B
        s["pool"] = _cache(g, blocks, case, dev)
        s["latent"] = _bf16(g, (T, L), dev) * torch.exp2(torch.randn((T, 1), generator=g, device=dev)).bfloat16()
        s["k_rope"] = _bf16(g, (T, ROPE), dev)
        s["positions"] = torch.randint(0, case["max_pos"], (T,), generator=g, device=dev, dtype=torch.int32)
        s["inv_freq"] = _frequencies(ROPE, 1.0, dev)
        order = torch.randperm(blocks, generator=g, device=dev)
        s["table"] = order[: (T + B - 1) // B].int()[None].contiguous()
        t = torch.arange(T, device=dev)
        s["slots"] = order[t // B] * B + t % B
        s["start"] = torch.tensor([0, T], dtype=torch.int32, device=dev)
        if case["dtype"] == "fp8":
            s["latent_out"] = torch.empty((T, L), dtype=torch.bfloat16, device=dev)
            s["rope_out"] = torch.empty((T, ROPE), dtype=torch.bfloat16, device=dev)
    elif op == "fetch":
        seqs = _lengths(case)
        s["table"], blocks = _tables(g, seqs, case["B"], dev)
        s["pool"] = _cache(g, blocks, case, dev)
        s["start"] = torch.tensor(np.cumsum([0] + seqs), dtype=torch.int32, device=dev)
        s["latent_out"] = torch.empty((sum(seqs), case["L"]), dtype=torch.bfloat16, device=dev)
        s["rope_out"] = torch.empty((sum(seqs), ROPE), dtype=torch.bfloat16, device=dev)
    elif op == "absorbed":
        seqs, q, H, L = _lengths(case), case["q_len"], case["H"], case["L"]
        s["table"], blocks = _tables(g, seqs, case["B"], dev)
        s["pool"] = _cache(g, blocks, case, dev)
        s["q"] = _bf16(g, (len(seqs) * q, H, L + ROPE), dev)
        s["out"] = torch.empty((len(seqs) * q, H, L), dtype=torch.bfloat16, device=dev)
        s["seq_host"] = np.array(seqs, np.int32)
        s["qsl_host"] = np.arange(len(seqs) + 1, dtype=np.int32) * np.int32(q)
        s["seq"], s["qsl"] = torch.from_numpy(s["seq_host"]).to(dev), torch.from_numpy(s["qsl_host"]).to(dev)
        s["scale"] = (NOPE + ROPE) ** -0.5
    else:
        qs, ks = _lengths(case)
        H = case["H"]
        s["q"] = _bf16(g, (sum(qs), H, NOPE + ROPE), dev)
        kv = _bf16(g, (sum(ks), H, NOPE + WIDE_V), dev)  # one product makes a head's key part and value together
        s["k_nope"], s["v"] = kv[..., :NOPE], kv[..., NOPE:]
        s["k_rope"] = _bf16(g, (sum(ks), ROPE), dev)
        s["out"] = torch.empty((sum(qs), H, WIDE_V), dtype=torch.bfloat16, device=dev)
        s["qsl_host"] = np.cumsum([0] + qs).astype(np.int32)
        s["ksl_host"] = np.cumsum([0] + ks).astype(np.int32)
        s["qsl"], s["ksl"] = torch.from_numpy(s["qsl_host"]).to(dev), torch.from_numpy(s["ksl_host"]).to(dev)
        s["scale"] = (NOPE + ROPE) ** -0.5
    if own:  # what a program that uses the framework keeps beside its tensors
        from paged_kv_cache_143_gb300 import pa

        if "pool" in s:
            s["handle"] = pa.LatentPool(*s["pool"])
        if op == "absorbed":
            n = pa.latent_workspace_size(case["H"], case["L"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device=dev)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _calls(s)
    return {"rope": _plain_rope, "store": _plain_store, "fetch": _plain_fetch, "absorbed": _plain_absorbed,
            "expanded": _plain_expanded}[s["case"]["op"]](s)


def _calls(s):
    """A user's calls of the framework."""
    from paged_kv_cache_143_gb300 import pa

    case, op = s["case"], s["case"]["op"]
    if op == "rope":
        pa.rope(s["x"], s["out"], s["positions"], s["inv_freq"], interleaved=case["interleaved"], factor=s["factor"])
        return s["out"]
    if op == "store":
        pa.write_latent(s["handle"], s["latent"], s["k_rope"], s["slots"], positions=s["positions"],
                        inv_freq=s["inv_freq"], interleaved=case["interleaved"])
        if case["dtype"] == "bf16":
            return s["pool"][0], s["pool"][1]
    if op in ("store", "fetch"):
        pa.read_latent(s["handle"], s["table"], s["start"], s["latent_out"], s["rope_out"])
        return s["latent_out"], s["rope_out"]
    if op == "absorbed":
        pa.latent_forward(s["q"], s["out"], s["qsl"], s["seq"], s["qsl_host"], s["seq_host"], s["table"], s["handle"],
                          s["scale"], workspace=s["workspace"])
        return s["out"]
    pa.latent_prefill(s["q"], s["k_nope"], s["k_rope"], s["v"], s["out"], s["qsl"], s["ksl"], s["qsl_host"],
                      s["ksl_host"], s["scale"])
    return s["out"]


def _turn(x, positions, inv_freq, interleaved, factor):
    """The leading 2 * len(inv_freq) columns of x [T][H][D] turned by position * frequency (angles in 64 bits)."""
    angle = positions.double()[:, None, None] * inv_freq.double()
    cos, sin = (angle.cos() * factor).float(), (angle.sin() * factor).float()
    n = inv_freq.numel()
    rot, rest = x[..., :2 * n].float(), x[..., 2 * n:]
    if interleaved:
        a, b = rot[..., 0::2], rot[..., 1::2]
        rot = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = rot[..., :n], rot[..., n:]
        rot = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((rot.to(x.dtype), rest), -1)


def _plain_rope(s):
    s["out"].copy_(_turn(s["x"], s["positions"], s["inv_freq"], s["case"]["interleaved"], s["factor"]))
    return s["out"]


def _plain_store(s):
    case = s["case"]
    latent, rope, scales = s["pool"]
    turned = _turn(s["k_rope"][:, None], s["positions"], s["inv_freq"], case["interleaved"], 1.0)[:, 0]
    rope.view(-1, ROPE)[s["slots"]] = turned
    if scales is None:
        latent.view(-1, case["L"])[s["slots"]] = s["latent"]
        return latent, rope
    x = s["latent"].float()
    # the smallest power of two that brings the row's largest magnitude to 448 = 0.875 * 2^9 or below
    m, e = torch.frexp(x.abs().amax(-1))
    scale = torch.where(m > 0, torch.exp2((e - 9 + (m > 0.875)).float()), 1.0)
    codes = (x / scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    latent.view(-1, case["L"])[s["slots"]] = codes
    scales.view(-1)[s["slots"]] = scale
    return _plain_fetch(s)


def _plain_rows(s, rows):
    """Cache rows as 32-bit values: latents, rotary parts."""
    latent, rope, scales = s["pool"]
    L = s["case"]["L"]
    rot = rope.view(-1, ROPE)[rows].float()
    if scales is None:
        return latent.view(-1, L)[rows].float(), rot
    codes = latent.view(-1, L)[rows].view(torch.float8_e4m3fn).float()
    return codes * scales.view(-1)[rows][..., None], rot


def _plain_fetch(s):
    B, start = s["case"]["B"], s["start"]
    t = torch.arange(s["latent_out"].shape[0], device=start.device)
    r = torch.searchsorted(start, t, right=True) - 1
    pos = t - start[r]
    latent, rot = _plain_rows(s, s["table"][r, pos // B].long() * B + pos % B)
    return latent.bfloat16(), rot.bfloat16()


def _softmax(x):
    p = torch.exp(x - x.amax(-1, keepdim=True))
    return p / p.sum(-1, keepdim=True)


def _plain_absorbed(s):
    case = s["case"]
    R, q_len, H, L, B = case["R"], case["q_len"], case["H"], case["L"], case["B"]
    dev = s["q"].device
    n = torch.arange(int(s["seq_host"].max()), device=dev)  # key positions, requests padded to the longest
    rows = s["table"].clamp(min=0).long()[:, n // B] * B + n % B
    latent, rot = _plain_rows(s, rows)                                            # [R][N][L], [R][N][ROPE]
    q = s["q"].float().view(R, q_len * H, L + ROPE)
    x = (q[..., :L] @ latent.mT + q[..., L:] @ rot.mT) * s["scale"]
    last = s["seq"].long()[:, None] - q_len + torch.arange(q_len, device=dev)     # [R][q]: the last visible key
    x = x.view(R, q_len, H, -1).masked_fill(n > last[:, :, None, None], -math.inf)
    p = _softmax(x).view(R, q_len * H, -1)
    return (p @ latent).view(R * q_len, H, L).bfloat16()


def _plain_expanded(s):
    """Requests padded to the longest on both sides."""
    dev, H = s["q"].device, s["case"]["H"]
    qsl, ksl = s["qsl"].long(), s["ksl"].long()
    q_len, k_len = qsl.diff(), ksl.diff()
    i = torch.arange(int(np.diff(s["qsl_host"]).max()), device=dev)
    n = torch.arange(int(np.diff(s["ksl_host"]).max()), device=dev)
    live = i < q_len[:, None]                                                      # [R][I]
    q = s["q"].float()[(qsl[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)]         # [R][I][H][192]
    k_rows = (ksl[:-1, None] + n).clamp(max=s["k_rope"].shape[0] - 1)
    k, v = s["k_nope"].float()[k_rows], s["v"].float()[k_rows]                      # [R][N][H][128]
    kr = s["k_rope"].float()[k_rows]                                               # [R][N][64]
    q, k, v = q.transpose(1, 2), k.transpose(1, 2), v.transpose(1, 2)
    x = (q[..., :NOPE] @ k.mT + q[..., NOPE:] @ kr[:, None].mT) * s["scale"]        # [R][H][I][N]
    last = (k_len - q_len)[:, None] + i                                            # [R][I]
    x.masked_fill_(n > last[:, None, :, None], -math.inf)
    out = (_softmax(x) @ v).transpose(1, 2)                                        # [R][I][H][128]
    return out[live].bfloat16()


# ------------------------------------------------------------------ in 64 bits, from the definitions

def _turned64(x, pos, freq, interleaved, factor):
    """Each pair as a complex number times factor * e^(i * angle)."""
    x = x.double()
    n = freq.numel()
    if interleaved:
        z = torch.view_as_complex(x[..., :2 * n].reshape(*x.shape[:-1], n, 2).contiguous())
    else:
        z = torch.complex(x[..., :n].contiguous(), x[..., n:2 * n].contiguous())
    z = z * torch.polar(torch.full_like(z.real, factor), pos.double()[:, None, None] * freq.double() + 0 * z.real)
    y = x.clone()
    if interleaved:
        y[..., 0:2 * n:2], y[..., 1:2 * n:2] = z.real, z.imag
    else:
        y[..., :n], y[..., n:2 * n] = z.real, z.imag
    return y


def _e4m3_64(x):
    """Doubles rounded to the nearest E4M3 value, ties to the even one: steps of 2^-9 up to 2^-6, eight steps to a
    power of two above."""
    _, e = torch.frexp(x.abs())
    step = torch.exp2((e - 4).clamp(min=-9).double())
    return (torch.round(x / step) * step).clamp(-448, 448)


def _codes64(codes):
    """E4M3 codes as doubles, from their bits."""
    c = codes.long()
    e, m = (c >> 3) & 15, c & 7
    v = torch.where(e == 0, m * 2.0 ** -9, (8 + m).double() * torch.exp2(e.double() - 10))
    return torch.where(c > 127, -v, v)


def _context64(s, r, length):
    """Latents and rotary parts of a request's cached tokens."""
    latent, rope, scales = s["pool"]
    blocks = s["table"][r, : -(-length // s["case"]["B"])].long()
    rot = rope[blocks].double().flatten(0, 1)[:length]
    if scales is None:
        return latent[blocks].double().flatten(0, 1)[:length], rot
    vals = _codes64(latent[blocks]) * scales[blocks].double()[..., None]
    return vals.flatten(0, 1)[:length], rot


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        return _turned64(s["x"], s["positions"], s["inv_freq"], case["interleaved"], s["factor"])
    if op == "store":
        turned = _turned64(s["k_rope"][:, None], s["positions"], s["inv_freq"], case["interleaved"], 1.0)[:, 0]
        if case["dtype"] == "bf16":
            latent, rope = s["pool"][0].double(), s["pool"][1].double()
            latent.view(-1, case["L"])[s["slots"]] = s["latent"].double()
            rope.view(-1, ROPE)[s["slots"]] = turned
            return latent, rope
        x = s["latent"].double()
        scale = torch.exp2(torch.ceil(torch.log2(x.abs().amax(-1, keepdim=True) / 448)))
        return _e4m3_64(x / scale) * scale, turned
    if op == "fetch":
        rows = [_context64(s, r, n) for r, n in enumerate(_lengths(case))]
        return torch.cat([a for a, _ in rows]), torch.cat([b for _, b in rows])
    if op == "absorbed":
        outs = []
        for r, n in enumerate(_lengths(case)):
            c, k = _context64(s, r, n)
            q = s["q"][r * case["q_len"]:(r + 1) * case["q_len"]].double()
            for j in range(case["q_len"]):
                m = n - case["q_len"] + j + 1
                w = torch.exp(torch.log_softmax(q[j] @ torch.cat((c, k), -1)[:m].T * s["scale"], -1))
                outs.append(w @ c[:m])
        return torch.stack(outs)
    qs, ks = s["qsl_host"], s["ksl_host"]
    outs = []
    for r in range(case["R"]):
        a, b, c, d = int(qs[r]), int(qs[r + 1]), int(ks[r]), int(ks[r + 1])
        hidden = torch.ones((b - a, d - c), device=s["q"].device).triu(d - c - (b - a) + 1) > 0
        heads = []
        for h in range(case["H"]):
            k = torch.cat((s["k_nope"][c:d, h], s["k_rope"][c:d]), -1).double()
            x = s["q"][a:b, h].double() @ k.T * s["scale"]
            heads.append(torch.softmax(x.masked_fill(hidden, -math.inf), -1) @ s["v"][c:d, h].double())
        outs.append(torch.stack(heads, 1))
    return torch.cat(outs)
