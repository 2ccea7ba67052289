"""Plain forms and cases of rotary positions and of the paged 16-bit cache.

Three operators of a serving step whose keys are rotated by their positions and kept in 16 bits:

  rope            rotates the heads of query and key rows by their positions
  kv16_append     a step's new keys and values into the cache's pages, keys and queries rotated on the way
  kv16_attention  causal attention of a step's new rows, one to thousands a request, over that cache

`run` computes them with elementary torch operations, or (`own`) with the framework's entry points.
A request's token p sits in row p % 64 of the page that its block table names for block p / 64. The new rows of
request b are rows row_start[b] .. row_start[b + 1] - 1 of the step, at positions lens[b] onwards.
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = 64
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}

# how the frequencies of a longer context follow from the trained ones
PLAIN = {"kind": "none"}
LINEAR = {"kind": "linear", "factor": 4.0}
NTK = {"kind": "ntk", "factor": 8.0}
BANDS = {"kind": "bands", "factor": 8.0, "low": 1.0, "high": 4.0, "trained": 8192}
YARN = {"kind": "yarn", "factor": 16.0, "fast": 32.0, "slow": 1.0, "trained": 4096}
SCALINGS = {"none": PLAIN, "linear": LINEAR, "ntk": NTK, "bands": BANDS, "yarn": YARN}


def listed():
    return [
        # queries and keys of a sequence draft, 16 requests of five rows each, far into a long context
        {"name": "rope_draft", "op": "rope", "T": 80, "heads": 72, "more": 8, "D": 128, "rot": 128, "inter": False,
         "scaling": "bands", "base": 500000.0, "far": 131071, "inverse": False, "type": "bf16"},
        # prompts' rows, half of each head rotated, adjacent pairs
        {"name": "rope_partial", "op": "rope", "T": 4093, "heads": 40, "more": 0, "D": 128, "rot": 64, "inter": True,
         "scaling": "yarn", "base": 10000.0, "far": 65000, "inverse": False, "type": "f16"},
        # the way back (a gradient, or keys taken to other positions) for a full chunk of rows
        {"name": "rope_back", "op": "rope", "T": 16381, "heads": 72, "more": 8, "D": 128, "rot": 128, "inter": False,
         "scaling": "none", "base": 500000.0, "far": 16381, "inverse": True, "type": "bf16"},
        # one decoded token a request, one layer
        {"name": "append_step", "op": "append", "B": 64, "n": 1, "per": 0, "every": 1, "pad": 0, "H": 64, "Hkv": 8,
         "D": 128, "lo": 40, "hi": 8100, "rot": 128, "inter": False, "scaling": "bands", "base": 500000.0, "type": "bf16"},
        # prompts of different lengths beside decoding requests, the step's last rows unused
        {"name": "append_prompts", "op": "append", "B": 13, "n": 1, "per": 2003, "every": 2, "pad": 37, "H": 64, "Hkv": 8,
         "D": 128, "lo": 0, "hi": 4100, "rot": 128, "inter": False, "scaling": "bands", "base": 500000.0, "type": "bf16"},
        # a lone decoding request
        {"name": "attn_one", "op": "attn", "B": 1, "n": 1, "per": 0, "every": 1, "pad": 0, "H": 64, "Hkv": 8, "D": 128,
         "lo": 1003, "hi": 1003, "window": 0, "type": "bf16"},
        # a sequence draft's rows for 16 requests
        {"name": "attn_chain", "op": "attn", "B": 16, "n": 5, "per": 0, "every": 1, "pad": 0, "H": 64, "Hkv": 8, "D": 128,
         "lo": 4096, "hi": 8191, "window": 0, "type": "bf16"},
        # long contexts, one token each
        {"name": "attn_long", "op": "attn", "B": 4, "n": 1, "per": 0, "every": 1, "pad": 0, "H": 64, "Hkv": 8, "D": 128,
         "lo": 120001, "hi": 131071, "window": 0, "type": "bf16"},
        # prompts of different lengths from their first token, one query head for each key/value head
        {"name": "attn_prompts", "op": "attn", "B": 7, "n": 1, "per": 1501, "every": 1, "pad": 0, "H": 16, "Hkv": 16,
         "D": 128, "lo": 0, "hi": 0, "window": 0, "type": "bf16"},
        # a long prompt's next chunk
        {"name": "attn_chunk", "op": "attn", "B": 1, "n": 2048, "per": 0, "every": 1, "pad": 0, "H": 64, "Hkv": 8,
         "D": 128, "lo": 30720, "hi": 30720, "window": 0, "type": "bf16"},
        # chunks of some requests beside decoding ones, narrow heads, a sliding window
        {"name": "attn_mixed", "op": "attn", "B": 49, "n": 1, "per": 1003, "every": 8, "pad": 11, "H": 24, "Hkv": 8,
         "D": 64, "lo": 100, "hi": 16000, "window": 4096, "type": "f16"},
    ]


def _spread(rng, lo, hi):
    """An integer of lo .. hi, over its logarithm where that spans more than a factor of ten."""
    if hi > 10 * max(lo, 1):
        return int(round(np.exp(rng.uniform(np.log(max(lo, 1)), np.log(hi))))) if rng.random() > 0.03 else lo
    return rng.randint(lo, hi)


def _draw_rotation(rng, D):
    return {"rot": rng.choice([D, D, D // 2, D // 4]), "inter": rng.random() < 0.4,
            "scaling": rng.choice(sorted(SCALINGS)), "base": rng.choice([10000.0, 500000.0])}


def draw(rng: random.Random):
    op = rng.choice(["rope", "append", "attn", "attn"])
    D = rng.choice([64, 128, 128])
    if op == "rope":
        heads, more = _spread(rng, 1, 96), rng.choice([0, 8])
        kind = rng.choice(["bf16", "bf16", "f16", "f32"])
        most = 16381 * 72 * 128 // ((heads + more) * D) // (2 if kind == "f32" else 1)
        return {"op": op, "T": _spread(rng, 1, min(most, 32768)), "heads": heads, "more": more, "D": D,
                **_draw_rotation(rng, D), "far": _spread(rng, 16, 1 << 20), "inverse": rng.random() < 0.3, "type": kind}
    hkv = rng.choice([1, 2, 4, 8, 16])
    g = rng.choice([1, 2, 3, 4, 5, 8, 16])
    shape = {"H": hkv * g, "Hkv": hkv, "D": D, "type": rng.choice(["bf16", "bf16", "f16"]),
             "pad": rng.choice([0, 0, 1, 29])}
    B = _spread(rng, 1, 100)
    hi = _spread(rng, 1, 8191)
    if op == "append":
        most = 14000 * 80 * 128 // ((g + 2) * hkv * D * 2)  # rows of the largest listed case, a request's twice the mean
        per = rng.choice([0, 1]) * _spread(rng, 1, max(1, min(most // B, 8192)))
        return {"op": op, "B": B, "n": rng.randint(0 if per else 1, 8), "per": per, "every": rng.choice([1, 1, 2, 5]),
                "lo": rng.choice([0, hi // 2, hi]), "hi": hi, **_draw_rotation(rng, D), **shape}
    window = rng.choice([0, 0, 0, _spread(rng, 1, 8192)])
    per, n = 0, rng.choice([1, rng.randint(2, 9), rng.randint(10, 64)])
    if rng.random() < 0.5:
        per, n = _spread(rng, 1, 4096 // B + 1), rng.choice([0, 1])
    # no more keys than the long contexts hold and no more scores than the chunk computes
    most = min(4_000_000 // (B * hkv), 64 * 2048 * 31000 // (B * hkv * g * (2 * per + n)) - 2 * per)
    hi = _spread(rng, 1, max(2, min(most, 131071)))
    return {"op": op, "B": B, "n": n, "per": per, "every": rng.choice([1, 1, 3, 8]) if per else 1,
            "lo": rng.choice([0, hi // 2, hi]), "hi": hi, "window": window, **shape}


# ------------------------------------------------------------------ inputs

def _lens(c, seed):
    """Tokens in the cache before the step, lo to hi, the same ones for every seed in another order."""
    step = np.arange(c["B"]) * 0.6180339887 % 1.0
    v = np.minimum(np.floor(c["lo"] + (c["hi"] - c["lo"] + 1) * step).astype(np.int64), c["hi"])
    return np.roll(v, seed % c["B"])


def _counts(c, seed):
    """Rows that each request brings: n, or for every `every`-th one a chunk of 0 .. 2 * per."""
    b = np.arange(c["B"])
    v = np.full(c["B"], c["n"], np.int64)
    if c["per"]:
        chunk = np.round(((b + 1) * 0.7548776662 % 1.0) * 2 * c["per"]).astype(np.int64)
        v = np.where(b % c["every"] == 0, chunk, v)
    return np.roll(v, seed % c["B"])


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _frequencies(c, device):
    """Angle a position of each pair, float64 [rot / 2], and the factor on what is rotated."""
    s = SCALINGS[c["scaling"]]
    d, base = c["rot"], c["base"]
    i = torch.arange(d // 2, dtype=torch.float64, device=device)
    if s["kind"] == "ntk":
        base = base * s["factor"] ** (d / (d - 2))
    f = base ** (-2.0 * i / d)
    if s["kind"] == "linear":
        f = f / s["factor"]
    if s["kind"] == "bands":  # short waves kept, long ones stretched, between them a blend
        turns = s["trained"] * f / (2 * math.pi)  # of the trained context
        keep = ((turns - s["low"]) / (s["high"] - s["low"])).clamp(0, 1)
        f = f * keep + f / s["factor"] * (1 - keep)
    if s["kind"] == "yarn":  # a ramp over the pairs between two numbers of turns
        at = [d * math.log(s["trained"] / (s[x] * 2 * math.pi)) / (2 * math.log(base)) for x in ("fast", "slow")]
        first, last = max(math.floor(at[0]), 0), min(math.ceil(at[1]), d - 1)
        ramp = ((i - first) / max(last - first, 1e-3)).clamp(0, 1)
        f = f / s["factor"] * ramp + f * (1 - ramp)
    return f, (0.1 * math.log(s["factor"]) + 1.0 if s["kind"] == "yarn" else 1.0)


def _handle(c):
    """What a user's program keeps for its rotation."""
    if not own:
        return _frequencies(c, "cuda")
    import speculative_decode_verify_w4a16_gb300 as sv

    return sv.rope_frequencies(c["rot"], c["base"], scaling=SCALINGS[c["scaling"]], interleaved=c["inter"])


def _table(rng, blocks, spare):
    """A block table with each request's pages anywhere in the cache."""
    pages = int(blocks.sum()) + spare
    table = np.full((len(blocks), max(int(blocks.max()), 1)), -1, np.int32)
    mask = np.arange(table.shape[1])[None, :] < blocks[:, None]
    table[mask] = rng.permutation(pages).astype(np.int32)[:int(blocks.sum())]
    return table, pages


def prepare(case, seed):
    c = case
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 1000003 + 29)

    def randn(*shape):
        kind = torch.float32 if c["type"] == "f32" else torch.bfloat16
        return torch.randn(*shape, generator=gen, device="cuda", dtype=kind).to(TYPES[c["type"]])

    D = c["D"]
    if c["op"] == "rope":
        return {"case": c, "rows": randn(c["T"], c["heads"] + c["more"], D), "freqs": _handle(c),
                "positions": _dev(rng.integers(0, c["far"] + 1, c["T"]).astype(np.int32))}
    lens, cnt = _lens(c, seed), _counts(c, seed)
    T, H, Hkv = int(cnt.sum()) + c["pad"], c["H"], c["Hkv"]
    start = np.concatenate([[0], np.cumsum(cnt)])
    s = {"case": c, "lens": _dev(lens.astype(np.int32)), "start": _dev(start.astype(np.int32)),
         "host_lens": lens.tolist(), "host_start": start.tolist()}
    blocks = -(-(lens + cnt) // BLOCK)
    if c["op"] == "append":  # the cache holds only the pages that this step writes
        first = lens // BLOCK
        table, pages = _table(rng, np.where(cnt > 0, blocks - first, 0), 1)
        wide = np.full((c["B"], int(blocks.max()) + 1), -1, np.int32)
        for b in range(c["B"]):
            own_blocks = int(blocks[b] - first[b]) if cnt[b] else 0
            wide[b, first[b]:first[b] + own_blocks] = table[b, :own_blocks]
        s["table"], s["freqs"] = _dev(wide), _handle(c)
        # the rows of the fused projection: q, k and v side by side
        s["qkv"] = randn(T, H + 2 * Hkv, D)
        s["q_out"] = torch.zeros(T, H, D, dtype=TYPES[c["type"]], device="cuda")
        for x in ("k", "v"):
            s[x] = torch.zeros(1, pages, Hkv, BLOCK, D, dtype=TYPES[c["type"]], device="cuda")
        return s
    table, pages = _table(rng, blocks, 3)
    s["table"] = _dev(table)
    chan = torch.exp(0.5 * torch.randn(Hkv, 1, D, generator=gen, device="cuda")).to(TYPES[c["type"]])
    for x in ("k", "v"):  # a cache in use, the step's own keys and values in it
        s[x] = randn(1, pages, Hkv, BLOCK, D)
        if x == "k":
            s[x] *= chan  # channels of unlike size
    s["q"] = randn(T, H, D)
    s["out"] = torch.zeros(T, H, D, dtype=TYPES[c["type"]], device="cuda")
    return s


# ------------------------------------------------------------- plain forms

def _rotate(x, positions, freqs, inter, inverse=False):
    """x [T, heads, D], angles in float64, the rotation in float32; not rounded."""
    f, factor = freqs
    a = positions.double()[:, None] * f[None, :]
    if inverse:
        a = -a
    cos, sin = ((t(a) * factor).float()[:, None, :] for t in (torch.cos, torch.sin))
    x = x.float()
    rot = 2 * f.numel()
    y = x.clone()
    if inter:
        u, v = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = u * cos - v * sin, v * cos + u * sin
    else:
        u, v = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = u * cos - v * sin, v * cos + u * sin
    return y


def _rope(s):
    c = s["case"]
    x = s["rows"][:, :c["heads"]]
    return _rotate(x, s["positions"], s["freqs"], c["inter"], c["inverse"]).to(x.dtype)


def _append(s):
    c = s["case"]
    H, Hkv, dt = c["H"], c["Hkv"], TYPES[c["type"]]
    start, lens = s["start"].long(), s["lens"].long()
    rows = s["host_start"][-1]
    i = torch.arange(rows, device=start.device)
    b = torch.searchsorted(start[1:], i, right=True)
    pos = lens[b] + i - start[b]
    page, row = s["table"][b, pos // BLOCK].long(), pos % BLOCK
    q, k, v = s["qkv"][:rows].split((H, Hkv, Hkv), 1)
    s["q_out"][:rows] = _rotate(q, pos, s["freqs"], c["inter"]).to(dt)
    s["k"][0, page, :, row] = _rotate(k, pos, s["freqs"], c["inter"]).to(dt)
    s["v"][0, page, :, row] = v


def _attend(s):
    """softmax(q . k / sqrt(D)) . v, a request and a part of its rows at a time."""
    c = s["case"]
    Hkv, G, D, W = c["Hkv"], c["H"] // c["Hkv"], c["D"], c["window"]
    for b in range(c["B"]):
        at, end, past = s["host_start"][b], s["host_start"][b + 1], s["host_lens"][b]
        if at == end:
            continue
        total = past + end - at
        page = s["table"][b, :-(-total // BLOCK)].long()
        k, v = (s[x][0, page].transpose(0, 1).reshape(Hkv, -1, D)[:, :total].float() for x in ("k", "v"))
        step = max(1, 300_000_000 // (Hkv * G * total))
        for r in range(at, end, step):
            q = s["q"][r:min(end, r + step)].float()
            n = q.shape[0]
            sc = q.view(n, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * n, D) @ k.transpose(1, 2) * D ** -0.5
            p = (past + r - at + torch.arange(n, device=q.device))[:, None]
            j = torch.arange(total, device=q.device)[None, :]
            seen = j <= p
            if W:
                seen &= j > p - W
            sc = sc.view(Hkv, G, n, total).masked_fill_(~seen, -torch.inf)
            w = sc.sub_(sc.amax(-1, keepdim=True)).exp_()
            o = (w.view(Hkv, G * n, total) @ v).view(Hkv, G, n, D) / w.sum(-1, keepdim=True)
            s["out"][r:r + n] = o.permute(2, 0, 1, 3).reshape(n, Hkv * G, D).to(s["out"].dtype)
            del sc, w


# --------------------------------------------------------------------- run

def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        return _run_own(s)
    if op == "rope":
        return _rope(s)
    if op == "append":
        _append(s)
        return {x: s[x] for x in ("q_out", "k", "v")}
    _attend(s)
    return s["out"]


def _run_own(s):
    import speculative_decode_verify_w4a16_gb300 as sv

    c = s["case"]
    if c["op"] == "rope":
        return sv.rope(s["rows"][:, :c["heads"]], s["positions"], s["freqs"], inverse=c["inverse"])
    cache = sv.KV16Cache(s["k"], s["v"])
    if c["op"] == "append":
        q, k, v = s["qkv"].split((c["H"], c["Hkv"], c["Hkv"]), 1)
        sv.kv16_append(cache, 0, k, v, s["table"], s["lens"], row_start=s["start"], rope=s["freqs"], q=q, q_out=s["q_out"])
        return {x: s[x] for x in ("q_out", "k", "v")}
    return sv.kv16_attention(s["q"], cache, 0, s["table"], s["lens"], row_start=s["start"], window=c["window"],
                             out=s["out"])


# -------------------------------------------------------------------- work

def work(case):
    c = case
    size = TYPES[c["type"]].itemsize
    if c["op"] == "rope":
        n = c["T"] * c["heads"]
        return {"bytes": 2 * n * c["D"] * size + 4 * c["T"], "flops": 3 * n * c["rot"]}
    lens, cnt = _lens(c, 0), _counts(c, 0)
    T, H, Hkv, D = int(cnt.sum()), c["H"], c["Hkv"], c["D"]
    if c["op"] == "append":
        return {"bytes": 2 * T * (H + 2 * Hkv) * D * size + 8 * T, "flops": 3 * T * (H + Hkv) * c["rot"]}
    keys = scores = 0
    for past, n in zip(lens.tolist(), cnt.tolist()):
        if n == 0:
            continue
        w = c["window"] or past + n
        first = max(0, past - w + 1)  # the first key that any row sees
        keys += past + n - first
        full = max(0, min(n, past + n - w))  # rows that see a whole window
        part = n - full
        scores += full * w + part * (past + 1) + part * (part - 1) // 2
    return {"bytes": (2 * keys * Hkv + 2 * T * H) * D * size, "flops": 4 * scores * H * D}


# ------------------------------------------------------------------- exact

def _turned(x, pos, c, inverse):
    """The rotation as a product of complex numbers, in float64."""
    f, factor = _frequencies(c, x.device)
    a = pos.double()[:, None, None] * f
    z = torch.polar(torch.full_like(a, factor), -a if inverse else a)
    x = x.double()
    rot, half = c["rot"], c["rot"] // 2
    pairs = x[..., :rot].unflatten(-1, (half, 2)) if c["inter"] else x[..., :rot].unflatten(-1, (2, half)).transpose(-1, -2)
    y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z)
    y = y.flatten(-2) if c["inter"] else y.transpose(-1, -2).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _exact_append(s, c):
    """Request by request, its positions counted up."""
    H, Hkv = c["H"], c["Hkv"]
    out = {x: s[x].double() for x in ("q_out", "k", "v")}
    table = s["table"].cpu()
    for b in range(c["B"]):
        at, end = s["host_start"][b], s["host_start"][b + 1]
        pos = torch.arange(s["host_lens"][b], s["host_lens"][b] + end - at)
        page, row = table[b][pos // BLOCK].long().cuda(), (pos % BLOCK).cuda()
        x = s["qkv"][at:end]
        out["q_out"][at:end] = _turned(x[:, :H], pos.cuda(), c, False)
        out["k"][0][page, :, row] = _turned(x[:, H:H + Hkv], pos.cuda(), c, False)
        out["v"][0][page, :, row] = x[:, H + Hkv:].double()
    return out


def _exact_attn(s, c):
    """Request by request and head by head in float64, some rows at a time, from the keys that they see."""
    G, D = c["H"] // c["Hkv"], c["D"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    table = s["table"].cpu()
    for b in range(c["B"]):
        at, end, past = s["host_start"][b], s["host_start"][b + 1], s["host_lens"][b]
        if at == end:
            continue
        page = table[b][:(past + end - at + BLOCK - 1) // BLOCK].long().cuda()
        for h in range(c["Hkv"]):
            k, v = (s[x][0, page, h].double().flatten(0, 1) for x in ("k", "v"))
            for r in range(at, end, 512):
                n = min(512, end - r)
                lo, hi = 0, past + r - at + n  # keys that any of these rows sees
                if c["window"]:
                    lo = max(0, past + r - at - c["window"] + 1)
                d = (past + r - at + torch.arange(n, device="cuda"))[:, None] - torch.arange(lo, hi, device="cuda")[None, :]
                hidden = d < 0 if not c["window"] else (d < 0) | (d >= c["window"])
                for g in range(G):
                    a = s["q"][r:r + n, h * G + g].double() @ k[lo:hi].T / math.sqrt(D)
                    out[r:r + n, h * G + g] = torch.softmax(a.masked_fill_(hidden, -torch.inf), 1) @ v[lo:hi]
    return out


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "rope":
        return _turned(s["rows"][:, :c["heads"]], s["positions"], c, c["inverse"])
    return _exact_append(s, c) if c["op"] == "append" else _exact_attn(s, c)
