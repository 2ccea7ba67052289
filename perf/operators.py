"""Plain forms and cases of the paged 8-bit cache operators and of the log-probability report.

Four operators of a verify step that keeps its keys and values in 8 bits:

  kv_block_plan       block tables, slot maps and the free list of a step, from the requests' lengths
  kv8_append          the step's kept keys and values into the cache, a scale for each 64-token block and head
  kv8_tree_attention  tree-masked verify attention over that cache
  token_logprobs      log probabilities of given tokens, entropy and the top alternatives of logit rows

`run` computes them with elementary torch operations, or (`own`) with the framework's entry points.
A request's tokens fill blocks of 64. A full block sits in a page in 8 bits, code * scale with one power-of-two
scale for the block's keys of a head and one for its values; the block being filled stays in bf16 in a tail page.
"""
import random

import numpy as np
import torch

own = False

BLOCK = 64
D = 128
FORMATS = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = {"e4m3": 9, "e5m2": 16}  # the largest code is 0.875 * 2^TOP
SKIP = -(2 ** 31)  # slot of a row past the kept ones


def listed():
    return [
        # the commit of a sequence-draft step: 16 requests, up to five kept rows each
        {"name": "plan_chain", "op": "plan", "mode": "draft", "B": 16, "n": 5, "tree": False, "lo": 1, "hi": 8191,
         "per": 0, "ended": 0},
        # a chunk of prompts for a full house, some requests ending
        {"name": "plan_prompts", "op": "plan", "mode": "ragged", "B": 1021, "n": 0, "tree": False, "lo": 0, "hi": 8191,
         "per": 63, "ended": 7},
        # one decoded token a request, one layer
        {"name": "append_one", "op": "append", "mode": "draft", "layers": 1, "B": 64, "n": 1, "tree": False, "Hkv": 8,
         "lo": 40, "hi": 4100, "per": 0, "fmt": "e5m2"},
        # the accepted rows of a sequence draft, every layer of the 80-layer stack at once
        {"name": "append_chain", "op": "append", "mode": "draft", "layers": 80, "B": 16, "n": 5, "tree": False,
         "Hkv": 8, "lo": 1, "hi": 8191, "per": 0, "fmt": "e4m3"},
        # prompts of different lengths, one layer
        {"name": "append_prompts", "op": "append", "mode": "ragged", "layers": 1, "B": 7, "n": 0, "tree": False,
         "Hkv": 8, "lo": 0, "hi": 130, "per": 4681, "fmt": "e4m3"},
        # a lone decoding request
        {"name": "attn_one", "op": "attn", "B": 1, "n": 1, "tree": False, "H": 64, "Hkv": 8, "lo": 1003, "hi": 1003,
         "fmt": "e4m3"},
        # a small tree draft, one query head for each key/value head
        {"name": "attn_mha", "op": "attn", "B": 3, "n": 17, "tree": True, "H": 16, "Hkv": 16, "lo": 65, "hi": 2100,
         "fmt": "e5m2"},
        # the sequence draft of the 80-layer stack's batch
        {"name": "attn_chain", "op": "attn", "B": 16, "n": 5, "tree": False, "H": 64, "Hkv": 8, "lo": 4096,
         "hi": 8191, "fmt": "e4m3"},
        # long contexts, one token each
        {"name": "attn_long", "op": "attn", "B": 4, "n": 1, "tree": False, "H": 64, "Hkv": 8, "lo": 120001,
         "hi": 131071, "fmt": "e4m3"},
        # 64-node trees
        {"name": "attn_tree", "op": "attn", "B": 16, "n": 64, "tree": True, "H": 64, "Hkv": 8, "lo": 2048, "hi": 4095,
         "fmt": "e4m3"},
        # what a decode step reports: 16 rows of fp32 logits
        {"name": "logprobs_step", "op": "logprobs", "R": 16, "V": 128256, "m": 1, "top": 5, "bits": 32},
        # every node of 16 trees, bf16 logits, two given tokens a row
        {"name": "logprobs_trees", "op": "logprobs", "R": 1024, "V": 128256, "m": 2, "top": 20, "bits": 16},
    ]


def _spread(rng, lo, hi):
    """An integer of lo .. hi, over its logarithm where that spans more than a factor of ten."""
    if hi > 10 * max(lo, 1):
        return int(round(np.exp(rng.uniform(np.log(max(lo, 1)), np.log(hi))))) if rng.random() > 0.03 else lo
    return rng.randint(lo, hi)


def draw(rng: random.Random):
    op = rng.choice(["plan", "append", "attn", "attn", "logprobs"])
    if op == "logprobs":
        V = rng.choice([128256, _spread(rng, 33, 160000)])
        return {"op": op, "R": max(1, min(_spread(rng, 1, 1024), 131_000_000 // V)), "V": V, "m": rng.randint(1, 4),
                "top": min(V, rng.choice([0, 1, 5, 20, 32])), "bits": rng.choice([16, 32])}
    if op == "plan":
        mode = rng.choice(["draft", "ragged"])
        return {"op": op, "mode": mode, "B": _spread(rng, 1, 1021), "n": rng.randint(1, 64) if mode == "draft" else 0,
                "tree": rng.random() < 0.5, "lo": 0, "hi": _spread(rng, 64, 8191),
                "per": _spread(rng, 1, 63) if mode == "ragged" else 0, "ended": rng.choice([0, 0, 5, 9])}
    if op == "append":
        mode = rng.choice(["draft", "ragged"])
        hkv = rng.choice([1, 2, 4, 8, 16])
        if mode == "draft":
            n, layers = rng.randint(1, 24), _spread(rng, 1, 80)
            most = max(1, 6400 * 8 // (layers * n * hkv))
            return {"op": op, "mode": mode, "layers": layers, "B": min(most, _spread(rng, 1, 64)), "n": n,
                    "tree": rng.random() < 0.5, "Hkv": hkv, "lo": 0, "hi": _spread(rng, 64, 8191), "per": 0,
                    "fmt": rng.choice(["e4m3", "e5m2"])}
        B = _spread(rng, 1, 16)
        return {"op": op, "mode": mode, "layers": 1, "B": B, "n": 0, "tree": False, "Hkv": hkv, "lo": 0,
                "hi": _spread(rng, 64, 8191), "per": _spread(rng, 1, 32767 * 8 // (B * max(hkv, 8))),
                "fmt": rng.choice(["e4m3", "e5m2"])}
    hkv = rng.choice([1, 2, 4, 8, 16])
    g = rng.choice([1, 2, 3, 4, 5, 8, 16])
    n = rng.choice([1, rng.randint(2, 9), rng.randint(10, 64)])
    B = _spread(rng, 1, 70)
    cap = 4_000_000 // (B * hkv)  # no more keys than the long contexts hold
    cap = min(cap, 16 * 8 * 512 * 3000 // (B * hkv * n * g))  # no more scores than the trees compute
    hi = _spread(rng, 1, max(2, min(cap, 131071)))
    return {"op": "attn", "B": B, "n": n, "tree": n > 1 and rng.random() < 0.6, "H": hkv * g, "Hkv": hkv,
            "lo": rng.choice([0, hi // 2, hi]), "hi": hi, "fmt": rng.choice(["e4m3", "e5m2"])}


# ------------------------------------------------------------------ inputs

def _lens(c, seed):
    """Lengths from lo to hi, the same ones for every seed in another order."""
    B = c["B"]
    step = np.arange(B) * 0.6180339887 % 1.0
    v = np.floor(c["lo"] + (c["hi"] - c["lo"] + 1) * step).astype(np.int32)
    v = np.minimum(v, c["hi"])
    return np.roll(v, seed % B) if B > 1 else v


def _counts(c):
    """Rows a ragged case brings for each request, 0 .. 2 * per and `per` on average."""
    return np.round((np.arange(1, c["B"] + 1) * 0.7548776662 % 1.0) * 2 * c["per"]).astype(np.int32)


def _parents(rng, B, n):
    p = np.full((B, n), -1, np.int32)
    depth = np.zeros((B, n), np.int32)
    for b in range(B):
        for j in range(1, n):
            k = int(rng.integers(0, j))
            while depth[b, k] >= 6:
                k = int(p[b, k])
            p[b, j], depth[b, j] = k, depth[b, k] + 1
    return p


def _step_inputs(c, seed, rng):
    """What the accept step and the scheduler leave for a plan: lengths, tables, free pages and rows."""
    B, n = c["B"], c["n"]
    lens = _lens(c, seed)
    s = {"mode": c["mode"], "n": n, "parents": None}
    if c["mode"] == "draft":
        rows = B * n
        node = (np.arange(B) * 7 + seed) % n
        if c["tree"]:
            s["parents"] = _dev(_parents(rng, B, n))
        s["node"] = _dev(node.astype(np.int32))
        grow = n
    else:
        cnt = _counts(c)
        s["row_start"] = _dev(np.concatenate([[0], np.cumsum(cnt)]).astype(np.int32))
        rows = int(cnt.sum())
        grow = int(cnt.max())
    full = lens // BLOCK
    maxb = int((c["hi"] + grow) // BLOCK + 1)
    if c["op"] == "append":  # the cache holds only the pages that this step fills
        used = np.zeros(B, np.int64)
    else:
        used = full.astype(np.int64)
    pages = int(used.sum()) + rows // BLOCK + B + 1
    perm = rng.permutation(pages).astype(np.int32)
    table = np.full((B, maxb), -1, np.int32)
    at = np.concatenate([[0], np.cumsum(used)])
    cols = np.arange(maxb)[None, :]
    mask = cols < used[:, None]
    table[mask] = perm[(at[:-1, None] + cols)[mask]]
    ring = np.zeros(pages, np.int32)
    free = pages - int(at[-1])
    head = int(rng.integers(0, pages))
    ring[(head + np.arange(free)) % pages] = perm[int(at[-1]):]
    s["release"] = None
    if c.get("ended"):
        s["release"] = _dev((np.arange(B) % c["ended"] == c["ended"] - 1).astype(np.int32))
    s.update(lens=_dev(lens), tails=_dev((2 * np.arange(B) + (lens // BLOCK) % 2).astype(np.int32)), table=_dev(table),
             ring=_dev(ring), queue=_dev(np.array([head, free, 0], np.int32)), rows=rows, pages=pages)
    s["plan"] = {"new_lens": _zeros(B), "new_tails": _zeros(B), "new_start": _zeros(B + 1), "queue": _zeros(3),
                 "src_rows": _zeros(max(rows, 1)), "slots": _zeros(max(rows, 1))}
    return s


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _zeros(n):
    return torch.zeros(n, dtype=torch.int32, device="cuda")


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.bfloat16)


def prepare(case, seed):
    c = case
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 1000003 + 17)
    if c["op"] == "logprobs":
        x = torch.randn(c["R"], c["V"], generator=gen, device="cuda") * 3.0
        ids = torch.randint(0, c["V"], (c["R"], c["m"]), generator=gen, device="cuda", dtype=torch.int32)
        return {"case": c, "logits": x if c["bits"] == 32 else x.bfloat16(), "ids": ids}
    if c["op"] == "plan":
        return {"case": c, **_step_inputs(c, seed, rng)}
    if c["op"] == "append":
        s = {"case": c, **_step_inputs(c, seed, rng)}
        L, H = c["layers"], c["Hkv"]
        s["k_new"], s["v_new"] = (_randn(gen, L, max(s["rows"], 1), H, D) for _ in range(2))
        s["k_new"] *= torch.exp(torch.randn(D, generator=gen, device="cuda")).bfloat16()  # channels of unlike size
        s["k_tail"], s["v_tail"] = (_randn(gen, L, 2 * c["B"], H, BLOCK, D) for _ in range(2))
        for name in ("k", "v"):
            s[name] = torch.zeros(L, s["pages"], H, BLOCK, D, dtype=torch.uint8, device="cuda").view(FORMATS[c["fmt"]])
            s[name + "_scale"] = torch.ones(L, s["pages"], H, device="cuda")
        if s["rows"]:  # the plan that the step made
            _plan(s)
        return s
    # attention: a cache in use, its pages in any order
    B, n, H, Hkv = c["B"], c["n"], c["H"], c["Hkv"]
    lens = _lens(c, seed)
    full = lens // BLOCK
    pages = int(full.sum()) + 3
    table = np.full((B, c["hi"] // BLOCK + 1), -1, np.int32)
    cols = np.arange(table.shape[1])[None, :]
    mask = cols < full[:, None]
    table[mask] = rng.permutation(pages).astype(np.int32)[:int(full.sum())]
    s = {"case": c, "lens": _dev(lens), "table": _dev(table), "max_len": c["hi"],
         "tails": _dev((2 * rng.permutation(B) + full % 2).astype(np.int32)), "parents": None}
    if c["tree"]:
        s["parents"] = _dev(_parents(rng, B, n))
    chan = torch.exp(0.7 * torch.randn(Hkv, 1, D, generator=gen, device="cuda")).bfloat16()
    for name in ("k", "v"):
        x = _randn(gen, pages, Hkv, BLOCK, D)
        if name == "k":
            x *= chan
        scale = _scale_of(x.abs().amax((2, 3)).float(), c["fmt"])
        s[name] = (x / scale.bfloat16()[:, :, None, None]).to(FORMATS[c["fmt"]])
        s[name + "_scale"] = scale
        del x
    s["k_tail"], s["v_tail"] = (_randn(gen, 2 * B, Hkv, BLOCK, D) for _ in range(2))
    s["k_tail"] *= chan
    # the rotated rows of the fused projection: q, k and v side by side
    s["qkv"] = _randn(gen, B, n, H + 2 * Hkv, D)
    return s


# ------------------------------------------------------------- plain forms

def _scale_of(amax, fmt):
    """The smallest power of two, 2^-100 at least, that brings amax (fp32) to the largest code or below; 1 for zero."""
    m, e = torch.frexp(amax)
    k = torch.where(m <= 0.875, e, e + 1) - TOP[fmt]
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), k.clamp(min=-100)), torch.ones_like(amax))


def _seen(parents, B, n, device):
    """[B, n, n]: node i sees node j (itself and its ancestors)."""
    if parents is None:
        return torch.ones(n, n, dtype=torch.bool, device=device).tril()[None].expand(B, n, n)
    up = (parents[:, :, None] == torch.arange(n, device=device)).double() + torch.eye(n, device=device).double()
    return torch.linalg.matrix_power(up, 64) > 0


def _plan(s):
    lens, table, ring = s["lens"].long(), s["table"], s["ring"]
    B, maxb, cap, rows, dev = lens.numel(), table.shape[1], ring.numel(), s["rows"], lens.device
    head, count = s["queue"][0].long(), s["queue"][1].long()
    ended = torch.zeros(B, dtype=torch.bool, device=dev) if s["release"] is None else s["release"] != 0
    if s["mode"] == "draft":
        n = s["n"]
        path = _seen(s["parents"], B, n, dev)[torch.arange(B, device=dev), s["node"].long()]
        order = torch.sort((~path).to(torch.int8), dim=1, stable=True).indices
        cnt = path.sum(1)
    else:
        first = s["row_start"][:-1].long()
        cnt = s["row_start"].long().diff()
    cnt = torch.where(ended, 0, cnt)
    need = (lens + cnt) // BLOCK - lens // BLOCK
    granted = (need == 0) | (need.cumsum(0) <= count)
    cnt, take = torch.where(granted, cnt, 0), torch.where(granted, need, 0)
    after = lens + cnt
    taken = take.cumsum(0)
    cols = torch.arange(maxb, device=dev)[None, :]
    # pages for the blocks that this step fills, in order from the ring's head
    fills = (cols >= (lens // BLOCK)[:, None]) & (cols < (after // BLOCK)[:, None])
    j = (taken - take)[:, None] + cols - (lens // BLOCK)[:, None]
    new_table = torch.where(fills, ring[(head + j) % cap], table)
    # the pages of the requests that ended, behind the free ones
    back = torch.where(ended, lens // BLOCK, 0)
    gone = ended[:, None] & (cols < back[:, None])
    at = (head + count + (back.cumsum(0) - back)[:, None] + cols) % cap
    longer = torch.cat([ring, ring.new_zeros(1)])
    longer.scatter_(0, torch.where(gone, at, cap).flatten(), table.flatten())
    start = torch.cat([cnt.new_zeros(1), cnt.cumsum(0)])
    i = torch.arange(max(rows, 1), device=dev)
    b = torch.searchsorted(start[1:], i, right=True).clamp(max=B - 1)
    off = (i - start[b]).clamp(min=0)
    if s["mode"] == "draft":
        src = b * n + order[b, off.clamp(max=n - 1)]
    else:
        src = first[b] + off
    pos = lens[b] + off
    page = new_table[b, (pos // BLOCK).clamp(max=maxb - 1)].long()
    slot = torch.where(pos // BLOCK < after[b] // BLOCK, page * BLOCK + pos % BLOCK, -1 - pos % BLOCK)
    kept = i < start[B]
    p = s["plan"]
    p["new_lens"].copy_(torch.where(ended, 0, after))
    p["new_tails"].copy_(torch.where(take > 0, s["tails"] ^ 1, s["tails"]))
    p["new_start"].copy_(start)
    p["src_rows"].copy_(torch.where(kept, src, -1))
    p["slots"].copy_(torch.where(kept, slot, SKIP))
    p["queue"].copy_(torch.stack([(head + taken[-1]) % cap, count - taken[-1] + back.sum(), need.sum() - taken[-1]]))
    table.copy_(new_table)
    ring.copy_(longer[:cap])


def _blocks(s):
    """The pieces of blocks that an append touches: request, first position, source rows, which rows are set."""
    p, c, dev = s["plan"], s["case"], s["lens"].device
    B, rows = c["B"], p["src_rows"].numel()
    start = p["new_start"].long()
    first = p["slots"][start[:-1].clamp(max=rows - 1)].long()
    t = torch.where(first >= 0, first % BLOCK, -1 - first)  # rows of the block already there
    cnt = start.diff()
    pieces = torch.where(cnt > 0, (t + cnt + BLOCK - 1) // BLOCK, 0)
    upto = pieces.cumsum(0)
    i = torch.arange(rows // BLOCK + 2 * B, device=dev)
    b = torch.searchsorted(upto, i, right=True).clamp(max=B - 1)
    k = i - (upto - pieces)[b]
    off = k[:, None] * BLOCK + torch.arange(BLOCK, device=dev) - t[b][:, None]  # kept rows' numbers
    there = (i < upto[-1])[:, None] & (off < cnt[b][:, None])
    at = (start[b][:, None] + off).clamp(0, rows - 1)
    return b, k, t, off, there, at


def _append(s):
    p, c = s["plan"], s["case"]
    b, k, t, off, there, at = _blocks(s)
    src, slot = p["src_rows"][at].long().clamp(min=0), p["slots"][at].long()
    old = there & (off < 0)
    full = there.all(1) & (slot[:, -1] >= 0)
    page = slot[:, -1] // BLOCK
    row = torch.arange(BLOCK, device=b.device)[None, :].expand_as(off)
    live = torch.nonzero(full)[:, 0]
    tl = torch.nonzero(there & ~full[:, None] & (off >= 0))
    for name in ("k", "v"):
        new, tail = s[name + "_new"], s[name + "_tail"]
        x = new[:, src[live]]  # [layers, pieces, 64, heads, D]
        x = torch.where(old[live][None, :, :, None, None], tail[:, s["tails"].long()[b[live]]].transpose(2, 3), x)
        x = x.transpose(2, 3).float()
        scale = _scale_of(torch.where(x.isfinite(), x.abs(), 0).amax((3, 4)), c["fmt"])
        most = 0.875 * 2.0 ** TOP[c["fmt"]]
        codes = (x / scale[..., None, None]).clamp(-most, most).to(FORMATS[c["fmt"]])
        s[name].view(torch.uint8)[:, page[live]] = codes.view(torch.uint8)
        s[name + "_scale"][:, page[live]] = scale
        tb, tr = tl[:, 0], tl[:, 1]
        tail[:, p["new_tails"].long()[b[tb]], :, row[tb, tr]] = new[:, src[tb, tr]].transpose(0, 1)


def _split(s):
    H, Hkv = s["case"]["H"], s["case"]["Hkv"]
    return s["qkv"][:, :, :H], s["qkv"][:, :, H:H + Hkv], s["qkv"][:, :, H + Hkv:]


def _attend(s, dt):
    """softmax(q . k / sqrt(D)) . v over the cached blocks, the tail rows and the tree's own rows."""
    c = s["case"]
    B, n, H, Hkv = c["B"], c["n"], c["H"], c["Hkv"]
    q, k_new, v_new = _split(s)
    dev = q.device
    lens = s["lens"].long()
    page = s["table"].clamp(min=0).long()
    nb = page.shape[1]
    pos = torch.arange(nb * BLOCK, device=dev)[None, :]
    in_tail = torch.arange(BLOCK, device=dev)[None, :] < (lens % BLOCK)[:, None]
    seen = torch.cat([(pos < (lens // BLOCK * BLOCK)[:, None])[:, None].expand(B, n, nb * BLOCK),
                      in_tail[:, None].expand(B, n, BLOCK), _seen(s["parents"], B, n, dev)], 2)

    def rows(name, new):
        x = s[name].view(torch.uint8)[page].view(s[name].dtype).to(dt) * s[name + "_scale"][page][..., None, None].to(dt)
        x = x.transpose(1, 2).reshape(B, Hkv, nb * BLOCK, D)
        return torch.cat([x, s[name + "_tail"][s["tails"].long()].to(dt), new.transpose(1, 2).to(dt)], 2)

    qg = q.to(dt).view(B, n, Hkv, H // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    sc = (qg @ rows("k", k_new).transpose(2, 3)) * D ** -0.5
    sc = sc.view(B, Hkv, n, H // Hkv, -1).masked_fill(~seen[:, None, :, None], -torch.inf)
    w = torch.exp(sc - sc.amax(-1, keepdim=True))
    v = rows("v", v_new)
    o = (w.view(B, Hkv, n * (H // Hkv), -1) @ v).view(B, Hkv, n, H // Hkv, D) / w.sum(-1, keepdim=True)
    return o.permute(0, 2, 1, 3, 4).reshape(B, n, H, D)


def _logprobs(s):
    c, x = s["case"], s["logits"].float()
    m = x.amax(1, keepdim=True)
    z = x - m
    lse = torch.exp(z).sum(1, keepdim=True).log()
    lp = z - lse
    ent = -(torch.exp(lp) * lp).sum(1)
    bits = (x + 0.0).view(torch.int32)
    key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() * 2 ** 32 + (c["V"] - 1 - torch.arange(c["V"], device=x.device))
    top = c["V"] - 1 - (torch.topk(key, c["top"], dim=1).values & 0xFFFFFFFF)
    return {"logp": lp.gather(1, s["ids"].long()), "entropy": ent, "top_ids": top.int(), "top_logp": lp.gather(1, top)}


# --------------------------------------------------------------------- run

def _plan_out(s):
    return {"table": s["table"], "ring": s["ring"], **s["plan"]}


def _append_out(s):
    return {x: s[x] for x in ("k", "v", "k_scale", "v_scale", "k_tail", "v_tail")}


def run(state):
    s = state
    c = s["case"]
    if own:
        return _run_own(s, c)
    if c["op"] == "plan":
        _plan(s)
        return _plan_out(s)
    if c["op"] == "append":
        if s["rows"]:
            _append(s)
        return _append_out(s)
    if c["op"] == "attn":
        return _attend(s, torch.float32).bfloat16()
    return _logprobs(s)


def _run_own(s, c):
    import speculative_decode_verify_w4a16_gb300 as sv

    if c["op"] == "plan":
        plan = sv.BlockPlan(**s["plan"])
        if c["mode"] == "draft":
            sv.kv_block_plan(s["lens"], s["tails"], s["table"], s["ring"], s["queue"], accepted_node=s["node"], n=c["n"],
                             tree_parents=s["parents"], release=s["release"], plan=plan)
        else:
            sv.kv_block_plan(s["lens"], s["tails"], s["table"], s["ring"], s["queue"], row_start=s["row_start"],
                             rows=s["rows"], release=s["release"], plan=plan)
        return _plan_out(s)
    if c["op"] == "append":
        cache = sv.KV8Cache(**_append_out(s))
        if s["rows"]:
            sv.kv8_append(cache, s["k_new"], s["v_new"], s["tails"], sv.BlockPlan(**s["plan"]))
        return _append_out(s)
    if c["op"] == "attn":
        cache = sv.KV8Cache(*(s[x][None] for x in ("k", "v", "k_scale", "v_scale", "k_tail", "v_tail")))
        q, k_new, v_new = _split(s)
        return sv.kv8_tree_attention(q, k_new, v_new, cache, 0, s["table"], s["lens"], s["tails"],
                                     tree_parents=s["parents"], max_len=s["max_len"])
    r = sv.token_logprobs(s["logits"], s["ids"], top=c["top"])
    return {"logp": r.logp, "entropy": r.entropy, "top_ids": r.top_ids, "top_logp": r.top_logp}


# -------------------------------------------------------------------- work

def work(case):
    c = case
    if c["op"] == "logprobs":
        n = c["R"] * c["V"]
        return {"bytes": n * c["bits"] // 8 + c["R"] * (8 * c["m"] + 4 + 8 * c["top"]), "flops": 6 * n}
    B = c["B"]
    lens = _lens(c, 0).astype(np.int64)
    if c["op"] == "attn":
        H, Hkv, n = c["H"], c["Hkv"], c["n"]
        keys = int(lens.sum()) + B * n
        data = int((lens // BLOCK).sum()) * Hkv * 2 * (BLOCK * D + 4) + int((lens % BLOCK).sum() + B * n) * Hkv * D * 4
        return {"bytes": data + 2 * B * n * H * D * 2 + int((lens // BLOCK).sum()) * 4, "flops": 4 * keys * n * H * D}
    cnt = _counts(c).astype(np.int64) if c["mode"] == "ragged" else (np.arange(B) * 7) % c["n"] // (3 if c["tree"] else 1) + 1
    rows, pages = int(cnt.sum()), int(((lens + cnt) // BLOCK - lens // BLOCK).sum())
    if c["op"] == "plan":
        total = rows if c["mode"] == "ragged" else B * c["n"]
        return {"bytes": 4 * (7 * B + 2 * total + 2 * pages) + (4 * total if c["tree"] else 0), "flops": 8 * (total + B)}
    heads = c["layers"] * c["Hkv"]
    fills = (lens + cnt) // BLOCK > lens // BLOCK
    kept = int(np.where(fills, (lens + cnt) % BLOCK, cnt).sum())  # rows that go to a tail
    old = int(np.where(fills, lens % BLOCK, 0).sum())  # tail rows that a page takes
    moved = heads * 2 * (2 * D * (rows + old + kept) + pages * (BLOCK * D + 4)) + 8 * rows
    return {"bytes": moved, "flops": 4 * heads * 2 * pages * BLOCK * D + rows}


# ------------------------------------------------------------------- exact

def _nearest(x, fmt):
    """x rounded to the nearest value of the 8-bit type, ties to even, in float64."""
    bits, low = (3, -6) if fmt == "e4m3" else (2, -14)  # fraction bits, exponent of the smallest normal value
    e = (torch.frexp(x).exponent - 1).clamp(min=low) - bits
    return torch.ldexp(torch.round(torch.ldexp(x, -e)), e)


def _exact_append(s, c):
    """Block by block in float64, the stored values where nothing is written."""
    out = {}
    p = {x: s["plan"][x].cpu().numpy() for x in ("new_start", "src_rows", "slots", "new_tails")}
    tails = s["tails"].cpu().numpy()
    for name in ("k", "v"):
        codes, scales = s[name].double(), s[name + "_scale"].double()
        tail = s[name + "_tail"].double()
        was = tail.clone()
        new = s[name + "_new"].double()
        for b in range(c["B"]):
            i, end = int(p["new_start"][b]), int(p["new_start"][b + 1])
            while i < end:
                sl = int(p["slots"][i])
                r = sl % BLOCK if sl >= 0 else -1 - sl
                take = min(BLOCK - r, end - i)
                src = torch.from_numpy(p["src_rows"][i:i + take].astype(np.int64)).cuda()
                x = new[:, src].transpose(1, 2)
                if sl >= 0:
                    x = torch.cat([was[:, int(tails[b]), :, :r], x], 2)
                    top = x.abs().amax((2, 3)) / (0.875 * 2.0 ** TOP[c["fmt"]])
                    scale = torch.exp2(torch.round(torch.log2(top)))  # then to the nearest power not below
                    scale = torch.where(scale < top, 2 * scale, scale)
                    scale = torch.where(top > 0, scale.clamp(min=2.0 ** -100), torch.ones_like(scale))
                    codes[:, sl // BLOCK] = _nearest(x / scale[:, :, None, None], c["fmt"])
                    scales[:, sl // BLOCK] = scale
                else:
                    tail[:, int(p["new_tails"][b]), :, r:r + take] = x
                i += take
        out[name], out[name + "_scale"], out[name + "_tail"] = codes, scales, tail
    return out


def _exact_attn(s, c):
    """Request by request and head by head in float64, each query's keys picked one by one from its own mask."""
    B, n, H, Hkv = c["B"], c["n"], c["H"], c["Hkv"]
    q, k_new, v_new = (x.double() for x in _split(s))
    lens, table = s["lens"].cpu().numpy(), s["table"].cpu().numpy()
    parents = None if s["parents"] is None else s["parents"].cpu().numpy()
    tails = s["tails"].cpu().numpy()
    out = torch.empty(B, n, H, D, dtype=torch.float64, device=q.device)
    for b in range(B):
        full, rest = divmod(int(lens[b]), BLOCK)
        page = torch.from_numpy(table[b, :full].astype(np.int64)).to(q.device)
        mask = torch.zeros(n, n, dtype=torch.bool)
        for j in range(n):
            up = j
            while up >= 0:
                mask[j, up] = True
                up = up - 1 if parents is None else int(parents[b, up])
        mask = mask.to(q.device)
        for h in range(Hkv):
            kv = []
            for name, new in (("k", k_new), ("v", v_new)):
                x = s[name].view(torch.uint8)[page, h].view(s[name].dtype).double()
                x = (x * s[name + "_scale"][page, h].double()[:, None, None]).reshape(-1, D)
                kv.append(torch.cat([x, s[name + "_tail"][int(tails[b]), h, :rest].double(), new[b, :, h]]))
            for g in range(H // Hkv):
                a = q[b, :, h * (H // Hkv) + g] @ kv[0].T / D ** 0.5
                a[:, full * BLOCK + rest:] = torch.where(mask, a[:, full * BLOCK + rest:], -torch.inf)
                out[b, :, h * (H // Hkv) + g] = torch.softmax(a, 1) @ kv[1]
    return out


def exact(case, seed):
    c = case
    if c["op"] == "plan":
        return None  # whole numbers throughout
    s = prepare(c, seed)
    if c["op"] == "append":
        return _exact_append(s, c)
    if c["op"] == "attn":
        return _exact_attn(s, c)
    logp, ent, top = [], [], []
    ids = s["ids"].long()
    for r in range(c["R"]):
        x = s["logits"][r].double()
        lp = x - torch.logsumexp(x, 0)
        logp.append(lp[ids[r]])
        ent.append(-torch.special.xlogy(lp.exp(), lp.exp()).sum())
        top.append(torch.sort(lp, descending=True).values[:c["top"]])
    return {"logp": torch.stack(logp), "entropy": torch.stack(ent), "top_ids": None, "top_logp": torch.stack(top)}
