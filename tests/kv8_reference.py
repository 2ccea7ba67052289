"""The paged 8-bit cache operators written plainly in 64 bits (test
infrastructure: request by request, row by row; shares no code with the
library)."""
import math

import numpy as np
import torch

BLOCK = 64
LARGEST = {torch.float8_e4m3fn: 448.0, torch.float8_e5m2: 57344.0}
SKIP = -(2 ** 31)


def chain(n):
    return np.arange(-1, n - 1, dtype=np.int32)


def random_tree(n, rng, depth=6):
    par, dep = np.full(n, -1, np.int32), np.zeros(n, int)
    for j in range(1, n):
        k = int(rng.integers(0, j))
        while dep[k] >= depth:
            k = par[k]
        par[j], dep[j] = k, dep[k] + 1
    return par


def root_path(parents, node):
    """Nodes on the root path, root first."""
    path = []
    while node >= 0:
        path.append(int(node))
        node = parents[node]
    return path[::-1]


def plan(lens, tails, table, ring, queue, rows, kept, release=None):
    """kept[b]: the source rows of request b, in order. Returns the tables
    after the step and the plan (all numpy int64)."""
    B, cap = len(lens), len(ring)
    table, ring = table.astype(np.int64).copy(), ring.astype(np.int64).copy()
    old_ring = ring.copy()
    head, count = int(queue[0]), int(queue[1])
    asked = taken = returned = 0
    new_lens, new_tails, start, src, slots = [], [], [0], [], []
    for b in range(B):
        n, rws = int(lens[b]), list(kept[b])
        if release is not None and release[b]:
            for j in range(n // BLOCK):
                ring[(head + count + returned) % cap] = table[b, j]
                returned += 1
            new_lens.append(0)
            new_tails.append(tails[b])
            start.append(start[-1])
            continue
        need = (n + len(rws)) // BLOCK - n // BLOCK
        asked += need
        if need and asked > count:
            rws, need = [], 0
        for j in range(need):
            table[b, n // BLOCK + j] = old_ring[(head + taken) % cap]
            taken += 1
        for i, r in enumerate(rws):
            pos = n + i
            src.append(r)
            slots.append(table[b, pos // BLOCK] * BLOCK + pos % BLOCK if pos // BLOCK < (n + len(rws)) // BLOCK
                         else -1 - pos % BLOCK)
        new_lens.append(n + len(rws))
        new_tails.append(tails[b] ^ 1 if need else tails[b])
        start.append(start[-1] + len(rws))
    pad = rows - len(src)
    return table, ring, {
        "new_lens": np.array(new_lens), "new_tails": np.array(new_tails), "new_start": np.array(start),
        "queue": np.array([(head + taken) % cap, count - taken + returned, asked - taken]),
        "src_rows": np.array(src + [-1] * pad), "slots": np.array(slots + [SKIP] * pad)}


def quantize(block, dtype):
    """One block [64, D] in bf16 -> (codes, scale): the smallest power of two,
    2^-100 at least, that brings the largest finite magnitude to the largest
    code or below."""
    x = block.double()
    mag = x.abs()[x.isfinite()]
    top = float(mag.max()) if mag.numel() else 0.0
    k = 0
    if top > 0.0:
        k = max(-100, math.frexp(top / LARGEST[dtype])[1] - 1)
        if math.ldexp(LARGEST[dtype], k) < top:
            k += 1
    scaled = (x / 2.0 ** k).clamp(-LARGEST[dtype], LARGEST[dtype])  # NaN stays NaN
    return scaled.float().to(dtype), 2.0 ** k


class Cache:
    """A cache built from whole histories: hist[b] = (keys, values) bf16 [Hkv, len, D] on the CPU."""

    def __init__(self, hist, dtype, rng, max_len, spare=3, stale=None):
        B = len(hist)
        Hkv, _, D = hist[0][0].shape
        self.lens = np.array([h[0].shape[1] for h in hist], np.int32)
        full = self.lens // BLOCK
        pages = int(full.sum()) + spare
        perm = rng.permutation(pages)
        self.table = np.full((B, max(1, max_len // BLOCK)), -1, np.int32)
        self.tails = (2 * rng.permutation(B) + rng.integers(0, 2, B)).astype(np.int32)
        fill = 1.0 if stale is None else stale
        self.codes = [torch.full((pages, Hkv, BLOCK, D), fill).to(dtype) for _ in range(2)]
        self.scales = [torch.ones(pages, Hkv) for _ in range(2)]
        self.tail = [torch.full((2 * B, Hkv, BLOCK, D), fill, dtype=torch.bfloat16) for _ in range(2)]
        self.values = []  # what the cache stands for, [Hkv, len, D] in float64
        at = 0
        for b in range(B):
            got = [[], []]
            for j in range(full[b]):
                page = int(perm[at])
                at += 1
                self.table[b, j] = page
                for c in range(2):
                    heads = []
                    for h in range(Hkv):
                        q, s = quantize(hist[b][c][h, j * BLOCK:(j + 1) * BLOCK], dtype)
                        self.codes[c][page, h], self.scales[c][page, h] = q, s
                        heads.append(q.double() * s)
                    got[c].append(torch.stack(heads))
            rest = int(self.lens[b]) % BLOCK
            for c in range(2):
                x = hist[b][c][:, full[b] * BLOCK:]
                self.tail[c][int(self.tails[b]), :, :rest] = x
                got[c].append(x.double())
            self.values.append([torch.cat(g, 1) for g in got])

    def to(self, sv, dev, layers=1, layer=0):
        """The library's KV8Cache (other layers hold zeros) and the table, lens and tails."""
        def put(x):
            raw = x.view(torch.uint8) if x.dtype.itemsize == 1 else x
            y = torch.zeros((layers,) + tuple(x.shape), dtype=raw.dtype)
            y[layer] = raw
            return y.to(dev).view(x.dtype)
        cache = sv.KV8Cache(put(self.codes[0]), put(self.codes[1]), put(self.scales[0]), put(self.scales[1]),
                            put(self.tail[0]), put(self.tail[1]))
        return cache, *(torch.from_numpy(a).to(dev) for a in (self.table, self.lens, self.tails))


def attention(values, q, k_new, v_new, parents, scale=None):
    """q [n, H, D], k_new, v_new [n, Hkv, D] of one request; values [Hkv, len,
    D] float64 pairs. Returns (out, weighted magnitudes) [n, H, D] float64."""
    n, H, D = q.shape
    Hkv = k_new.shape[1]
    scale = D ** -0.5 if scale is None else scale
    out, mag = torch.zeros(n, H, D, dtype=torch.float64), torch.zeros(n, H, D, dtype=torch.float64)
    for j in range(n):
        path = root_path(parents, j)
        for h in range(H):
            g = h // (H // Hkv)
            K = torch.cat([values[0][g], k_new[path, g].double()])
            V = torch.cat([values[1][g], v_new[path, g].double()])
            w = torch.softmax(K @ q[j, h].double() * scale, 0)
            out[j, h] = w @ V
            mag[j, h] = w @ V.abs()
    return out, mag
