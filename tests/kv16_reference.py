"""Plain 64-bit implementations of rotary positions, the paged 16-bit cache's
append and its attention, for the tests to compare with."""
from fractions import Fraction

import numpy as np
import torch

PI = Fraction(314159265358979323846264338327950288419716939937511, 10 ** 50)
BLOCK = 64
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def cos_sin(positions, angles):
    """cos, sin float64 [T, pairs] of positions * angles, the whole turns taken
    off exactly."""
    turns = [Fraction(a) / (2 * PI) for a in angles]
    a = [[float((int(p) * t) % 1 * 2 * PI) for t in turns] for p in positions]
    a = torch.tensor(a, dtype=torch.float64).view(len(positions), len(turns))
    return a.cos(), a.sin()


def rotate(x, cos, sin, interleaved, factor=1.0, inverse=False):
    """x [T, heads, D] -> (float64 result, the sum of the magnitudes that went into each element)."""
    x = x.double()
    rot = 2 * cos.shape[1]
    c, s = (y[:, None].to(x.device) * factor for y in (cos, sin))
    if inverse:
        s = -s
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    y, mag = x.clone(), torch.zeros_like(x)
    u, v = x[..., first], x[..., second]
    y[..., first], y[..., second] = u * c - v * s, v * c + u * s
    mag[..., first] = mag[..., second] = (u.abs() + v.abs()) * factor
    return y, mag


def rotation_bound(y, mag, dtype):
    """Half a step of the type, and in fp32: the sine's and the cosine's errors
    (the angle's: a rounding of at most pi / 4 and 2^-32 turns, 4.8e-8; the
    function's ulp, 6e-8; the factor's rounding, 6e-8) and the products' and the
    sum's roundings (1.2e-7), all times the magnitudes. fp16 also rounds to its
    smallest step, 2^-24."""
    low = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}[dtype]
    return 1.001 * HALF_STEP[dtype] * y.abs() + 3e-7 * mag + low


def paged(rng, lens, counts, spare=2):
    """(block table int32 [B, max_blocks], pages): the pages of each request anywhere."""
    blocks = [-(-(a + n) // BLOCK) for a, n in zip(lens, counts)]
    pages = sum(blocks) + spare
    perm = rng.permutation(pages)
    table = np.full((len(lens), max(max(blocks), 1)), -1, np.int32)
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = perm[at:at + n]
        at += n
    return torch.from_numpy(table), pages


def rows_of(table, b, cache, first, last):
    """Positions first .. last - 1 of request b: [Hkv, n, D] of a layer's cache [pages, Hkv, 64, D]."""
    pos = torch.arange(first, last)
    page = table[b, pos // BLOCK].long().to(cache.device)
    return cache[page, :, (pos % BLOCK).to(cache.device)].transpose(0, 1)


def attention(q, k, v, past, window=0, scale=None):
    """One request: q [n, H, D] at positions past .., k, v [Hkv, past + n, D];
    (out float64 [n, H, D], the weighted sum of the values' magnitudes)."""
    n, H, D = q.shape
    Hkv = k.shape[0]
    scale = D ** -0.5 if scale is None else scale
    p = past + torch.arange(n, device=q.device)[:, None]
    j = torch.arange(past + n, device=q.device)[None, :]
    seen = j <= p
    if window:
        seen &= j > p - window
    plain = bool(k.isfinite().all() and v.isfinite().all())
    out = torch.empty(n, H, D, dtype=torch.float64, device=q.device)
    mag = torch.empty_like(out)
    for h in range(H):
        qh, kh, vh = q[:, h].double(), k[h * Hkv // H].double(), v[h * Hkv // H].double()
        if plain:
            w = torch.softmax((qh @ kh.T * scale).masked_fill_(~seen, -torch.inf), 1)
            out[:, h], mag[:, h] = w @ vh, w @ vh.abs()
            continue
        for i in range(n):  # from what the row sees alone
            w = torch.softmax((kh[seen[i]] @ qh[i]) * scale, 0)
            out[i, h], mag[i, h] = w @ vh[seen[i]], w @ vh[seen[i]].abs()
    return out, mag


def attention_bound(out, mag, v, dtype):
    """The weights' rounding (half a step each, so that of the weighted
    magnitudes) and the result's; 5 percent and 1e-6 of the largest value for
    what is done in fp32."""
    return 1.05 * HALF_STEP[dtype] * (mag + out.abs()) + 1e-6 * float(v.double().abs().nan_to_num(0, 0, 0).max())
