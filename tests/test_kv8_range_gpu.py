"""The 8-bit attention's number range: where a part of the work holds a
request's bf16 rows and many 8-bit tiles, so that one softmax reference serves
both.

Softmax output scales with the values. Among the cached keys a row's largest
score is 16 bits at most above those that count here, so their weights stay in
fp16's normal range (2^-14 and above, the largest being 2^7 when the reference is
set), and the bound of test_kv8_gpu holds as it is derived there, whatever the
size of the values and however far above the row's own keys are."""
import numpy as np
import pytest
import torch

import kv8_reference as ref
import speculative_decode_verify_w4a16_gb300 as sv
from helpers import dev
from test_kv8_gpu import E4M3, E5M2

pytestmark = pytest.mark.gpu
D, H, HEADS, L = 128, 160, 8, 1290  # 160 heads: the keys and values of 8 over and over, each with queries of its own


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decode_verify_w4a16_gb300 import build
    build.build()


def _parts():
    """The parts (first tile, end) that the kernel's CTAs take: the tiles of all
    heads end to end, one run of them an SM."""
    sms = torch.cuda.get_device_properties(dev()).multi_processor_count
    tiles = 1 + (L // 64 + 1) // 2
    T = tiles * H
    assert tiles <= 16 and T >= 4 * sms  # (units of more tiles, and few tiles, are cut otherwise)
    edges = np.cumsum([0] + [T // sms + (r < T % sms) for r in range(sms)])
    out = []
    for h in range(H):
        at = h * tiles
        cuts = [at, *(e for e in edges if at < e < at + tiles), at + tiles]
        out += [(int(a - at), int(b - at)) for a, b in zip(cuts, cuts[1:])]
    return out


def _case(seed, n, above, mean=1.0):
    """One request of L tokens, one query head a head: keys of small scores,
    values with a mean, and own keys `above` bits over the rest."""
    rng = np.random.default_rng(seed)
    k = torch.from_numpy(0.3 * rng.standard_normal((HEADS, L, D))).bfloat16()
    v = torch.from_numpy(rng.standard_normal((HEADS, L, D)) + mean).bfloat16()
    q = torch.from_numpy(rng.standard_normal((1, n, H, D))).bfloat16()
    size = q.double().square().sum(-1, keepdim=True) * D ** -0.5 * np.log2(np.e)
    own_k = (q.double() * (above / size)).bfloat16()
    own_v = torch.from_numpy(rng.standard_normal((1, n, H, D)) + mean).bfloat16()
    return rng, k, v, q, own_k, own_v


def _cache(k, v, dtype, rng):
    cache = ref.Cache([(k, v)], dtype, rng, L)
    for name in ("codes", "scales", "tail"):  # [pages, HEADS, ..] -> [pages, H, ..]
        setattr(cache, name, [x.repeat_interleave(H // HEADS, 1) if x.dtype.itemsize > 1 else
                              x.view(torch.uint8).repeat_interleave(H // HEADS, 1).view(dtype)
                              for x in getattr(cache, name)])
    cache.values = [[x.repeat_interleave(H // HEADS, 0) for x in cache.values[0]]]
    return cache


def _attend(cache, q, k, v):
    c, table, lens, tails = cache.to(sv, dev())
    out = sv.kv8_tree_attention(q.to(dev()), k.to(dev()), v.to(dev()), c, 0, table, lens, tails,
                                max_len=int(cache.lens.max()))
    torch.cuda.synchronize()
    assert sv.check_device_status() == 0
    return out.cpu().double()


def _compare(cache, q, k, v, what):
    """Against the definition in 64 bits, all heads at once; test_kv8_gpu's bound."""
    got = _attend(cache, q, k, v)[0]
    n = q.shape[1]
    K, V = (torch.cat([c, x[0].double().transpose(0, 1)], 1) for c, x in zip(cache.values[0], (k, v)))
    s = torch.einsum("nhd,hld->nhl", q[0].double(), K) * D ** -0.5
    s.masked_fill_(torch.arange(L + n)[None, None] > L + torch.arange(n)[:, None, None], -torch.inf)
    w = torch.softmax(s, -1)
    want, mag = (torch.einsum("nhl,hld->nhd", w, x) for x in (V, V.abs()))
    bound = 1.05 * 2.0 ** -8 * (mag + want.abs()) + 1e-7 * float(V.abs().max())
    worst = float(((got - want).abs() / bound).nan_to_num(nan=torch.inf).max())
    print(f"{what}: max |err| / bound = {worst:.3f}")
    assert worst <= 1.0, what


def test_parts_hold_the_bf16_rows_and_8_bit_tiles():
    assert sum(lo == 0 and hi >= 4 for lo, hi in _parts()) >= 16


@pytest.mark.parametrize("dtype", [E4M3, E5M2])
@pytest.mark.parametrize("above", [0, 10, 16])
def test_the_output_scales_with_the_values(dtype, above):
    rng, k, v, q, own_k, own_v = _case(20 + above, 2, above)
    cache = _cache(k, v, dtype, rng)
    for bits in (0, 7, 14, 20, 40):
        small = 2.0 ** -bits
        for x in (cache.scales[1], cache.tail[1], cache.values[0][1]):
            x *= small  # powers of two: the codes stay as they are
        _compare(cache, q, own_k, own_v * small, f"above {above}, values 2^-{bits}")
        for x in (cache.scales[1], cache.tail[1], cache.values[0][1]):
            x /= small


@pytest.mark.parametrize("dtype", [E4M3, E5M2])
@pytest.mark.parametrize("above", [14, 20])
def test_own_keys_that_take_the_weight_and_bring_no_value(dtype, above):
    """What is left of the output is the cached values', with small weights."""
    rng, k, v, q, own_k, own_v = _case(70 + above, 1, above)
    cache = _cache(k, v, dtype, rng)
    _compare(cache, q, own_k, own_v * 0.0, f"own keys {above} bits above, without values")


@pytest.mark.parametrize("dtype", [E4M3, E5M2])
def test_own_rows_of_another_size_than_the_cache(dtype):
    """The cache's values small and the own rows' large, and the other way."""
    rng, k, v, q, own_k, own_v = _case(31, 2, 6)
    for cached, own in ((2.0 ** -20, 1.0), (2.0 ** -9, 2.0 ** 9), (2.0 ** 12, 1.0), (2.0 ** 12, 2.0 ** -20)):
        cache = _cache(k, (v * cached).bfloat16(), dtype, rng)
        cache.tail[1] *= own / cached
        cache.values[0][1][:, L // 64 * 64:] *= own / cached
        _compare(cache, q, own_k, (own_v * own).bfloat16(), f"cached {cached}, own {own}")


@pytest.mark.parametrize("dtype", [E4M3, E5M2])
@pytest.mark.parametrize("size", [1.0, 2.0 ** -20])
def test_blocks_of_zeros_among_small_values(dtype, size):
    """A block of zeros has scale 1, whatever its neighbours have. Also: a page
    of zeros but for its last code, with scale 1, which counts."""
    rng, k, v, q, own_k, own_v = _case(41, 2, 5)
    v = v * size
    v[:, 64 * 3:64 * 4] = 0.0
    v[:, 64 * 10:64 * 11] = -0.0
    v[::3, :64 * 2] = 0.0
    v[1::3, 64 * 18:64 * 20] = 0.0
    cache = _cache(k, v, dtype, rng)
    _compare(cache, q, own_k, own_v * size, f"zero blocks, values of {size}")
    top = ref.LARGEST[dtype]
    v[:, 64 * 5:64 * 6] = 0.0
    v[:, 64 * 6 - 1, D - 1] = top
    cache = _cache(k, v, dtype, rng)
    assert (cache.scales[1][int(cache.table[0, 5])] == 1.0).all()
    _compare(cache, q, own_k, own_v * size, f"one code, values of {size}")


@pytest.mark.parametrize("dtype", [E4M3, E5M2])
@pytest.mark.parametrize("size", [1.0, 2.0 ** -12])
def test_the_reference_rises_within_a_part(dtype, size):
    """Scores that grow along the request by some 40 bits, and values whose
    blocks differ by many powers of two: the reference is raised after the first
    tile of a part, the output's sums rescaled."""
    rng, k, v, q, own_k, own_v = _case(51, 2, 0)
    direction = torch.from_numpy(rng.standard_normal((HEADS, 1, D)))
    q = (q.double() * 0.2 + direction[:, 0].repeat_interleave(H // HEADS, 0)).bfloat16()
    grow = torch.linspace(0.0, 40.0, L).double()[None, :, None] / (D ** 0.5 * np.log2(np.e))
    k = (k.double() + direction * grow).bfloat16()
    cache = _cache(k, v * size, dtype, rng)
    # scores in bits, of the first node, and the largest of each tile
    s = torch.einsum("hd,hld->hl", q[0, 0].double(), cache.values[0][0]) * D ** -0.5 * np.log2(np.e)
    tile = [s[:, 128 * i:128 * (i + 1)].amax(1) for i in range(L // 128)]
    rises = 0
    for lo, hi in _parts():
        rises += hi - max(lo, 1) >= 4 and bool((tile[hi - 2] - tile[max(lo, 1) - 1]).max() > 10.0)
    assert rises >= 16  # a weight would pass 2^15 where the score is 8 bits above the first tile's
    _compare(cache, q, own_k, own_v * size, f"rising, values of {size}")
    mult = torch.tensor([2.0 ** m for m in (-40, 8, 0, -8, 12, -30, -3, 5, 3, 0, -20, 9, 0, 1, -12, 4, 0, 2, 7, -6, 0)])
    wide = (v * size * mult.repeat_interleave(64)[None, :L, None]).bfloat16()
    cache = _cache(k, wide, dtype, rng)
    _compare(cache, q, own_k, own_v * size, f"rising and unlike blocks, values of {size}")


def test_a_first_key_that_takes_the_weight_and_brings_no_value():
    """A block's first token 14 bits above the rest, of value zero."""
    rng, k, v, q, own_k, own_v = _case(61, 1, 0)
    q = (q.double().abs() * 0.1 + 1.0).bfloat16()
    k = (k * 0.1).bfloat16()
    k[:, 0] = 14.0 / (D ** 0.5 * np.log2(np.e))
    v[:, 0] = 0.0
    cache = _cache(k, v, E4M3, rng)
    _compare(cache, q, own_k, own_v, "sink")
