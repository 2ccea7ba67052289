"""The paged 16-bit cache: append with rotation and causal attention against
plain 64-bit implementations; what the rows do not see; refusals."""
import numpy as np
import pytest
import torch

import kv16_reference as ref
import speculative_decode_verify_w4a16_gb300 as sv
from helpers import dev

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16
INPUT = 5  # W4A16_ERR_DEVICE_INPUT


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decode_verify_w4a16_gb300 import build
    build.build()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=dev())


def _starts(counts):
    return [0, *np.cumsum(counts).tolist()]


def _randn(rng, *shape, dtype=BF16):
    gen = torch.Generator(device=dev())
    gen.manual_seed(int(rng.integers(1 << 30)))
    return torch.randn(*shape, generator=gen, device=dev()).to(dtype)


class Case:
    """A cache in use with a step's rows in it, other layers and pages holding NaN."""

    def __init__(self, seed, dtype, D, H, Hkv, lens, counts, pad=0, layers=2, layer=1):
        rng = np.random.default_rng(seed)
        self.lens, self.counts, self.D, self.H, self.Hkv, self.layer = lens, counts, D, H, Hkv, layer
        self.table, pages = ref.paged(rng, lens, counts)
        self.cache = sv.KV16Cache(*(torch.full((layers, pages, Hkv, 64, D), torch.nan, dtype=dtype, device=dev())
                                    for _ in range(2)))
        self.T = sum(counts) + pad
        self.q = _randn(rng, self.T, H, D, dtype=dtype)
        chan = torch.exp(0.5 * _randn(rng, Hkv, 1, D)).to(dtype)
        self.kv = []
        for b, (past, n) in enumerate(zip(lens, counts)):
            k, v = (_randn(rng, Hkv, past + n, D, dtype=dtype) for _ in range(2))
            self.kv.append([k * chan, v])
            self.put(b)

    def put(self, b):
        """Request b's keys and values into its pages; the last page's other rows stay NaN."""
        for x, rows in zip((self.cache.k, self.cache.v), self.kv[b]):
            L = rows.shape[1]
            if L:
                pos = torch.arange(L)
                page = self.table[b, pos // 64].long().to(dev())
                x[self.layer][page, :, (pos % 64).to(dev())] = rows.transpose(0, 1)

    def run(self, **kw):
        kw.setdefault("row_start", _i32(_starts(self.counts)))
        return sv.kv16_attention(self.q, self.cache, self.layer, self.table.to(dev()), _i32(self.lens), **kw)

    def check(self, got, window=0, scale=None, requests=None):
        worst, at = 0.0, _starts(self.counts)
        for b in range(len(self.lens)) if requests is None else requests:
            if self.counts[b] == 0:
                continue
            k, v = self.kv[b]
            want, mag = ref.attention(self.q[at[b]:at[b + 1]], k, v, self.lens[b], window, scale)
            g = got[at[b]:at[b + 1]].double()
            assert torch.equal(g.isfinite(), want.isfinite()), b
            bound = ref.attention_bound(want, mag, v, self.q.dtype)
            e = ((g - want).abs() / bound)[want.isfinite()]
            if e.numel():
                worst = max(worst, float(e.max()))
        print(f"max |err| / bound = {worst:.3f}")
        assert worst <= 1.0


SHAPES = [
    # lens, counts
    ([0], [1]), ([63], [1]), ([64], [1]), ([127], [2]), ([1003], [1]), ([5000], [5]),
    ([0], [300]), ([0, 0, 17], [65, 128, 129]), ([100, 0, 700, 64], [64, 1, 0, 63]),
    ([0, 1, 2, 3, 0], [0, 0, 7, 0, 0]), ([777], [513]), ([3000, 90, 1], [1, 400, 1]),
]


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F16, 64), (F16, 128), (BF16, 64)])
@pytest.mark.parametrize("H,Hkv", [(8, 1), (4, 4), (10, 2), (3, 1)])
@pytest.mark.parametrize("lens,counts", SHAPES)
def test_attention(dtype, D, H, Hkv, lens, counts):
    c = Case(len(lens) + H, dtype, D, H, Hkv, lens, counts, pad=3)
    out = torch.full((c.T, H, D), 7.0, dtype=dtype, device=dev())
    assert c.run(out=out) is out
    torch.cuda.synchronize()
    assert sv.check_device_status() == 0
    c.check(out)
    assert (out[sum(counts):] == 7).all()  # rows of no request stay


@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 100, 128, 200, 1000, 100000])
@pytest.mark.parametrize("lens,counts", [([0, 500], [300, 1]), ([1000], [70]), ([130, 2000, 63], [5, 33, 1])])
def test_windows(window, lens, counts):
    c = Case(window, BF16, 128, 6, 2, lens, counts)
    # what no row of a request sees any more may be gone: NaN, pages without an id
    for b, past in enumerate(lens):
        gone = max(0, past - window + 1)
        for x in c.kv[b]:
            x[:, :gone] = torch.nan
        c.put(b)
        c.table[b, :gone // 64] = -1
        for x in c.kv[b]:
            x[:, :gone] = 0  # (for the reference: weights of zero)
    out = c.run(window=window)
    torch.cuda.synchronize()
    assert sv.check_device_status() == 0
    c.check(out, window)


@pytest.mark.parametrize("H,Hkv,D", [(64, 8, 128), (32, 2, 64), (16, 16, 128), (20, 4, 128), (71, 1, 64)])
def test_head_groups_and_many_requests(H, Hkv, D):
    rng = np.random.default_rng(H)
    B = 70
    lens = rng.integers(0, 400, B).tolist()
    counts = rng.choice([0, 1, 1, 1, 5, 40], B).tolist()
    c = Case(H, BF16, D, H, Hkv, lens, counts, pad=1)
    out = c.run()
    torch.cuda.synchronize()
    assert sv.check_device_status() == 0
    c.check(out)


@pytest.mark.parametrize("lens,counts,H,Hkv", [([40000, 9], [1, 1], 8, 2), ([20000], [64], 16, 2), ([9000], [700], 8, 2),
                                               ([0], [5000], 4, 1), ([3], [1], 64, 8)])
def test_long_and_cut(lens, counts, H, Hkv):
    c = Case(11, BF16, 128, H, Hkv, lens, counts, layers=1, layer=0)
    out = c.run()
    again = c.run()
    torch.cuda.synchronize()
    assert sv.check_device_status() == 0
    c.check(out)
    assert torch.equal(out, again)  # the same sums in the same order


def test_hundreds_of_requests():
    rng = np.random.default_rng(1)
    B = 1100
    lens, counts = rng.integers(0, 90, B).tolist(), rng.choice([0, 1, 2], B).tolist()
    c = Case(2, F16, 64, 4, 2, lens, counts)
    out = c.run()
    torch.cuda.synchronize()
    assert sv.check_device_status() == 0
    c.check(out)


def test_same_number_of_rows_each_and_strides():
    """row_start left out; q a slice of the fused projection [B, n, .., D]."""
    c = Case(5, BF16, 128, 8, 2, [5, 70, 200], [4, 4, 4])
    qkv = torch.full((3, 4, 8 + 4, 128), torch.nan, dtype=BF16, device=dev())
    qkv[:, :, 1:9] = c.q.view(3, 4, 8, 128)
    q = qkv[:, :, 1:9]
    out = sv.kv16_attention(q, c.cache, 1, c.table.to(dev()), _i32(c.lens))
    assert out.shape == q.shape and out.is_contiguous()
    c.check(out.view(12, 8, 128))
    out2 = sv.kv16_attention(q, c.cache, 1, c.table.to(dev()), _i32(c.lens), scale=0.03)
    c.check(out2.view(12, 8, 128), scale=0.03)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_scores_that_rise_and_fall(dtype):
    """Later keys with far larger scores, then far smaller ones: the sums are rescaled."""
    for sign in (1, -1):
        c = Case(6, dtype, 128, 8, 1, [900], [40])
        ramp = torch.linspace(-3, 3, 940, device=dev())[None, :, None] * sign
        c.q = (c.q.abs() + 0.25).to(dtype)
        c.kv[0][0] = (c.kv[0][0] * 0.1 + ramp).to(dtype)
        c.put(0)
        out = c.run()
        torch.cuda.synchronize()
        c.check(out)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("down", [4, 10, 16])
def test_many_small_weights_beside_a_large_one(dtype, down):
    """One key `down` bits above thousands of equal ones, whose values count."""
    L = 8000
    c = Case(7, dtype, 128, 2, 1, [L - 1], [1])
    k, v = c.kv[0]
    k.zero_()
    q = torch.zeros_like(c.q)
    q[..., 0] = 8.0
    c.q = q
    k[:, 4000, 0] = down * 0.6931471805599453 * 128 ** 0.5 / 8.0
    v.fill_(1.0)
    v[:, 4000] = 0.0
    c.put(0)
    out = c.run()
    torch.cuda.synchronize()
    c.check(out)


def test_what_a_row_does_not_see_does_not_touch_it():
    """NaN and infinities among the later keys and values of the same step."""
    for seed, (n, H, Hkv) in enumerate([(9, 4, 1), (200, 2, 1), (300, 8, 2)]):
        c = Case(8 + seed, BF16, 128, H, Hkv, [70], [n])
        k, v = c.kv[0]
        k[0, 70 + n // 2, 3] = torch.nan
        v[0, 70 + 2 * n // 3, 5] = torch.inf
        v[0, 70 + 2 * n // 3, 9] = -torch.inf
        v[0, 70 + n - 2, 7] = torch.nan
        c.put(0)
        out = c.run()
        torch.cuda.synchronize()
        assert sv.check_device_status() == 0
        first = out[:n // 2].double()
        assert first.isfinite().all()
        c.check(out)
        # rows between: NaN for the heads of the group that sees the bad key
        assert out[n // 2:, :H // Hkv].isnan().all() if Hkv == 1 else True


def test_infinite_values_that_are_seen():
    c = Case(15, BF16, 64, 4, 1, [0], [150])
    k, v = c.kv[0]
    v[0, 100, 5], v[0, 120, 5], v[0, 130, 6] = torch.inf, torch.inf, -torch.inf
    c.put(0)
    out = c.run()
    torch.cuda.synchronize()
    c.check(out)
    assert (out[100:, :, 5] == torch.inf).all() and (out[130:, :, 6] == -torch.inf).all()
    assert out[:100].isfinite().all()


def test_bad_pages_and_lengths():
    c = Case(20, BF16, 128, 4, 2, [200, 300, 100], [5, 6, 7])
    good = c.run()
    for bad in (-1, -2, c.cache.k.shape[1], 2 ** 31 - 1):  # reads as zeros
        table = c.table.clone()
        table[1, 2] = bad
        out = sv.kv16_attention(c.q, c.cache, 1, table.to(dev()), _i32(c.lens), row_start=_i32(_starts(c.counts)))
        torch.cuda.synchronize()
        assert sv.check_device_status() == INPUT
        saved = [x.clone() for x in c.kv[1]]
        for x in c.kv[1]:
            x[:, 128:192] = 0
        c.check(out)
        c.kv[1] = saved
    max_blocks = c.table.shape[1]
    for lens, starts, left in (([200, -1, 100], [0, 5, 11, 18], [1]), ([200, max_blocks * 64, 100], [0, 5, 11, 18], [1]),
                               ([200, 2 ** 31 - 1, 100], [0, 5, 11, 18], [1]), ([200, 300, 100], [0, 5, 11, 19], [2]),
                               ([200, 300, 100], [-1, 5, 11, 18], [0])):
        out = torch.full_like(good, 7.0)
        sv.kv16_attention(c.q, c.cache, 1, c.table.to(dev()), _i32(lens), row_start=_i32(starts), out=out)
        torch.cuda.synchronize()
        assert sv.check_device_status() == INPUT, (lens, starts)
        at = _starts(c.counts)
        assert all((out[at[b]:at[b + 1]] == 7).all() for b in left), (lens, starts)
        # the others' rows, by the bound: where a request's keys are cut depends on the batch, and so the sums' order
        c.check(out, requests=[b for b in range(3) if b not in left])
    # a request that brings nothing may have any length
    out = torch.full_like(good, 7.0)
    sv.kv16_attention(c.q, c.cache, 1, c.table.to(dev()), _i32([200, -5, 100]), row_start=_i32([0, 5, 5, 5]), out=out)
    torch.cuda.synchronize()
    assert sv.check_device_status() == 0
    c.check(out, requests=[0])
    assert (out[5:] == 7).all()
    # falling rows: reported, nothing out of bounds
    sv.kv16_attention(c.q, c.cache, 1, c.table.to(dev()), _i32(c.lens), row_start=_i32([0, 12, 5, 18]), out=out)
    torch.cuda.synchronize()
    assert sv.check_device_status() == INPUT


def test_offsets_past_32_bits():
    """Pages whose elements lie beyond 2^31 of the cache's start, both kinds of bytes and elements."""
    pages = 40000  # 40000 * 8 * 64 * 128 = 2.6e9 elements
    cache = sv.KV16Cache(*(torch.empty((1, pages, 8, 64, 128), dtype=BF16, device=dev()) for _ in range(2)))
    small = Case(30, BF16, 128, 16, 8, [300], [9], layers=1, layer=0)
    table = torch.tensor([[pages - 1 - 7 * i for i in range(small.table.shape[1])]], dtype=torch.int32)
    k, v = small.kv[0]
    lens = _i32([0])
    sv.kv16_append(cache, 0, k.transpose(0, 1).contiguous(), v.transpose(0, 1).contiguous(), table.to(dev()), lens)
    for x, rows in zip((cache.k, cache.v), (k, v)):
        assert torch.equal(ref.rows_of(table, 0, x[0], 0, 309), rows)
    out = sv.kv16_attention(small.q, cache, 0, table.to(dev()), _i32([300]))
    torch.cuda.synchronize()
    assert sv.check_device_status() == 0
    small.check(out)


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F16, 64)])
@pytest.mark.parametrize("rot,interleaved", [(0, False), (64, False), (32, True), (16, False)])
@pytest.mark.parametrize("lens,counts,pad", [([0], [1], 0), ([63, 64, 5], [2, 1, 130], 2), ([7, 900, 0, 128], [0, 3, 65, 0], 1),
                                             (list(range(40)), [1] * 40, 0)])
def test_append(dtype, D, rot, interleaved, lens, counts, pad):
    rng = np.random.default_rng(len(lens) + rot)
    H, Hkv, T = 6, 2, sum(counts) + pad
    table, pages = ref.paged(rng, lens, counts)
    qkv = _randn(rng, T, H + 2 * Hkv, D, dtype=dtype)
    before = qkv.clone()
    cache = sv.kv16_cache(2, pages, Hkv, D, dtype)
    for x in (cache.k, cache.v):
        x.fill_(3.0)
    freqs = sv.rope_frequencies(rot, 500000.0, interleaved=interleaved) if rot else None
    q_out = torch.full((T, H, D), 7.0, dtype=dtype, device=dev())
    q, k, v = qkv.split((H, Hkv, Hkv), 1)
    got = sv.kv16_append(cache, 1, k, v, table.to(dev()), _i32(lens), row_start=_i32(_starts(counts)), rope=freqs, q=q,
                         q_out=q_out)
    torch.cuda.synchronize()
    assert sv.check_device_status() == 0 and got is q_out and torch.equal(qkv, before)
    assert (q_out[sum(counts):] == 7).all()
    positions = np.concatenate([np.arange(n) + a for a, n in zip(lens, counts)])
    rows = len(positions)
    angles = sv.rope_angles(rot, 500000.0)[0] if rot else []
    cos, sin = ref.cos_sin(positions, angles)
    written = torch.zeros(cache.k.shape, dtype=torch.bool, device=dev())
    at = _starts(counts)
    for x, src in ((q_out, q), (cache.k[1], k), (cache.v[1], v)):
        if x is not q_out:
            x = torch.cat([ref.rows_of(table, b, x, a, a + n).transpose(0, 1) for b, (a, n) in enumerate(zip(lens, counts))])
        x = x[:rows].cpu()
        if src is v or not rot:
            assert torch.equal(x, src[:rows].cpu())
            continue
        y, mag = ref.rotate(src[:rows].cpu(), cos, sin, interleaved)
        assert ((x.double() - y).abs() <= ref.rotation_bound(y, mag, dtype)).all()
        assert torch.equal(x[..., rot:], src[:rows, :, rot:].cpu())
        # as rope() gives it
        assert torch.equal(x.to(dev()), sv.rope(src[:rows], _i32(positions.tolist()), freqs))
    for b, (a, n) in enumerate(zip(lens, counts)):
        pos = torch.arange(a, a + n)
        written[1][table[b, pos // 64].long().to(dev()), :, (pos % 64).to(dev())] = True
    assert (cache.k[~written] == 3).all() and (cache.v[~written] == 3).all() and len(at) == len(lens) + 1


def test_append_in_place_and_without_queries():
    rng = np.random.default_rng(3)
    table, pages = ref.paged(rng, [60, 3], [6, 6])
    qkv = _randn(rng, 2, 6, 4, 128)
    freqs = sv.rope_frequencies(128)
    a, b = sv.kv16_cache(1, pages, 1), sv.kv16_cache(1, pages, 1)
    q, k, v = qkv.split((2, 1, 1), 2)
    turned = sv.kv16_append(a, 0, k, v, table.to(dev()), _i32([60, 3]), rope=freqs, q=q)
    assert turned.shape == q.shape and turned.is_contiguous()
    assert sv.kv16_append(b, 0, k, v, table.to(dev()), _i32([60, 3]), rope=freqs) is None
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
    assert sv.kv16_append(b, 0, k, v, table.to(dev()), _i32([60, 3]), rope=freqs, q=q, q_out=q) is q
    assert torch.equal(q, turned)
    torch.cuda.synchronize()
    assert sv.check_device_status() == 0


def test_append_bad_input_is_skipped():
    rng = np.random.default_rng(4)
    table, pages = ref.paged(rng, [60, 3], [6, 6])
    k, v, q = (_randn(rng, 12, h, 128) for h in (2, 2, 4))
    starts = [0, 6, 12]

    def run(table=table, lens=(60, 3), starts=starts):
        c = sv.kv16_cache(1, pages, 2)
        q_out = torch.full_like(q, 7.0)
        sv.kv16_append(c, 0, k, v, table.to(dev()), _i32(list(lens)), row_start=_i32(starts), q=q, q_out=q_out)
        torch.cuda.synchronize()
        return c, q_out, sv.check_device_status()

    good, q_good, status = run()
    assert status == 0
    for bad in (-1, -7, pages, 2 ** 31 - 1):
        t = table.clone()
        t[0, 1] = bad  # positions 64, 65 of request 0
        c, q_out, status = run(table=t)
        assert status == INPUT and torch.equal(q_out, q_good)
        lost = int(table[0, 1])
        assert (c.k[0, lost] == 0).all() and (c.v[0, lost] == 0).all()
        others = [i for i in range(pages) if i != lost]
        assert torch.equal(c.k[0, others], good.k[0, others]) and torch.equal(c.v[0, others], good.v[0, others])
    for lens, st in (((-1, 3), starts), ((2 ** 31 - 1, 3), starts), ((table.shape[1] * 64 - 5, 3), starts),
                     ((60, 3), [-2, 6, 12])):
        c, q_out, status = run(lens=lens, starts=st)
        assert status == INPUT and (q_out[:6] == 7).all() and torch.equal(q_out[6:], q_good[6:])
        pos = torch.arange(3, 9)
        assert torch.equal(ref.rows_of(table, 1, c.k[0], 3, 9), ref.rows_of(table, 1, good.k[0], 3, 9)) and len(pos) == 6
    c, q_out, status = run(starts=[0, 6, 13])
    assert status == INPUT and torch.equal(q_out[:6], q_good[:6]) and (q_out[6:] == 7).all()
    _, _, status = run(starts=[0, 13, 12])
    assert status == INPUT


def test_no_rows_at_all():
    c = sv.kv16_cache(1, 2, 1)
    e = torch.empty(0, 1, 128, dtype=BF16, device=dev())
    args = (torch.full((2, 1), -1, dtype=torch.int32, device=dev()), _i32([0, 0]))
    assert sv.kv16_append(c, 0, e, e, *args, row_start=_i32([0, 0, 0])) is None
    assert sv.kv16_attention(e, c, 0, *args, row_start=_i32([0, 0, 0])).shape == (0, 1, 128)
    pad = torch.full((3, 1, 128), 7.0, dtype=BF16, device=dev())  # rows, none of them a request's
    sv.kv16_append(c, 0, pad, pad, *args, row_start=_i32([0, 0, 0]))
    out = pad.clone()
    sv.kv16_attention(pad * 2, c, 0, *args, row_start=_i32([0, 0, 0]), out=out)
    torch.cuda.synchronize()
    assert sv.check_device_status() == 0
    assert torch.equal(out, pad) and (c.k == 0).all()


# ----------------------------------------------------------- used together

@pytest.mark.parametrize("dtype", [BF16, F16])
def test_a_prompt_in_chunks_is_the_prompt_at_once(dtype):
    """rope, append and attention step by step: chunks, then single tokens,
    beside another request; the sums run over the same keys."""
    rng = np.random.default_rng(9)
    L, H, Hkv, D = 700, 8, 2, 128
    qkv = _randn(rng, L, H + 2 * Hkv, D, dtype=dtype)
    freqs = sv.rope_frequencies(D, 500000.0)
    table, pages = ref.paged(rng, [L, 40], [0, 300])
    once = sv.kv16_cache(1, pages, Hkv, D, dtype)
    q, k, v = qkv.split((H, Hkv, Hkv), 1)
    qr = sv.kv16_append(once, 0, k, v, table[:1].to(dev()), _i32([0]), rope=freqs, q=q)
    whole = sv.kv16_attention(qr, once, 0, table[:1].to(dev()), _i32([0]))
    cache, at, other = sv.kv16_cache(1, pages, Hkv, D, dtype), 0, 0
    for n in (1, 130, 64, 5, 200, 290, *[1] * 10):
        m = int(rng.integers(0, 9))  # the other request's rows: the same tokens over and over
        rows = torch.cat([qkv[:m], qkv[at:at + n]])
        # the other request comes first in the step, second in the batch's tables
        t = table[[1, 0]].to(dev())
        q, k, v = rows.split((H, Hkv, Hkv), 1)
        start, lens = _i32([0, m, m + n]), _i32([other, at])
        qr = sv.kv16_append(cache, 0, k, v, t, lens, row_start=start, rope=freqs, q=q)
        out = sv.kv16_attention(qr, cache, 0, t, lens, row_start=start)
        got, want = out[m:].double(), whole[at:at + n].double()
        kk, vv = (ref.rows_of(table, 0, x[0], 0, at + n) for x in (cache.k, cache.v))
        _, mag = ref.attention(qr[m:], kk, vv, at)
        assert ((got - want).abs() <= 2 * ref.attention_bound(want, mag, vv, dtype)).all()
        at, other = at + n, other + m
    assert at == L
    for x, y in ((cache.k, once.k), (cache.v, once.v)):
        assert torch.equal(ref.rows_of(table, 0, x[0], 0, L), ref.rows_of(table, 0, y[0], 0, L))
    torch.cuda.synchronize()
    assert sv.check_device_status() == 0


def test_pages_from_the_block_plan():
    """kv_block_plan gives the pages when it is asked with lens + 63: a block
    then gets its page with its first token."""
    rng = np.random.default_rng(12)
    B, H, Hkv, D, pages = 3, 4, 2, 128, 30
    lens = _i32([0, 0, 0])
    table = torch.full((B, 8), -1, dtype=torch.int32, device=dev())
    ring = torch.from_numpy(rng.permutation(pages).astype(np.int32)).to(dev())
    queue, tails = _i32([0, pages, 0]), _i32([0, 2, 4])
    cache, kept = sv.kv16_cache(1, pages, Hkv, D), [[] for _ in range(B)]
    for counts in ([65, 1, 0], [0, 63, 64], [1, 1, 1], [130, 0, 2]):
        T, start = sum(counts), _i32(_starts(counts))
        q, k, v = (_randn(rng, T, h, D) for h in (H, Hkv, Hkv))
        plan = sv.kv_block_plan(lens + 63, tails, table, ring, queue, row_start=start, rows=T)
        sv.kv16_append(cache, 0, k, v, table, lens, row_start=start)
        out = sv.kv16_attention(q, cache, 0, table, lens, row_start=start)
        at = _starts(counts)
        for b in range(B):
            kept[b].append((k[at[b]:at[b + 1]], v[at[b]:at[b + 1]]))
            if counts[b]:
                kk, vv = (torch.cat([x[i] for x in kept[b]]).transpose(0, 1) for i in range(2))
                want, mag = ref.attention(q[at[b]:at[b + 1]], kk, vv, int(lens[b]))
                bound = ref.attention_bound(want, mag, vv, BF16)
                assert ((out[at[b]:at[b + 1]].double() - want).abs() <= bound).all()
        lens, queue = plan.new_lens - 63, plan.queue
    torch.cuda.synchronize()
    assert sv.check_device_status() == 0
    held = table[table >= 0].tolist()
    assert len(held) == len(set(held)) == sum(-(-n // 64) for n in lens.tolist())


# --------------------------------------------------- streams and graphs

def test_streams_have_workspaces_of_their_own():
    cases = [Case(40 + i, BF16, 128, 16, 2, [1900 + 500 * i, 700], [3, 90 + i]) for i in range(2)]
    want = [c.run().clone() for c in cases]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for _ in range(30):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(cases[i].run())
    torch.cuda.synchronize()
    assert sv.check_device_status() == 0
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])


def test_the_stream_argument():
    c, s = Case(50, BF16, 128, 8, 2, [3000], [3]), torch.cuda.Stream()
    want = c.run()
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    c.run(out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, want)


def test_graphs_and_eager_calls_in_between():
    """Two captured graphs and eager calls; lengths that move between replays."""
    cases = [Case(60 + i, BF16, 128, 8, 2, [2000, 100], [2, 70]) for i in range(2)]
    args = [(c.table.to(dev()), _i32(c.lens), _i32(_starts(c.counts))) for c in cases]
    graphs, outs = [], []
    side = torch.cuda.Stream()
    for c, (t, lens, start) in zip(cases, args):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(sv.kv16_attention(c.q, c.cache, 1, t, lens, row_start=start))
        graphs.append(g)
    big = Case(70, BF16, 128, 64, 8, [4000], [300])
    for past in (2000, 1500, 130):
        for i, c in enumerate(cases):
            args[i][1][0] = past
            graphs[i].replay()
            big.run()
            graphs[i].replay()
            eager = sv.kv16_attention(c.q, c.cache, 1, *args[i][:2], row_start=args[i][2])
            assert torch.equal(outs[i], eager)
    graphs[0].replay()
    graphs[1].replay()
    torch.cuda.synchronize()
    assert sv.check_device_status() == 0


def test_refusals():
    c = Case(80, BF16, 128, 4, 2, [10, 20], [3, 3])
    t, lens, start = c.table.to(dev()), _i32(c.lens), _i32([0, 3, 6])
    ok = dict(row_start=start)
    q, k = c.q, c.q[:, :2]

    def attn(q=q, cache=c.cache, layer=1, t=t, lens=lens, **kw):
        return sv.kv16_attention(q, cache, layer, t, lens, **{**ok, **kw})

    def append(k=k, v=k, cache=c.cache, layer=0, t=t, lens=lens, **kw):
        return sv.kv16_append(cache, layer, k, v, t, lens, **{**ok, **kw})

    half = sv.KV16Cache(c.cache.k[:, ::2], c.cache.v[:, ::2])
    other = sv.KV16Cache(c.cache.k, c.cache.v.half())
    eight = sv.KV16Cache(c.cache.k[:, :, :, :8], c.cache.v[:, :, :, :8])
    for call in (attn, append):
        for kw in (dict(cache=half), dict(cache=other), dict(cache=eight), dict(layer=2), dict(layer=-1), dict(t=t[:1]),
                   dict(t=t.long()), dict(t=torch.cat([t, t], 1)[:, ::2]), dict(lens=lens.long()), dict(lens=lens.cpu()),
                   dict(row_start=start[:2]), dict(row_start=start.long()), dict(t=t.cpu())):
            with pytest.raises(ValueError):
                call(**kw)
    three = _i32([1, 2, 3, 4])
    for kw in (dict(q=q.half()), dict(q=q[..., :64]), dict(q=q.cpu()), dict(q=q.transpose(1, 2)), dict(out=q[:, :2]),
               dict(out=q.float()), dict(out=torch.empty(8, 4, 128, dtype=BF16, device=dev())[1:7, ::2]),
               dict(lens=three, t=t[:1].expand(4, -1).contiguous(), row_start=None), dict(ws=torch.zeros(1 << 20))):
        with pytest.raises(ValueError):
            attn(**kw)
    for kw in (dict(k=k.half()), dict(v=k[:3]), dict(k=c.q[:, :1]), dict(q=q[:3]), dict(q=q.half()), dict(q_out=q),
               dict(rope=sv.rope_frequencies(256)), dict(rope=sv.rope_frequencies(128, device="cpu")),
               dict(q=q, q_out=q.float())):
        with pytest.raises(ValueError):
            append(**kw)
    for kw in (dict(window=-1), dict(scale=0.0), dict(scale=float("nan")), dict(q=q[:, :3])):
        with pytest.raises(sv.W4A16Error):
            attn(**kw)
    for dtype in (torch.float32, torch.float8_e4m3fn):
        with pytest.raises(ValueError):
            sv.kv16_cache(1, 4, 2, dtype=dtype)
    torch.cuda.synchronize()
    assert sv.check_device_status() == 0
