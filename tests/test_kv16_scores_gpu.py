"""The paged 16-bit attention with scores far from zero: finite scores give what
the definition gives, however large they are. But for the last test the scores
are whole numbers that fp32 holds, so that the weights depend on their
differences alone."""
import numpy as np
import pytest
import torch

import kv16_reference as ref
import speculative_decode_verify_w4a16_gb300 as sv
from helpers import dev
from test_kv16_gpu import BF16, F16, Case, _starts

pytestmark = pytest.mark.gpu

# one row, slots that share the rows and ones that do not, cut units, the queue's
SHAPES = [([5], [1]), ([1003], [1]), ([900], [40]), ([0], [300]), ([20000], [3]), ([9000], [200]),
          ([100 + b for b in range(80)], [1 + b % 3 for b in range(80)])]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decode_verify_w4a16_gb300 import build
    build.build()


def _run(c, **kw):
    for b in range(len(c.lens)):
        c.put(b)
    out = c.run(**kw)
    torch.cuda.synchronize()
    assert sv.check_device_status() == 0
    return out


@pytest.mark.parametrize("dtype,D,dims,first,second", [
    (F16, 128, 4, 32752.0, 61408.0), (F16, 64, 4, 32752.0, 61408.0), (F16, 64, 1, 32752.0, 44704.0),
    (BF16, 128, 128, 1.9296875 * 2.0 ** 45, 1.8046875 * 2.0 ** 45), (BF16, 64, 1, 1.9296875 * 2.0 ** 20, 1.8046875 * 2.0 ** 20),
])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("lens,counts", SHAPES)
def test_the_largest_scores_share_the_row(dtype, D, dims, first, second, sign, lens, counts):
    """Scores dims * first * second * 2^-a, a = 0 .. 5 by the key: those that are largest of what a row sees weigh the
    same, the others nothing. fp16: up to 2^33, 2^30 in powers of two; bf16: up to 2^99. The products have 22 bits (fp16)
    or 16, and so up to 24 for four of them, or 128: fp32 holds every sum."""
    rng = np.random.default_rng(len(lens) + int(sign))
    c = Case(1, dtype, D, 8, 4, lens, counts)
    c.q.zero_()
    c.q[..., :dims] = sign * first
    for k, v in c.kv:
        keys = torch.from_numpy(second * 2.0 ** -rng.integers(0, 6, k.shape[:2]).astype(np.float64)).to(dev())
        k.zero_()
        k[..., :dims] = keys[..., None]
        assert (k[..., 0].double() == keys).all() and c.q[0, 0, 0].double() == sign * first
    out = _run(c)
    assert out.isfinite().all()
    c.check(out)


@pytest.mark.parametrize("dtype,D", [(F16, 128), (BF16, 64), (BF16, 128)])
@pytest.mark.parametrize("first,second", [(64, 125), (8, 125), (64, 512), (512, 2048), (-64, 125), (-512, 2048)])
@pytest.mark.parametrize("lens,counts", SHAPES)
def test_differences_of_large_scores(dtype, D, first, second, lens, counts):
    """Scores first * second + j, j = 0 .. 255 by the key: on both sides of where the weights are taken another way (8000
    is 1020 powers of two at D 128), and beyond it."""
    rng = np.random.default_rng(len(lens) + abs(first))
    c = Case(2, dtype, D, 8, 4, lens, counts)
    c.q.zero_()
    c.q[..., 0], c.q[..., 1] = first, 1
    for k, v in c.kv:
        k.zero_()
        k[..., 0] = second
        k[..., 1] = torch.from_numpy(rng.integers(0, 256, k.shape[:2])).to(dev())
    c.check(_run(c))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("lens,counts", SHAPES)
def test_scores_that_leave_and_come_back(dtype, lens, counts):
    """A few keys far above the others, and rows that see none of them yet.

    A far score is 2^15 and some tens, a sum of D = 128 products in fp32: it is off by at most D 2^-24 times the products'
    magnitudes, which are below 2^15 + 2^11 (by Cauchy's inequality, norms of less than 45 each for the other 127, which is
    asserted). So the weights are off by the factor exp(2 e), e that times the scale, in the worst case, and a row by
    exp(2 e) - 1 times the weighted magnitudes and itself."""
    rng = np.random.default_rng(3)
    c = Case(3, dtype, 128, 8, 4, lens, counts)
    c.q[..., 0] = 64
    for k, v in c.kv:
        far = torch.from_numpy(rng.integers(0, 50, k.shape[:2]) == 0).to(dev())
        k[..., 0] = torch.where(far, 512.0, 0.0).to(dtype)
        assert k[..., 1:].double().norm(dim=-1).max() < 45
    assert c.q[..., 1:].double().norm(dim=-1).max() < 45
    out = _run(c)
    factor = np.expm1(2 * 128 * 2.0 ** -24 * (2 ** 15 + 2 ** 11) * 128 ** -0.5)
    at = _starts(counts)
    for b, (k, v) in enumerate(c.kv):
        want, mag = ref.attention(c.q[at[b]:at[b + 1]], k, v, lens[b])
        bound = ref.attention_bound(want, mag, v, dtype) + factor * (mag + want.abs())
        assert ((out[at[b]:at[b + 1]].double() - want).abs() <= bound).all(), b


@pytest.mark.parametrize("dtype,big", [(F16, 32752.0), (BF16, 1.9296875 * 2.0 ** 30)])
@pytest.mark.parametrize("window", [0, 70])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lens,counts", SHAPES)
def test_beside_ordinary_rows(dtype, big, window, in_place, lens, counts):
    """Every third row has scores of more than 2^24 powers of two, of one element; the others have zeros there, and get what
    they get without them, to the bit. In place of the queries, with a window and a page that is none too."""
    rng = np.random.default_rng(len(lens))
    c = Case(4, dtype, 128, 8, 4, lens, counts, pad=1)
    c.q[..., 0] = 0
    far = torch.arange(c.T, device=dev()) % 3 == 1
    for k, v in c.kv:
        k[..., 0] = torch.from_numpy(44704.0 * 2.0 ** -rng.integers(0, 6, k.shape[:2]).astype(np.float64)).to(dev())
    ordinary = c.q.clone()
    ordinary[far] = 0
    c.q[far] = 0
    c.q[far, :, 0] = big
    if lens[0] == 900:  # a page that is none reads as zeros
        for x in c.kv[0]:
            x[:, 128:192] = 0
    for b in range(len(lens)):
        c.put(b)
    if lens[0] == 900:
        c.table[0, 2] = -1
    q = c.q
    out = c.run(window=window, out=c.q.clone() if not in_place else None)
    torch.cuda.synchronize()
    status = sv.check_device_status()
    assert status == (5 if lens[0] == 900 and not window else 0)
    if in_place:
        want, c.q = out, q.clone()
        out = c.run(window=window, out=c.q)
        torch.cuda.synchronize()
        assert sv.check_device_status() == status
        assert out is c.q and torch.equal(out[:sum(counts)], want[:sum(counts)])
    c.q = q
    c.check(out, window)
    c.q = ordinary
    assert torch.equal(c.run(window=window)[:sum(counts)][~far[:sum(counts)]], out[:sum(counts)][~far[:sum(counts)]])
    sv.check_device_status()


def test_values_that_are_not_finite():
    """Rows that are done over see the values of their keys alone, guarded ones among them."""
    for lens, counts in (([100], [150]), ([20000], [40])):
        c = Case(5, F16, 128, 4, 1, lens, counts)
        c.q.zero_()
        c.q[..., 0] = 32752.0
        k, v = c.kv[0]
        k.zero_()
        k[..., 0] = 44704.0
        at = lens[0] + counts[0] // 2
        v[0, at, 5], v[0, at + 1, 6], v[0, at + 2, 7] = torch.inf, -torch.inf, torch.nan
        out = _run(c)
        n = counts[0] // 2
        assert out[:n].isfinite().all() and (out[n:, :, 5] == torch.inf).all()
        assert (out[n + 1:, :, 6] == -torch.inf).all() and out[n + 2:, :, 7].isnan().all()
        c.check(out)


@pytest.mark.parametrize("lens,counts", SHAPES + [([100] * 79 + [8000], [1] * 80)])
def test_in_the_bounds_checked_build(lens, counts):
    """Rows that are done over, in whole units, pieces and from the queue: nothing out of bounds, and the same bits."""
    from speculative_decode_verify_w4a16_gb300 import _lib, build

    c = Case(6, F16, 64, 8, 4, lens, counts, pad=1)
    c.q.zero_()
    c.q[::2, :, 0] = 32752.0
    for k, _ in c.kv:
        k[..., 0] = (k[..., 0].abs() * 2.0 ** 13).to(F16)
    want = _run(c, window=150)
    with _lib.use_library(build.build_bounds()):
        got = c.run(window=150)
        torch.cuda.synchronize()
        assert sv.check_device_status() == 0  # W4A16_ERR_BOUNDS would be 7
    n = sum(counts)  # (some keys are infinite: NaN to the rows that see them)
    torch.testing.assert_close(got[:n], want[:n], rtol=0, atol=0, equal_nan=True)
    c.check(want, 150)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("lens,counts", [([400], [40]), ([0], [300]), ([9000], [200])])
def test_scores_far_below_the_others(dtype, lens, counts):
    """Even rows see most keys 2^26 powers of two and more below the first ones: no weight, and nothing to be done over,
    whether the other rows' references rise with those keys or not."""
    c = Case(7, dtype, 128, 8, 4, lens, counts)
    even = torch.arange(c.T, device=dev()) % 2 == 0
    c.q[..., 0] = 0
    c.q[even, :, 0] = 32752.0 if dtype is F16 else 32768.0
    for k, _ in c.kv:
        k[..., 0] = 0
        k[:, 64:, 0] = -44704.0
    low = _run(c)
    c.check(low)
    c.q[~even, :, 0] = -2.0 ** -8
    raised = c.run()
    torch.cuda.synchronize()
    assert sv.check_device_status() == 0
    c.check(raised)
    assert torch.equal(raised[even], low[even])
