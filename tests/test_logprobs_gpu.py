"""GPU parity of token_logprobs against float64.

Tolerance: x - max and its product with log2 e are rounded once each (2^-24 of
a difference up to some 40, so an exponential is off by 40 * 2^-24 * 2 of
itself, and weighted with itself by far less), the sums of 32-bit terms by a
few 2^-24 per level of the tree, and the results (up to ~30) are stored in fp32:
4e-6 absolute + 2^-22 relative covers all of it with a factor of two."""
import numpy as np
import pytest
import torch

import speculative_decode_verify_w4a16_gb300 as sv
from helpers import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decode_verify_w4a16_gb300 import build
    build.build()


def _reference(x, ids, top):
    x = x.double().cpu()
    z = x - x.amax(1, keepdim=True)  # first: logits as low as -3e38 would swallow the sum's logarithm
    lp = z - z.exp().sum(1, keepdim=True).log()
    ent = -torch.special.xlogy(lp.exp(), lp.exp()).sum(1)
    pick = torch.where(ids >= 0, lp.gather(1, ids.clamp(min=0).long()), 0.0)
    order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :top]
    return pick, ent, order, lp.gather(1, order)


def _close(a, b):
    a, b = a.cpu().double(), b.double()
    same = (a == b) | (a.isnan() & b.isnan())
    return bool((same | ((a - b).abs() <= 4e-6 + 2.0 ** -22 * b.abs())).all())


def _check(x, ids, top):
    r = sv.token_logprobs(x.to(dev()), ids.to(dev()), top=top)
    torch.cuda.synchronize()
    assert sv.check_device_status() == 0
    pick, ent, order, tl = _reference(x, ids, top)
    assert _close(r.logp, pick) and _close(r.entropy, ent)
    assert torch.equal(r.top_ids.cpu().long(), order)
    assert _close(r.top_logp, tl)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,V,m,top", [
    (1, 1, 1, 1), (3, 2, 2, 2), (5, 33, 4, 33), (2, 64, 1, 64), (4, 255, 0, 1), (3, 1023, 1, 20), (3, 1024, 1, 20),
    (3, 1025, 3, 20), (7, 4099, 2, 32), (6, 50257, 1, 64), (16, 128256, 1, 5), (2, 300001, 64, 0), (1, 1 << 20, 1, 20),
])
def test_against_float64(dtype, R, V, m, top):
    g = torch.Generator().manual_seed(R * 31 + V)
    x = (torch.randn(R, V, generator=g) * 3).to(dtype)
    ids = torch.randint(0, V, (R, m), generator=g, dtype=torch.int32)
    if m > 2:
        ids[:, 1] = -1
    _check(x, ids, top)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ties_go_to_the_lower_index(dtype):
    g = torch.Generator().manual_seed(3)
    few = torch.randint(-2, 3, (4, 9001), generator=g).to(dtype)  # thousands of equal logits
    _check(few, torch.zeros(4, 1, dtype=torch.int32), 40)
    flat = torch.full((2, 70000), -1.5).to(dtype)
    flat[1, 60000:60003] = 2.0
    _check(flat, torch.zeros(2, 1, dtype=torch.int32), 64)
    zeros = torch.zeros(1, 5000)
    zeros[0, ::2] = -0.0  # the two zeros are equal
    _check(zeros.to(dtype), torch.zeros(1, 1, dtype=torch.int32), 10)


def test_masked_tokens():
    g = torch.Generator().manual_seed(4)
    x = torch.randn(6, 5003, generator=g) * 4
    x[0, torch.rand(5003, generator=g) < 0.9] = -torch.inf
    x[1, :] = -torch.inf
    x[1, 4999] = 3.0                                 # one token left
    x[2, :2048] = -torch.inf                         # whole windows
    x[3, 1:] = torch.finfo(torch.float32).min        # the type's lowest value as a mask
    x[4, :] = torch.finfo(torch.float32).min         # ... everywhere: uniform
    x[5, 7] = 1e30
    _check(x, torch.tensor([[0, 1], [4999, 0], [5, 3000], [0, 1], [2, 3], [7, 8]], dtype=torch.int32), 20)


def _extremes():
    """Rows whose maximum is far from zero, in every window or in some."""
    f32 = np.float32
    rows = [torch.full((5003,), v) for v in (-1e4, -1e9, -1e10, -1e20, 1e10, 5e29, 2e38, -2.0 ** 20, 2.0 ** 20 - 1)]
    for top in (f32(2.0 ** 20), f32(1e9), f32(1.9000001e30)):  # neighbours, in windows of their own
        r = torch.full((5003,), -1e9)
        r[4000], r[10], r[2500] = float(np.nextafter(top, f32(3e38))), float(top), float(np.nextafter(top, f32(0)))
        rows.append(r)
    r = torch.full((5003,), -2.0 ** 21)  # windows far away from a maximum that is near
    r[17] = 3.0
    rows.append(r)
    r = torch.full((5003,), -torch.inf)
    r[3000:] = 1048575.9375
    r[2] = 1048576.0
    rows.append(r)
    return torch.stack(rows)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows", [1, 50])  # 700 of them: more than a few an SM
def test_maxima_far_from_zero(dtype, rows):
    x = _extremes().repeat(rows, 1).to(dtype)
    ids = torch.tensor([[10, 4000, 2500, 2, 17]], dtype=torch.int32).repeat(x.shape[0], 1)
    _check(x, ids, 3)


@pytest.mark.parametrize("R", [3, 640])
@pytest.mark.parametrize("V,top", [(257, 5), (300, 64), (1000, 32), (1023, 1), (2000, 20), (8000, 33)])
def test_short_rows(R, V, top):
    """Fewer quarters than alternatives, or not many more: other ways to the candidates."""
    g = torch.Generator().manual_seed(V)
    x = torch.randn(R, V, generator=g) * 3
    x[1::3] = torch.randint(-4, 5, x[1::3].shape, generator=g).float()
    x[2::3, V // 3:] = -torch.inf
    _check(x, torch.randint(0, V // 3, (R, 1), generator=g, dtype=torch.int32), top)


def test_many_rows_with_masks_and_ties():
    g = torch.Generator().manual_seed(8)
    x = torch.randint(-3, 4, (640, 4099), generator=g).float()
    x[::3, 2000:] = -torch.inf
    x[1::3, :4000] = torch.finfo(torch.float32).min
    x[2::6] = torch.randn(x[2::6].shape, generator=g) * 4
    ids = torch.randint(-1, 4099, (640, 2), generator=g, dtype=torch.int32)
    _check(x, ids, 33)


def test_rows_without_a_distribution_are_nan():
    x = torch.randn(4, 3000)
    x[0, :] = -torch.inf
    x[1, 17] = torch.nan
    x[2, 2999] = torch.inf
    r = sv.token_logprobs(x.to(dev()), torch.zeros(4, 1, dtype=torch.int32, device=dev()), top=3)
    torch.cuda.synchronize()
    assert r.logp[:3].isnan().all() and r.entropy[:3].isnan().all() and r.top_logp[:3].isnan().all()
    assert r.logp[3].isfinite().all() and r.entropy[3].isfinite()
    assert r.top_ids[0].tolist() == [0, 1, 2]
    assert r.top_ids[1, 0] == 17 and r.top_ids[2, 0] == 2999
    assert sv.check_device_status() == 0


def test_bad_ids_are_reported():
    x = torch.randn(2, 100, device=dev())
    r = sv.token_logprobs(x, torch.tensor([[3, 100], [-2, -1]], dtype=torch.int32, device=dev()))
    torch.cuda.synchronize()
    assert sv.check_device_status() == 5
    assert r.logp[0, 1].isnan() and r.logp[1, 0].isnan() and r.logp[1, 1] == 0 and r.logp[0, 0].isfinite()


def test_rows_of_the_accept_step():
    """Beside the accept step: [B, n + 1, V] logits flattened, ids of one token a row, another stream."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn(16 * 5, 128256, generator=g) * 3
    ids = torch.randint(0, 128256, (80,), generator=g, dtype=torch.int32)
    dx, di = x.to(dev()), ids.to(dev())
    first = sv.token_logprobs(dx, di, top=5)
    s = torch.cuda.Stream()
    ws = torch.empty(sv.token_logprobs_workspace_bytes(80, 128256, 5), dtype=torch.uint8, device=dev())
    torch.cuda.synchronize()
    again = sv.token_logprobs(dx, di, top=5, ws=ws, stream=s)
    s.synchronize()
    assert first.logp.shape == (80,)
    for a, b in ((first.logp, again.logp), (first.entropy, again.entropy), (first.top_ids, again.top_ids),
                 (first.top_logp, again.top_logp)):
        assert torch.equal(a, b)
    pick, ent, order, tl = _reference(x, ids[:, None], 5)
    assert _close(first.logp, pick[:, 0]) and _close(first.entropy, ent)
    assert torch.equal(first.top_ids.cpu().long(), order) and _close(first.top_logp, tl)
