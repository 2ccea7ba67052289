"""Batches of many short requests and a few long ones: right wherever the long ones
stand, and a unit far longer than the others is not left whole for the end."""
import numpy as np
import pytest
import torch

import speculative_decode_verify_w4a16_gb300 as sv
from helpers import dev
from test_kv16_gpu import BF16, F16, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decode_verify_w4a16_gb300 import build
    build.build()


def _pieces(c, **kw):
    """Whether a call stored pieces of a unit: what lies in its workspace behind the counters, zero before."""
    ws = torch.zeros(sv.kv16_attention_workspace_bytes(c.T, c.H, c.Hkv, c.D), dtype=torch.uint8, device=dev())
    out = c.run(ws=ws, **kw)
    ctas = torch.cuda.get_device_properties(0).multi_processor_count
    assert sv.check_device_status() == 0
    assert not ws[:4 * (ctas + 2)].any()
    return out, bool(ws[-(-4 * (ctas + 2) // 256) * 256:].any())


@pytest.mark.parametrize("short,many,long,whole", [(100, 79, 100, True), (100, 79, 8000, False), (500, 100, 8000, False),
                                                   (100, 200, 16000, False), (1000, 100, 1000, True)])
@pytest.mark.parametrize("at", ["first", "middle", "last"])
def test_a_long_request_among_short_ones_is_cut(short, many, long, whole, at):
    """One row and 8 heads of their own a request. A unit of 2 or 8 tiles weighs some 12 or 18 with its start and end, one of
    126 tiles ten or seven times as much; with 251 there are too many tiles for any batch."""
    i = {"first": 0, "middle": many // 2, "last": many}[at]
    lens = [short] * many
    lens.insert(i, long)
    c = Case(1, BF16, 128, 8, 8, lens, [1] * (many + 1))
    out, cut = _pieces(c)
    assert cut == (not whole)
    c.check(out, requests=[0, 1, i, many - 1, many])


@pytest.mark.parametrize("dtype,D,H,Hkv", [(BF16, 128, 16, 8), (F16, 64, 24, 8)])
@pytest.mark.parametrize("lens,counts", [
    ([60] * 79 + [1000], [1] * 80), ([1000] + [60] * 79, [1] * 80), ([60] * 40 + [900] + [60] * 300, [1] * 341),
    ([0] * 41, [100] * 40 + [2000]), ([0] * 41, [2000] + [100] * 40), ([0, 5] * 45, [0, 40] * 44 + [0, 1200]),
    ([30] * 383 + [700], [1] * 384), ([30] * 384 + [700], [1] * 385), ([30, 0] * 500 + [700], [1, 0] * 500 + [1]),
])
def test_units_far_longer_than_the_others(dtype, D, H, Hkv, lens, counts):
    """Whole or cut, wherever they stand: every row once, the same bits in every call."""
    c = Case(2, dtype, D, H, Hkv, lens, counts, pad=2)
    first = None
    for _ in range(4):
        out = torch.full((c.T, H, D), 7.0, dtype=dtype, device=dev())
        c.run(out=out)
        first = out if first is None else first
        assert torch.equal(out, first)
    assert sv.check_device_status() == 0
    assert (first[sum(counts):] == 7).all()
    n = len(lens)
    c.check(first, requests=sorted({*range(0, n, max(1, n // 40)), n // 2, n - 2, n - 1}))


def test_any_order_of_the_requests():
    """The same requests in other orders: their rows do not change where no unit is cut."""
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(0, 300, 90)] + [900, 1000]
    c = Case(4, BF16, 128, 8, 8, lens, [1] * 92)
    out, cut = _pieces(c)
    assert not cut
    tensors = c.table, c.q
    for _ in range(4):
        p = torch.from_numpy(rng.permutation(92))
        c.table, c.q, c.lens = tensors[0][p], tensors[1][p.to(dev())].contiguous(), [lens[i] for i in p.tolist()]
        again, cut = _pieces(c)
        assert not cut and torch.equal(again, out[p.to(dev())])
