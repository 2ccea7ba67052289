"""Rows of a step that lie outside it: the append and the attention report the same
inputs, whether a row of the step leads to the bad request or not, and leave out
the bad requests alone."""
import numpy as np
import pytest
import torch

import kv16_reference as ref
import speculative_decode_verify_w4a16_gb300 as sv
from helpers import dev
from test_kv16_gpu import _i32, _randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decode_verify_w4a16_gb300 import build
    build.build()


@pytest.mark.parametrize("starts,served,status", [
    ([0, 5, 12], [0, 1], 0), ([0, 0, 12], [1], 0), ([3, 3, 9], [1], 0), ([12, 12, 12], [], 0),
    # no row of 0 .. 11 lies in the bad request
    ([0, 12, 17], [0], 5), ([-2, 0, 12], [1], 5), ([0, 12, 11], [0], 5), ([12, 12, 13], [], 5), ([-1, 0, 0], [], 5),
    ([-2 ** 31, 0, 12], [1], 5), ([0, 12, 2 ** 31 - 1], [0], 5),
    # some do
    ([-2, 6, 12], [1], 5), ([0, 6, 13], [0], 5),
])
@pytest.mark.parametrize("rotated", [False, True])
def test_rows_outside_are_reported(starts, served, status, rotated):
    rng = np.random.default_rng(1)
    T, Hkv, D, lens = 12, 2, 64, [60, 130]
    table, pages = ref.paged(rng, lens, [T, T])
    cache = sv.kv16_cache(1, pages, Hkv, D)
    for x in (cache.k, cache.v):
        x.fill_(3.0)
    k, v, q = (_randn(rng, T, h, D) for h in (Hkv, Hkv, 4))
    out = torch.full_like(q, 7.0)
    freqs = sv.rope_frequencies(D) if rotated else None
    sv.kv16_append(cache, 0, k, v, table.to(dev()), _i32(lens), row_start=_i32(starts), rope=freqs, q=q, q_out=out)
    assert sv.check_device_status() == status
    taken, places = torch.zeros(T, dtype=torch.bool), 0
    for b in served:
        n = starts[b + 1] - starts[b]
        taken[starts[b]:starts[b + 1]] = True
        places += n
        assert torch.equal(ref.rows_of(table, b, cache.v[0], lens[b], lens[b] + n).transpose(0, 1), v[starts[b]:starts[b + 1]])
    assert int((cache.v[0] != 3).any(-1).any(1).sum()) == places and int((cache.k[0] != 3).any(-1).any(1).sum()) == places
    assert torch.equal((out != 7).any(-1).any(-1).cpu(), taken)
    # the attention reports what the append reports
    o = torch.full_like(q, 7.0)
    sv.kv16_attention(q, cache, 0, table.to(dev()), _i32(lens), row_start=_i32(starts), out=o)
    assert sv.check_device_status() == status
    assert torch.equal((o != 7).any(-1).any(-1).cpu(), taken)
