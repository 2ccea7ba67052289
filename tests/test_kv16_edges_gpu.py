"""Calls at the edge of what the paged 16-bit cache's and the rotation's contracts
allow: an out on 16 bytes, windows past every position, shared prefixes, calls
right after those whose results they read, in a graph too, two graphs at once."""
import numpy as np
import pytest
import torch

import kv16_reference as ref
import speculative_decode_verify_w4a16_gb300 as sv
from helpers import dev
from test_kv16_gpu import BF16, F16, Case, _i32, _randn, _starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decode_verify_w4a16_gb300 import build
    build.build()


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F16, 64)])
@pytest.mark.parametrize("at", [8, 16])
@pytest.mark.parametrize("lens,counts", [([0, 700], [130, 3]), ([20000], [4]), ([9000], [300])])
def test_an_out_on_sixteen_bytes(dtype, D, at, lens, counts):
    c = Case(at, dtype, D, 8, 2, lens, counts, pad=1)
    n = c.T * 8 * D
    space = torch.full((n + 32,), 7.0, dtype=dtype, device=dev())
    out = space[at:at + n].view(c.T, 8, D)
    c.run(out=out)
    assert sv.check_device_status() == 0
    c.check(out)
    assert (space[:at] == 7).all() and (space[at + n - 8 * D:] == 7).all()


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 64, 1 << 20])
def test_a_window_past_every_position_is_none(window):
    c = Case(3, BF16, 128, 8, 2, [0, 5000, 100], [300, 1, 17])
    assert torch.equal(c.run(window=window), c.run())
    c.check(c.run(window=window), window=window)


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F16, 64)])
def test_requests_that_share_a_prefix(dtype, D):
    """Three requests over the same first pages: each as if it had copies of its own."""
    c = Case(5, dtype, D, 8, 2, [640, 640, 640], [1, 65, 300])
    for b in (1, 2):
        for x, mine, first in zip((c.cache.k, c.cache.v), c.kv[b], c.kv[0]):
            mine[:, :640] = first[:, :640]
        c.put(b)
    own = c.run()
    c.table[1:, :10] = c.table[0, :10]
    assert torch.equal(c.run(), own)
    c.check(own)


def test_one_request_twice():
    """The same request's row in two places of the batch: two rows for one place of a page, the same one."""
    rng = np.random.default_rng(1)
    cache = sv.kv16_cache(1, 4, 2)
    k, v = (_randn(rng, 1, 2, 128).expand(2, -1, -1).contiguous() for _ in range(2))
    q = _randn(rng, 1, 8, 128).expand(2, -1, -1).contiguous()
    table, lens = _i32([[2, 3], [2, 3]]), _i32([70, 70])
    q = sv.kv16_append(cache, 0, k, v, table, lens, rope=sv.rope_frequencies(128), q=q)
    out = sv.kv16_attention(q, cache, 0, table, lens)
    assert torch.equal(out[0], out[1]) and torch.equal(q[0], q[1]) and torch.equal(cache.v[0, 3, :, 6], v[0])
    assert sv.check_device_status() == 0


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_each_call_reads_what_the_one_before_wrote(dtype):
    """Rotation, append and attention of twelve layers, each fed by the layer before, back to back and in a graph:
    as with a synchronisation behind each."""
    rng = np.random.default_rng(2)
    layers, H, Hkv, D = 12, 8, 2, 128
    f = sv.rope_frequencies(D)
    lens, counts = [63, 1000, 0, 7], [3, 1, 150, 0]
    table, pages = ref.paged(rng, lens, counts)
    table, lens, start = table.to(dev()), _i32(lens), _i32(_starts(counts))
    filled = [_randn(rng, layers, pages, Hkv, 64, D, dtype=dtype) for _ in range(2)]
    first = _randn(rng, sum(counts), H + 2 * Hkv, D, dtype=dtype)

    def step(cache, sync=lambda: None):
        x = first
        for i in range(layers):
            q, k, v = x.split((H, Hkv, Hkv), 1)
            q = sv.kv16_append(cache, i, k, v, table, lens, row_start=start, rope=f, q=q)
            sync()
            o = sv.kv16_attention(q, cache, i, table, lens, row_start=start)
            sync()
            x = torch.cat([o, k, v], 1)
            sync()
        return o

    cache = sv.KV16Cache(*(x.clone() for x in filled))
    want = step(cache, torch.cuda.synchronize).clone()
    assert torch.isfinite(want).all()
    again = sv.KV16Cache(*(x.clone() for x in filled))
    got = step(again)
    assert torch.equal(got, want) and torch.equal(again.k, cache.k) and torch.equal(again.v, cache.v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(again)
    for _ in range(5):
        for x, y in zip((again.k, again.v), filled):
            x.copy_(y)
        graph.replay()
        assert torch.equal(got, want) and torch.equal(again.k, cache.k)
    assert sv.check_device_status() == 0


def test_two_graphs_at_once():
    """Graphs captured apart share no workspace: replayed on two streams at the same time, each gives its own."""
    cases = [Case(s, BF16, 128, 16, 2, [30000, 77], [4, 1]) for s in (1, 2)]
    want = [c.run().clone() for c in cases]
    graphs, outs = [], []
    for c in cases:
        tensors = c.table.to(dev()), _i32(c.lens), _i32(_starts(c.counts))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(sv.kv16_attention(c.q, c.cache, c.layer, tensors[0], tensors[1], row_start=tensors[2]))
        graphs.append((g, tensors))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (g, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert sv.check_device_status() == 0
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


@pytest.mark.parametrize("dtype", [BF16, F16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rows_of_every_width(dtype, interleaved):
    """Heads from the narrowest to the widest, and items that do not divide by the threads."""
    rng = np.random.default_rng(4)
    for heads, D, rot in ((1, 16, 16), (1, 24, 16), (37, 40, 32), (5, 1024, 1024), (3, 1000, 16), (129, 64, 64)):
        f = sv.rope_frequencies(rot, interleaved=interleaved)
        x = _randn(rng, 3, heads, D, dtype=dtype)
        positions = [0, 2 ** 31 - 1, -2 ** 31]
        got = sv.rope(x, _i32(positions), f)
        cos, sin = ref.cos_sin(positions, sv.rope_angles(rot)[0])
        want, mag = ref.rotate(x, cos, sin, interleaved)
        assert ((got.double() - want).abs() <= ref.rotation_bound(want, mag, dtype)).all(), (heads, D, rot)
    assert sv.check_device_status() == 0


@pytest.mark.parametrize("dtype,D,H,Hkv", [(BF16, 128, 16, 8), (F16, 64, 24, 8)])
@pytest.mark.parametrize("lens,counts,window", [
    ([int(x) for x in np.random.default_rng(5).integers(0, 1900, 60)], [1 + b % 5 * (b % 2) for b in range(60)], 0),
    ([0] * 12, [900, 0, 1, 64, 65, 300, 1500, 2, 128, 129, 700, 33], 0),
    ([int(x) for x in np.random.default_rng(6).integers(0, 5000, 40)], [b * 13 % 700 for b in range(40)], 500),
    ([5] * 300, [b % 3 for b in range(300)], 0),
])
def test_many_short_units(dtype, D, H, Hkv, lens, counts, window):
    """More units than CTAs several times over: taken whole, from a queue that every call leaves as it was."""
    c = Case(8, dtype, D, H, Hkv, lens, counts, pad=2)
    ws = torch.zeros(sv.kv16_attention_workspace_bytes(c.T, H, Hkv, D), dtype=torch.uint8, device=dev())
    first = None
    for _ in range(4):
        out = torch.full((c.T, H, D), 7.0, dtype=dtype, device=dev())
        c.run(out=out, window=window, ws=ws)
        first = out if first is None else first
        assert torch.equal(out, first)  # whichever CTA has a unit
    assert sv.check_device_status() == 0
    assert (first[sum(counts):] == 7).all()
    c.check(first, window=window, requests=[b for b in range(len(lens)) if counts[b]][::3])
    # a request alone, cut or not, is the same within the bound: and a batch of them is again whole afterwards
    alone = Case(9, dtype, D, H, Hkv, [3000], [2])
    alone.check(alone.run(ws=ws))
    assert torch.equal(c.run(window=window, ws=ws)[:sum(counts)], first[:sum(counts)])


def test_many_short_units_with_bad_requests():
    """Requests that are left out, and pages that are none, among many: the others are served."""
    lens, counts = [100 + b for b in range(80)], [1 + b % 4 for b in range(80)]
    c = Case(10, BF16, 128, 8, 8, lens, counts)
    good = c.run()
    assert sv.check_device_status() == 0
    bad = list(lens)
    bad[7], bad[40] = -1, 1 << 20
    table = c.table.clone()
    table[79, 0] = 1 << 20
    out = sv.kv16_attention(c.q, c.cache, c.layer, table.to(dev()), _i32(bad), row_start=_i32(_starts(counts)))
    torch.cuda.synchronize()
    assert sv.check_device_status() == 5  # W4A16_ERR_DEVICE_INPUT
    at = _starts(counts)
    for b in range(79):
        if b not in (7, 40):
            assert torch.equal(out[at[b]:at[b + 1]], good[at[b]:at[b + 1]]), b
    assert torch.equal(c.run(), good)
    assert sv.check_device_status() == 0


@pytest.mark.parametrize("lens,counts", [([0, 700, 90], [300, 3, 70]), ([20000], [40]), ([9000], [300]),
                                         ([50 + b for b in range(80)], [1 + b % 4 for b in range(80)])])
def test_out_in_place_of_the_queries(lens, counts):
    """Whole units, cut ones and the queue's."""
    c = Case(11, BF16, 128, 16, 8, lens, counts)
    want, before = c.run(), c.q.clone()
    assert c.run(out=c.q) is c.q
    assert sv.check_device_status() == 0
    assert torch.equal(c.q, want)
    c.q = before
    c.check(want)


def test_queries_that_are_not_finite_stay_with_their_rows():
    c = Case(12, BF16, 128, 8, 2, [300, 2000], [130, 5])
    want = c.run().clone()
    for row, head, x in ((0, 0, torch.nan), (77, 3, torch.inf), (131, 7, -torch.inf), (134, 1, torch.nan)):
        c.q[row, head, 5] = x
    got = c.run()
    hit = torch.zeros(c.T, 8, dtype=torch.bool, device=dev())
    for row, head in ((0, 0), (77, 3), (131, 7), (134, 1)):
        hit[row, head] = True
    assert torch.equal(got[~hit], want[~hit])
    assert not got[hit].isfinite().any()
    assert sv.check_device_status() == 0


def test_as_many_requests_as_are_taken():
    """4096 requests (a CTA looks through them 32 at a time), some without rows."""
    rng = np.random.default_rng(13)
    lens = [int(x) for x in rng.integers(0, 130, 4096)]
    counts = [int(x) for x in rng.integers(0, 3, 4096)]
    c = Case(13, BF16, 128, 4, 1, lens, counts, pad=5)
    out = torch.full((c.T, 4, 128), 7.0, dtype=BF16, device=dev())
    c.run(out=out)
    assert sv.check_device_status() == 0
    assert (out[sum(counts):] == 7).all()
    c.check(out, requests=[*range(0, 4096, 61), 4094, 4095])


@pytest.mark.parametrize("lens,counts,window", [([50 + 7 * b for b in range(90)], [1 + b % 4 for b in range(90)], 0),
                                                ([0] * 9, [700, 3, 128, 129, 0, 65, 300, 900, 1], 200),
                                                ([1003], [1], 0), ([1000], [300], 0), ([40000, 3], [70, 1], 0)])
def test_in_the_bounds_checked_build(lens, counts, window):
    """The queue, whole units, pieces and their merges: nothing out of bounds, and the same bits."""
    from speculative_decode_verify_w4a16_gb300 import _lib, build

    c = Case(14, BF16, 128, 16, 8, lens, counts, pad=1)
    want = c.run(window=window)
    with _lib.use_library(build.build_bounds()):
        got = c.run(window=window)
        torch.cuda.synchronize()
        assert sv.check_device_status() == 0  # W4A16_ERR_BOUNDS would be 7
    n = sum(counts)
    assert torch.equal(got[:n], want[:n])
    c.check(want, window=window)
