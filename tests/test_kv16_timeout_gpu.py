"""The paged 16-bit attention's bounded waits, made to run out: the kernel
reports W4A16_ERR_DEVICE_TIMEOUT, returns, and leaves the device usable.

In the debug build of the library (its waits give up after 5 ms) a test hook
makes the producer of the first CTA leave out one copy of its run: a tile's keys
(even numbers) or values (odd ones). The MMA warps' wait for it runs out, then
the softmax warps', the guard's, and the producer's for the next free buffer: all
of them leave in bounds, the copies in flight awaited."""
import ctypes

import pytest
import torch

import kv16_reference as ref
import speculative_decode_verify_w4a16_gb300 as sv
from helpers import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hook():
    from speculative_decode_verify_w4a16_gb300 import _lib, build

    build.build()
    with _lib.use_library(build.build_debug()) as L:
        f = L.w4a16_test_set_skip_copy
        f.argtypes, f.restype = [ctypes.c_int], ctypes.c_int
        yield f


@pytest.mark.parametrize("dtype,D", [(torch.bfloat16, 128), (torch.float16, 64)])
@pytest.mark.parametrize("n,H,Hkv,first,skip", [
    (1, 2, 1, 51200, 0), (1, 2, 1, 51200, 7), (5, 8, 1, 51200, 12),  # one row tile, cut units
    (40, 8, 1, 51200, 6), (40, 8, 1, 51200, 33),                     # two row tiles
    (5, 4, 1, 30, 1), (5, 4, 1, 130, 4), (40, 8, 1, 100, 3),         # a short request first: guarded values, its last keys
])
def test_a_wait_that_runs_out(hook, dtype, D, n, H, Hkv, first, skip):
    g = torch.Generator(device=dev())
    g.manual_seed(skip)
    B, pages = 4, 13
    cache = sv.KV16Cache(*(torch.randn(1, pages, Hkv, 64, D, generator=g, device=dev()).to(dtype) for _ in range(2)))
    q = torch.randn(B, n, H, D, generator=g, device=dev()).to(dtype)
    lens = torch.tensor([first, 51200, 51200, 51200], dtype=torch.int32, device=dev())
    table = (torch.arange(B * 802, dtype=torch.int32, device=dev()) % pages).view(B, 802)  # the same pages over and over
    ws = torch.zeros(sv.kv16_attention_workspace_bytes(B * n, H, Hkv, D), dtype=torch.uint8, device=dev())

    def run():
        out = sv.kv16_attention(q, cache, 0, table, lens, ws=ws)
        torch.cuda.synchronize()
        return out.cpu(), sv.check_device_status()

    good, status = run()
    assert status == 0 and torch.isfinite(good).all()
    assert hook(skip) == 0
    try:
        bad, status = run()
        assert status == 4  # W4A16_ERR_DEVICE_TIMEOUT
        assert sv.check_device_status() == 0  # the read cleared it
        assert torch.equal(bad[2:], good[2:])  # the first CTA has tiles of the first requests alone
    finally:
        assert hook(-1) == 0
    ws.zero_()  # (a cut unit's count may be left in it)
    out, status = run()
    assert status == 0 and torch.equal(out, good)
    k, v = (x[0][table[0, :(first + n + 63) // 64].long()].transpose(0, 1).flatten(1, 2)[:, :first + n]
            for x in (cache.k, cache.v))
    want, mag = ref.attention(q[0], k, v, first)
    assert ((out[0].to(dev()).double() - want).abs() <= ref.attention_bound(want, mag, v, dtype)).all()


def test_default_workspaces_are_renewed(hook):
    """The same without a workspace of one's own: after the report the next calls give what the first one gave."""
    g = torch.Generator(device=dev())
    g.manual_seed(1)
    cache = sv.KV16Cache(*(torch.randn(1, 9, 1, 64, 128, generator=g, device=dev()).bfloat16() for _ in range(2)))
    q = torch.randn(1, 3, 4, 128, generator=g, device=dev()).bfloat16()
    lens = torch.tensor([60000], dtype=torch.int32, device=dev())
    table = (torch.arange(940, dtype=torch.int32, device=dev()) % 9).view(1, 940)
    good = sv.kv16_attention(q, cache, 0, table, lens)
    assert sv.check_device_status() == 0
    assert hook(2) == 0
    try:
        sv.kv16_attention(q, cache, 0, table, lens)
        assert sv.check_device_status() == 4
    finally:
        assert hook(-1) == 0
    for _ in range(2):
        assert torch.equal(sv.kv16_attention(q, cache, 0, table, lens), good)
    assert sv.check_device_status() == 0
