"""The paged 16-bit attention's bounded waits are for what has stopped: a warp that
has nothing to do for longer than the limit, while its CTA works on, waits on.

In the debug build of the library (its limit is 5 ms) every CTA has a unit of some
ten thousand tiles, which take more: the guard waits for the last of them."""
import pytest
import torch

import speculative_decode_verify_w4a16_gb300 as sv
from helpers import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,D,window", [(torch.bfloat16, 128, 0), (torch.float16, 64, 0), (torch.float16, 64, 1 << 19)])
def test_units_that_take_longer_than_the_limit(dtype, D, window):
    from speculative_decode_verify_w4a16_gb300 import _lib, build

    build.build()
    g = torch.Generator(device=dev())
    g.manual_seed(1)
    n, past, pages = 160 * 256, 900_000, 11
    blocks = (past + n + 63) // 64
    cache = sv.KV16Cache(*(torch.randn(1, pages, 1, 64, D, generator=g, device=dev()).to(dtype) for _ in range(2)))
    q = torch.randn(n, 1, D, generator=g, device=dev()).to(dtype)
    table = (torch.arange(blocks, dtype=torch.int32, device=dev()) % pages).view(1, -1)  # the same pages over and over
    lens = torch.tensor([past], dtype=torch.int32, device=dev())
    want = sv.kv16_attention(q, cache, 0, table, lens, window=window)
    assert sv.check_device_status() == 0
    ws = torch.zeros(sv.kv16_attention_workspace_bytes(n, 1, 1, D), dtype=torch.uint8, device=dev())
    with _lib.use_library(build.build_debug()):
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        got = sv.kv16_attention(q, cache, 0, table, lens, window=window, ws=ws)
        end.record()
        torch.cuda.synchronize()
        assert sv.check_device_status() == 0
    assert start.elapsed_time(end) > 5  # (else this test shows nothing)
    assert torch.equal(got, want) and torch.isfinite(want).all()
