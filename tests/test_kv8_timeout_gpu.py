"""The 8-bit attention's bounded waits, made to run out: the kernel reports
W4A16_ERR_DEVICE_TIMEOUT, returns, and leaves the device usable.

In the debug build of the library (its waits give up after 5 ms) a test hook
makes the producer of the first CTA leave out one tile's keys. The MMA warps'
wait for them runs out, then the softmax warps', the producer's for the next
free stage and the widening warps': all of them go through the rest of their
work in bounds."""
import ctypes

import numpy as np
import pytest
import torch

import kv8_reference as ref
import speculative_decode_verify_w4a16_gb300 as sv
from helpers import dev
from test_kv8_gpu import E4M3, E5M2, _attn_inputs, _check, _history

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hook():
    from speculative_decode_verify_w4a16_gb300 import _lib, build

    build.build()
    with _lib.use_library(build.build_debug()) as L:
        f = L.w4a16_test_set_skip_tile
        f.argtypes, f.restype = [ctypes.c_int], ctypes.c_int
        yield f


@pytest.mark.parametrize("dtype,n,H,Hkv,skip", [(E4M3, 1, 2, 1, 3), (E5M2, 16, 4, 2, 0), (E4M3, 9, 5, 1, 7), (E4M3, 8, 8, 1, 5)])
def test_a_wait_that_runs_out(hook, dtype, n, H, Hkv, skip):
    rng = np.random.default_rng(skip)
    B, L = 4, 128 * 400 // Hkv  # some ten tiles a run
    hist = [_history(rng, Hkv, 700)] * B
    cache = ref.Cache(hist, dtype, rng, 700)
    c, table, lens, tails = cache.to(sv, dev())
    full = 700 // 64
    table = table[:, :full].repeat(1, L // (64 * full) + 1)  # the same pages over and over: a long request
    long = torch.full_like(lens, full * 64 * (L // (64 * full)) + 700 % 64)
    qkv, cols = _attn_inputs(rng, B, n, H, Hkv)
    dq = [qkv.to(dev())[:, :, s].unflatten(2, (-1, 128)) for s in cols]
    ws = torch.zeros(sv.kv8_tree_attention_workspace_bytes(B, n, H, Hkv, 128, L + 64), dtype=torch.uint8, device=dev())

    def run(lens, **kw):
        out = sv.kv8_tree_attention(*dq, c, 0, table, lens, tails, ws=ws, **kw)
        torch.cuda.synchronize()
        return out.cpu(), sv.check_device_status()

    good, status = run(long)
    assert status == 0 and torch.isfinite(good).all()
    assert hook(skip) == 0  # the first CTA leaves out that tile's keys
    try:
        bad, status = run(long)
        assert status == 4  # W4A16_ERR_DEVICE_TIMEOUT
        assert sv.check_device_status() == 0  # the read cleared it
        assert torch.equal(bad[1:], good[1:])  # the first CTA has tiles of request 0 alone
    finally:
        assert hook(-1) == 0
    # the context is usable, and the counters are where they were
    out, status = run(long)
    assert status == 0 and torch.equal(out, good)
    out, status = run(lens)
    assert status == 0
    q, k, v = (qkv[:, :, s].unflatten(2, (-1, 128)) for s in cols)
    _check(out.double(), cache, (q, k, v), [ref.chain(n)] * B, "after the timeout")
