"""Edges of the paged 8-bit cache operators."""
import numpy as np
import pytest
import torch

import kv8_reference as ref
import speculative_decode_verify_w4a16_gb300 as sv
from helpers import dev
from test_kv8_gpu import E4M3, _attn_inputs, _history, _i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decode_verify_w4a16_gb300 import build
    build.build()


def test_a_negative_table_entry_is_a_bad_page():
    """Whatever its value: it is reported and reads as zeros."""
    rng = np.random.default_rng(1)
    B, n, H, Hkv, D = 3, 3, 8, 2, 128
    cache = ref.Cache([_history(rng, Hkv, L) for L in (130, 300, 70)], E4M3, rng, 320)
    c, table, lens, tails = cache.to(sv, dev())
    qkv, cols = _attn_inputs(rng, B, n, H, Hkv)
    dq = [qkv.to(dev())[:, :, s].unflatten(2, (-1, D)) for s in cols]

    def run(value=None):
        t = table.clone()
        if value is not None:
            t[1, 2] = value
        out = sv.kv8_tree_attention(*dq, c, 0, t, lens, tails, max_len=320)
        torch.cuda.synchronize()
        return out.cpu(), sv.check_device_status()

    good, status = run()
    assert status == 0
    zeros = cache.values[1]
    for x in zeros:
        x[:, 128:192] = 0.0
    q, k, v = (qkv[:, :, s].unflatten(2, (-1, D)) for s in cols)
    want, mag = ref.attention(zeros, q[1], k[1], v[1], ref.chain(n))
    for value in (-1, -2, -3, -(2 ** 31)):
        out, status = run(value)
        assert status == 5 and torch.equal(out[0], good[0]) and torch.equal(out[2], good[2]), value
        # test_kv8_gpu's bound
        assert ((out[1].double() - want).abs() <= 1.05 * 2.0 ** -8 * (mag + want.abs()) + 1e-6).all(), value


@pytest.mark.parametrize("layers", [1, 3])
def test_a_step_of_no_rows(layers):
    """The plan allows it (all requests ended, or none brought a row); the append
    has nothing to do, and refuses what it always refuses."""
    B, Hkv, D = 3, 2, 128
    cache = sv.kv8_cache(layers, 4, B, Hkv, device=dev())
    tails = _i32(2 * np.arange(B))
    plan = sv.kv_block_plan(_i32([5, 64, 0]), tails, _i32([[-1], [0], [-1]]), _i32([1, 2, 3, 0]), _i32([0, 3, 0]),
                            row_start=_i32(np.zeros(B + 1)), rows=0, release=_i32([0, 1, 0]))
    assert plan.new_lens.tolist() == [5, 0, 0] and plan.queue.tolist() == [0, 4, 0]
    none = torch.empty(layers, 0, Hkv, D, dtype=torch.bfloat16, device=dev())
    before = [x.view(torch.uint8).clone() for x in (cache.k, cache.v, cache.k_tail, cache.v_tail)]
    sv.kv8_append(cache, none, none, tails, plan)
    keep = torch.zeros(0, dtype=torch.int64, device=dev())
    some = torch.ones(layers, 7, Hkv, D, dtype=torch.bfloat16, device=dev())
    sv.kv8_append(cache, some[:, keep], some[:, :0], tails, plan)
    if layers == 1:
        sv.kv8_append(cache, none[0], none[0], tails, plan)
    torch.cuda.synchronize()
    assert sv.check_device_status() == 0
    for x, y in zip((cache.k, cache.v, cache.k_tail, cache.v_tail), before):
        assert torch.equal(x.view(torch.uint8), y)
    for bad in (none.float(), none.cpu(), none[:, :, :1], none.transpose(2, 3)):
        with pytest.raises(ValueError):
            sv.kv8_append(cache, bad, bad, tails, plan)


@pytest.mark.parametrize("layers,rows,Hkv", [(1, 70, 2), (1, 70, 1), (2, 70, 1), (2, 1, 2), (1, 1, 3)])
def test_append_looks_at_the_strides_that_matter(layers, rows, Hkv):
    """Keys and values whose strides differ in dimensions of size one are the
    same call; ones whose rows or layers lie differently are refused."""
    B, D = 1, 128
    rng = np.random.default_rng(6)
    data = [torch.from_numpy(rng.standard_normal((layers, rows, Hkv, D))).bfloat16().to(dev()) for _ in range(2)]
    tails = _i32([0])
    plan = sv.kv_block_plan(_i32([0]), tails, _i32([[-1, -1]]), _i32([1, 0]), _i32([0, 2, 0]),
                            row_start=_i32([0, rows]), rows=rows)

    def run(k, v):
        cache = sv.kv8_cache(layers, 2, B, Hkv, device=dev())
        sv.kv8_append(cache, k, v, tails, plan)
        torch.cuda.synchronize()
        assert sv.check_device_status() == 0
        return [x.view(torch.uint8) for x in (cache.k, cache.v, cache.k_tail, cache.v_tail)]

    def laid(x, *strides):
        y = torch.zeros(8 * layers * rows * Hkv * D, dtype=torch.bfloat16, device=dev())
        return y.as_strided(x.shape, strides).copy_(x)

    want = run(*data)
    row, layer = Hkv * D + 8, rows * (Hkv * D + 8) + 64
    k = laid(data[0], layer, row, D, 1)
    odd = [layer if layers > 1 else 7 * layer, row if rows > 1 else layer, D if Hkv > 1 else 16, 1]
    assert all(torch.equal(a, b) for a, b in zip(run(k, laid(data[1], *odd)), want))
    for bad in ([layer + 8, row, D, 1] if layers > 1 else None, [layer, row + 8, D, 1] if rows > 1 else None):
        if bad:
            with pytest.raises(ValueError):
                run(k, laid(data[1], *bad))
