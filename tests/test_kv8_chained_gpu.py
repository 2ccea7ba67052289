"""Calls one right after the other, without a synchronisation or another kernel
in between: each may be launched before the one whose results it reads has
ended."""
import numpy as np
import pytest
import torch

import kv8_reference as ref
import speculative_decode_verify_w4a16_gb300 as sv
from helpers import dev
from test_kv8_gpu import E4M3, E5M2, _i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decode_verify_w4a16_gb300 import build
    build.build()


@pytest.mark.parametrize("M", [4, 64])
def test_log_probabilities_right_after_the_logits(M):
    V, K = 32768, 1024
    g = torch.Generator(device="cuda")
    g.manual_seed(M)
    w = sv.prepack(*sv.quantize(torch.randn(V, K, generator=g, device="cuda") * K ** -0.5))
    xs = [torch.randn(M, K, generator=g, device="cuda").bfloat16() for _ in range(6)]
    ids = torch.randint(0, V, (M, 2), generator=g, device="cuda", dtype=torch.int32)
    want = []
    for x in xs:
        logits, _ = sv.linear_logits(x, w)
        torch.cuda.synchronize()
        r = sv.token_logprobs(logits, ids, top=7)
        torch.cuda.synchronize()
        want.append([t.clone() for t in (r.logp, r.entropy, r.top_ids, r.top_logp)])
    logits, stats = torch.empty(M, V, device="cuda"), torch.empty(M, V // 32, 2, device="cuda")
    for _ in range(5):
        for x, exp in zip(xs, want):
            sv.linear_logits(x, w, logits=logits, stats=stats)
            r = sv.token_logprobs(logits, ids, top=7)  # of the buffer that the last pass's logits were in
            assert all(torch.equal(a, b) for a, b in zip((r.logp, r.entropy, r.top_ids, r.top_logp), exp))
    assert sv.check_device_status() == 0


@pytest.mark.parametrize("dtype", [E4M3, E5M2])
def test_plan_append_and_attention_one_after_the_other(dtype):
    """Prompts into an empty cache, and attention over them at once; the pages
    hold another pass's tokens until then."""
    rng = np.random.default_rng(12)
    B, Hkv, H, n, D, passes = 6, 4, 16, 3, 128, 5
    counts = np.array([700, 64, 1300, 1, 129, 400])
    rows, pages = int(counts.sum()), int((counts // 64).sum())
    start = _i32(np.concatenate([[0], np.cumsum(counts)]))
    cache = sv.kv8_cache(1, pages, B, Hkv, dtype=dtype, device=dev())
    lens, tails, queue = _i32(np.zeros(B)), _i32(2 * np.arange(B)), _i32([0, pages, 0])
    data = []
    for _ in range(passes):
        k, v = (torch.from_numpy(rng.standard_normal((rows, Hkv, D))).bfloat16().to(dev()) for _ in range(2))
        q, own_k, own_v = (torch.from_numpy(rng.standard_normal((B, n, h, D))).bfloat16().to(dev()) for h in (H, Hkv, Hkv))
        data.append((k, v, q, own_k, own_v))
    rings = [_i32(rng.permutation(pages)) for _ in range(passes)]

    def run(i, between):
        k, v, q, own_k, own_v = data[i]
        ring, table = rings[i].clone(), torch.full((B, 21), -1, dtype=torch.int32, device=dev())
        between()
        plan = sv.kv_block_plan(lens, tails, table, ring, queue, row_start=start, rows=rows)
        between()
        sv.kv8_append(cache, k, v, tails, plan)
        between()
        return sv.kv8_tree_attention(q, own_k, own_v, cache, 0, table, plan.new_lens, plan.new_tails)

    want = [run(i, torch.cuda.synchronize).clone() for i in range(passes)]
    assert all(torch.isfinite(w).all() for w in want)
    for _ in range(4):
        got = [run(i, lambda: None) for i in range(passes)]
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))
    assert sv.check_device_status() == 0
    # and they are what the definition gives
    k, v, q, own_k, own_v = (x.cpu() for x in data[-1])
    at = np.concatenate([[0], np.cumsum(counts)])
    for b in (1, 3, 4):
        values = []
        for x in (k, v):
            x, heads = x[at[b]:at[b + 1]].transpose(0, 1), []
            for h in range(Hkv):
                blocks = [ref.quantize(x[h, 64 * j:64 * j + 64], dtype) for j in range(counts[b] // 64)]
                heads.append(torch.cat([c.double() * s for c, s in blocks] + [x[h, counts[b] // 64 * 64:].double()]))
            values.append(torch.stack(heads))
        exp, mag = ref.attention(values, q[b], own_k[b], own_v[b], ref.chain(n))
        assert ((want[-1][b].cpu().double() - exp).abs() <= 1.05 * 2.0 ** -8 * (mag + exp.abs()) + 1e-6).all()
