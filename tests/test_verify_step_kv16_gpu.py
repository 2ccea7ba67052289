"""The verify loop over the paged 16-bit cache, and with a rotation over either
cache: rotation, append and attention together, as a target runs them."""
import math

import pytest
import torch

import speculative_decode_verify_w4a16_gb300 as sv
from speculative_decode_verify_w4a16_gb300 import verify_step as vs

pytestmark = pytest.mark.gpu

BASE = 500.0


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decode_verify_w4a16_gb300 import build
    build.build()


@pytest.fixture(scope="module")
def target():
    return vs.Target(layers=2, seed=3, rope=sv.rope_frequencies(vs.D, BASE))


def _prompts(target, lengths):
    g = torch.Generator().manual_seed(7)
    return [torch.randint(0, target.vocab, (n,), generator=g).tolist() for n in lengths]


def _weight_of(w, K):
    """The packed weight's matrix, transposed: the identity times it, row by row (exact: a code times a scale, rounded
    to bf16 on the way out)."""
    rows = []
    for i in range(0, K, 64):
        x = torch.zeros(min(64, K - i), K, device="cuda", dtype=torch.bfloat16)
        x[torch.arange(x.shape[0]), i + torch.arange(x.shape[0])] = 1
        rows.append(sv.linear(x, w).double())
    return torch.cat(rows)  # [K, N]


def _plain_logits(target, ids):
    """One request's logits in 64 bits, with no cache. (The weights carry bf16's rounding, 2^-9 on average.)"""
    n, H, Hk, D = len(ids), target.heads, target.kv_heads, vs.D
    h = target.embed[torch.tensor(ids, device="cuda")].double()
    pos = torch.arange(n, device="cuda", dtype=torch.float64)

    def norm(x):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)

    def turn(x):
        f = torch.tensor([BASE ** (-2 * i / D) for i in range(D // 2)], dtype=torch.float64, device="cuda")
        c, s = torch.cos(pos[:, None] * f)[:, None], torch.sin(pos[:, None] * f)[:, None]
        a, b = x[..., :D // 2], x[..., D // 2:]
        return torch.cat([a * c - b * s, a * s + b * c], -1)

    for qkv_w, o_w, gate_up, down in target.layers:
        qkv = (norm(h) @ _weight_of(qkv_w, target.hidden)).view(n, H + 2 * Hk, D)
        q, k, v = turn(qkv[:, :H]), turn(qkv[:, H:H + Hk]), qkv[:, H + Hk:]
        k, v = k.repeat_interleave(H // Hk, 1), v.repeat_interleave(H // Hk, 1)
        s = torch.einsum("ihd,jhd->hij", q, k) / math.sqrt(D)
        s = s.masked_fill(torch.ones(n, n, device="cuda").triu(1).bool(), -math.inf)
        a = torch.einsum("hij,jhd->ihd", s.softmax(-1), v).reshape(n, H * D)
        h = h + a @ _weight_of(o_w, H * D)
        gate, up = (norm(h) @ _weight_of(gate_up, target.hidden)).chunk(2, 1)
        h = h + (torch.nn.functional.silu(gate) * up) @ _weight_of(down, target.inner)
    return norm(h) @ _weight_of(target.lm_head, target.hidden)


@pytest.mark.parametrize("cache", ["kv8", "kv16"])
def test_the_logits_are_the_model_s(target, cache):
    """60 tokens (all in bf16 in either cache), in chunks of 7: against 64 bits without a cache."""
    ids = _prompts(target, (60,))[0]
    want = _plain_logits(target, ids)
    if cache == "kv16":
        state, kv = vs.Requests.resident(1, 2), sv.kv16_cache(len(target.layers), 2, target.kv_heads)
    else:
        state, kv = vs.Requests.empty(1, 2, 2), sv.kv8_cache(len(target.layers), 2, 1, target.kv_heads)
    got = []
    for at in range(0, 60, 7):
        part = torch.tensor([ids[at:at + 7]], dtype=torch.int32, device="cuda")
        n = part.shape[1]
        logits, k, v = target.forward(part, kv, state, 128)
        got.append(logits[0])
        if cache == "kv16":
            assert k is None and v is None
            state.lens = state.lens + n
        else:
            start = torch.tensor([0, n], dtype=torch.int32, device="cuda")
            plan = sv.kv_block_plan(state.lens, state.tails, state.table, state.ring, state.queue, row_start=start, rows=n)
            sv.kv8_append(kv, k, v, state.tails, plan)
            state.advance(plan)
    got = torch.cat(got).double()
    assert sv.check_device_status() == 0
    # Roundings to bf16, 2^-9 of a value in the mean, one after another on the way to the logits: embedding to logits
    # goes through some 10 a layer (norm, projection, rotation, weights, attention, output, sum, norm, gate, product,
    # down, sum) and as many in the plain form's weights, each of which moves a logit by about its own relative size
    # (independent terms of a dot product): sqrt(2 * 24) * 2^-9 = 1.4 %. Four times that.
    assert (got - want).norm() < 4 * 48 ** 0.5 * 2.0 ** -9 * want.norm()
    # a rotation left out is told apart
    target.rope, rope = None, target.rope
    try:
        state = vs.Requests.resident(1, 2)
        bare = target.forward(torch.tensor([ids], dtype=torch.int32, device="cuda"),
                              sv.kv16_cache(len(target.layers), 2, target.kv_heads), state, 128)[0][0].double()
    finally:
        target.rope = rope
    assert (bare - want).norm() > 2 * (got - want).norm()


def test_drafts_do_not_change_the_tokens(target):
    prompts = _prompts(target, (3, 60, 64, 131))
    plain = vs.decode(target, prompts, 24, 0, lambda b, t, K: [], cache="kv16")
    known = [p + [t for t, _ in o] for p, o in zip(prompts, plain)]

    def draft_of(b, tokens, K):
        at = len(tokens)
        return [known[b][at + i] if at + i < len(known[b]) and (at + i) % 4 else 5 for i in range(K)]

    out = vs.decode(target, prompts, 6, 4, draft_of, cache="kv16")
    assert sv.check_device_status() == 0
    for b, o in enumerate(out):
        for i, ((t, lp), (want, want_lp)) in enumerate(zip(o, plain[b])):
            assert abs(lp - want_lp) < 0.05, (b, i)  # as with the 8-bit cache
            if t != want:
                break  # a near tie: from here on the contexts differ
        assert i > 0 or t == want, b
    assert sum(map(len, out)) > 6 * len(prompts)  # drafts were accepted


def test_rejected_rows_leave_no_trace(target):
    """After a step whose drafts were all wrong the next step's logits are those of a request that never saw them."""
    ids = _prompts(target, (70,))[0]
    one = torch.tensor([ids], dtype=torch.int32, device="cuda")
    logits = []
    for wrong in (False, True):
        state, kv = vs.Requests.resident(1, 3), sv.kv16_cache(len(target.layers), 3, target.kv_heads)
        target.forward(one[:, :60].contiguous(), kv, state, 192)
        state.lens = state.lens + 60
        if wrong:  # past the page's end
            target.forward(one[:, :9].contiguous(), kv, state, 192)
        logits.append(target.forward(one[:, 60:66].contiguous(), kv, state, 192)[0])
    assert torch.equal(*logits)


def test_a_step_in_a_graph(target):
    """The step, captured and replayed with the lengths moved on inside: as eager steps."""
    B, prompts = 2, _prompts(target, (20, 61))

    def begin():
        state, kv = vs.Requests.resident(B, 3), sv.kv16_cache(len(target.layers), 3 * B, target.kv_heads)
        start = torch.tensor([0, 20, 81], dtype=torch.int32, device="cuda")
        ids = torch.tensor(sum(prompts, []), dtype=torch.int32, device="cuda")
        target.forward(ids[:79, None].contiguous(), kv, state, 192, row_start=start.clamp(max=79))
        state.lens = state.lens + start.clamp(max=79).diff()
        return state, kv

    draft = torch.full((B, 3), 7, dtype=torch.int32, device="cuda")
    first = torch.tensor([4, 9], dtype=torch.int32, device="cuda")
    state, kv = begin()
    want, last = [], first
    for _ in range(3):
        e = vs.verify_step(target, kv, state, last, draft, 192)
        want.append(e.tokens.clone())
        n = (e.tokens >= 0).sum(1, keepdim=True) - 1
        last = e.tokens.gather(1, n)[:, 0].contiguous()
    state, kv = begin()
    lens, last = state.lens, first.clone()

    def step():
        state.lens = lens
        e = vs.verify_step(target, kv, state, last, draft, 192)
        lens.copy_(state.lens)
        last.copy_(e.tokens.gather(1, (e.tokens >= 0).sum(1, keepdim=True) - 1)[:, 0])
        return e.tokens

    s = torch.cuda.Stream()
    keep = lens.clone(), last.clone()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        lens.copy_(keep[0])
        last.copy_(keep[1])
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tokens = step()
    for w in want:
        graph.replay()
        assert torch.equal(tokens, w)
    assert sv.check_device_status() == 0


def test_a_page_of_no_cache_raises(target, monkeypatch):
    resident = vs.Requests.resident

    def bad(*sizes):
        state = resident(*sizes)
        state.table[1, 0] = 1 << 25
        return state

    args = (target, [list(range(7)), list(range(70))], 2, 2, lambda b, t, K: [t[-1]] * K, "kv16")
    assert len(vs.decode(*args)) == 2
    monkeypatch.setattr(vs.Requests, "resident", bad)
    with pytest.raises(sv.W4A16Error) as e:
        vs.decode(*args)
    assert e.value.status == 5  # W4A16_ERR_DEVICE_INPUT
    assert sv.check_device_status() == 0  # read and cleared


def test_steps_in_the_bounds_checked_build(target):
    from speculative_decode_verify_w4a16_gb300 import _lib, build

    args = target, _prompts(target, (1, 70, 200)), 4, 3, lambda b, t, K: [t[-1]] * K, "kv16"
    want = vs.decode(*args)
    with _lib.use_library(build.build_bounds()):
        got = vs.decode(*args)
        # ragged rows over page ends and past the last request's, 64-wide heads, cut units, rows of fp32 and a window
        g = torch.Generator(device="cuda").manual_seed(1)
        start = torch.tensor([0, 130, 130, 690], dtype=torch.int32, device="cuda")
        lens = torch.tensor([0, 5, 3000], dtype=torch.int32, device="cuda")
        table = torch.arange(3 * 60, dtype=torch.int32, device="cuda").view(3, 60)
        for dtype, D, H, Hk, inter in ((torch.bfloat16, 128, 8, 2, False), (torch.float16, 64, 6, 3, True)):
            cache = sv.kv16_cache(1, 180, Hk, D, dtype)
            qkv = torch.randn(700, H + 2 * Hk, D, generator=g, device="cuda").to(dtype)
            q, k, v = qkv.split((H, Hk, Hk), 1)
            f = sv.rope_frequencies(D // 2, interleaved=inter)
            q = sv.kv16_append(cache, 0, k, v, table, lens, row_start=start, rope=f, q=q, q_out=q)
            sv.kv16_attention(q, cache, 0, table, lens, row_start=start)
            sv.kv16_attention(q, cache, 0, table, lens, row_start=start, window=77)
            x = torch.randn(37, 3, D, generator=g, device="cuda")
            sv.rope(x, torch.arange(37, dtype=torch.int32, device="cuda"), f, inverse=inter)
        torch.cuda.synchronize()
        assert sv.check_device_status() == 0  # W4A16_ERR_BOUNDS would be 7
    assert [[t for t, _ in o] for o in got] == [[t for t, _ in o] for o in want]
