"""The verify loop over the paged 8-bit cache: drafts change how many tokens a
step emits, not which ones; the reported log probabilities are the emitted
tokens' own; every call also runs in the bounds-checked build."""
import numpy as np
import pytest
import torch

import speculative_decode_verify_w4a16_gb300 as sv
from speculative_decode_verify_w4a16_gb300 import verify_step as vs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decode_verify_w4a16_gb300 import build
    build.build()


@pytest.fixture(scope="module")
def target():
    return vs.Target(layers=2, seed=3)


def _prompts(target, lengths):
    g = torch.Generator().manual_seed(7)
    return [torch.randint(0, target.vocab, (n,), generator=g).tolist() for n in lengths]


def test_drafts_do_not_change_the_tokens(target):
    prompts = _prompts(target, (3, 60, 64, 131))  # blocks complete during the steps
    plain = vs.decode(target, prompts, 24, 1, lambda b, t, K: [0] * K)
    known = [p + [t for t, _ in o] for p, o in zip(prompts, plain)]

    def draft_of(b, tokens, K):
        at = len(tokens)
        return [known[b][at + i] if at + i < len(known[b]) and (at + i) % 4 else 5 for i in range(K)]

    out = vs.decode(target, prompts, 6, 4, draft_of)
    assert sv.check_device_status() == 0
    for b, o in enumerate(out):
        for i, ((t, lp), (want, want_lp)) in enumerate(zip(o, plain[b])):
            # the best token's log probability moves by no more than the logits do, whichever of two near ties it is
            assert abs(lp - want_lp) < 0.05, (b, i)
            if t != want:
                break  # a near tie: from here on the contexts differ
        assert i > 0 or t == want, b
    assert sum(map(len, out)) > 6 * len(prompts)  # drafts were accepted


def test_a_step_in_the_bounds_checked_build(target):
    from speculative_decode_verify_w4a16_gb300 import _lib, build

    want = vs.decode(target, _prompts(target, (1, 70, 200)), 4, 3, lambda b, t, K: [t[-1]] * K)
    with _lib.use_library(build.build_bounds()):
        got = vs.decode(target, _prompts(target, (1, 70, 200)), 4, 3, lambda b, t, K: [t[-1]] * K)
        # ragged rows that fill blocks, a log-probability call of many rows, a row block and cut units
        rng = np.random.default_rng(2)
        x = torch.from_numpy(rng.standard_normal((700, 1003)).astype(np.float32)).cuda()
        sv.token_logprobs(x, torch.zeros(700, 1, dtype=torch.int32, device="cuda"), top=7)
        state = vs.Requests.empty(3, 12, 40)
        cache = sv.kv8_cache(1, 40, 3, 2)
        start = torch.tensor([0, 130, 130, 700], dtype=torch.int32, device="cuda")
        k = torch.randn(700, 2, 128, device="cuda").bfloat16()
        plan = sv.kv_block_plan(state.lens, state.tails, state.table, state.ring, state.queue, row_start=start, rows=700)
        sv.kv8_append(cache, k, k, state.tails, plan)
        q = torch.randn(3, 33, 8, 128, device="cuda").bfloat16()
        sv.kv8_tree_attention(q, k[:99].view(3, 33, 2, 128), k[99:198].view(3, 33, 2, 128), cache, 0, state.table,
                              plan.new_lens, plan.new_tails)
        torch.cuda.synchronize()
        assert sv.check_device_status() == 0  # W4A16_ERR_BOUNDS would be 7
    assert [[t for t, _ in o] for o in got] == [[t for t, _ in o] for o in want]
