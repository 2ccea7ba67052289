"""The verify loop without drafts: a step of one row a request."""
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


def test_a_step_without_a_draft_emits_the_most_probable_token(target):
    B = 3
    state = vs.Requests.empty(B, 2, 2 * B)
    cache = sv.kv8_cache(len(target.layers), 2 * B, B, target.kv_heads)
    last = torch.tensor([5, 9, 70], dtype=torch.int32, device="cuda")
    for step in range(66):  # past a block's end
        if step in (0, 1, 63, 64, 65):
            logits, _, _ = target.forward(last[:, None], cache, state, 128)
            want = logits[:, 0].double().log_softmax(1)
        e = vs.verify_step(target, cache, state, last, last.new_empty((B, 0)), 128)
        last = e.tokens[:, 0].contiguous()
        if step in (0, 1, 63, 64, 65):
            assert e.tokens.shape == e.logp.shape == (B, 1) and e.top_ids.shape == (B, 3)
            assert torch.equal(last.long(), want.argmax(1)) and torch.equal(e.top_ids[:, 0], last)
            assert (e.logp[:, 0] - want.amax(1)).abs().max() < 1e-5
    assert state.lens.tolist() == [66] * B
    assert sv.check_device_status() == 0


def test_plain_decoding_gives_the_same_with_and_without_a_dummy_draft(target):
    g = torch.Generator().manual_seed(7)
    prompts = [torch.randint(0, target.vocab, (n,), generator=g).tolist() for n in (1, 60, 131)]
    plain = vs.decode(target, prompts, 12, 0, lambda b, t, K: [])
    other = vs.decode(target, prompts, 12, 1, lambda b, t, K: [0] * K)
    for b in range(3):
        assert len(plain[b]) == 12
        for (t, lp), (want, want_lp) in zip(plain[b], other[b]):
            assert abs(lp - want_lp) < 0.05, b  # as in test_verify_step_gpu
            if t != want:
                break  # a near tie: from here on the contexts differ
