"""The verify loop tells its user of the errors that its kernels report."""
import pytest
import torch

import speculative_decode_verify_w4a16_gb300 as sv
from speculative_decode_verify_w4a16_gb300 import verify_step as vs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decode_verify_w4a16_gb300 import build
    build.build()


@pytest.mark.parametrize("page", [-1, 1 << 25])
def test_a_bad_page_in_the_free_list_raises(monkeypatch, page):
    target = vs.Target(layers=1, vocab=1024)
    args = (target, [list(range(7)), list(range(70))], 2, 2, lambda b, t, K: [t[-1]] * K)
    assert len(vs.decode(*args)) == 2  # the same loop with a sound free list
    empty = vs.Requests.empty

    def bad(*sizes):
        state = empty(*sizes)
        state.ring.fill_(page)  # a page id that no cache has: the plan reports it
        return state

    monkeypatch.setattr(vs.Requests, "empty", bad)
    with pytest.raises(sv.W4A16Error) as e:
        vs.decode(*args)
    assert e.value.status == 5  # W4A16_ERR_DEVICE_INPUT
    torch.cuda.synchronize()
    assert sv.check_device_status() == 0  # read and cleared
