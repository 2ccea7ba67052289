"""The default workspaces of kv8_tree_attention and token_logprobs: calls on
several streams share nothing, a captured graph and eager calls share nothing,
and a call that needs more takes nothing from a graph."""
import numpy as np
import pytest
import torch

import kv8_reference as ref
import speculative_decode_verify_w4a16_gb300 as sv
from helpers import dev
from speculative_decode_verify_w4a16_gb300 import api
from test_kv8_gpu import E4M3, _attn_inputs, _history

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decode_verify_w4a16_gb300 import build
    build.build()


def _attention(seed, B, n, H, Hkv, lens):
    """A call of the operator: cut units, so that counters and partial results are used."""
    rng = np.random.default_rng(seed)
    cache = ref.Cache([_history(rng, Hkv, L) for L in lens], E4M3, rng, max(lens))
    c, table, dl, tails = cache.to(sv, dev())
    qkv, cols = _attn_inputs(rng, B, n, H, Hkv)
    dq = [qkv.to(dev())[:, :, s].unflatten(2, (-1, 128)) for s in cols]
    return lambda **kw: sv.kv8_tree_attention(*dq, c, 0, table, dl, tails, max_len=max(lens), **kw)


def _logprobs(seed, R, V):
    x = torch.randn(R, V, generator=torch.Generator().manual_seed(seed)).to(dev())
    ids = torch.zeros(R, dtype=torch.int32, device=dev())
    return lambda **kw: sv.token_logprobs(x, ids, top=5, **kw).top_logp


CALLS = [lambda seed: _attention(seed, 2, 5, 16, 2, (1900 + 64 * seed, 700)), lambda seed: _logprobs(seed, 5, 60000)]


@pytest.mark.parametrize("make", CALLS)
def test_each_stream_has_its_own(make):
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    here = api._stream_workspace(1000, "kv8_attention")
    on_a, on_b = (api._stream_workspace(1000, "kv8_attention", s) for s in (a, b))
    assert len({x.data_ptr() for x in (here, on_a, on_b)}) == 3
    assert api._stream_workspace(1000, "kv8_attention", a).data_ptr() == on_a.data_ptr()
    with torch.cuda.stream(a):
        assert api._stream_workspace(1000, "kv8_attention").data_ptr() == on_a.data_ptr()
    calls = [make(1), make(2)]
    want = [f().clone() for f in calls]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(40):  # both streams busy at once
        for i, s in enumerate((a, b)):
            with torch.cuda.stream(s):
                got[i].append(calls[i]())
    torch.cuda.synchronize()
    assert sv.check_device_status() == 0
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])


@pytest.mark.parametrize("make", CALLS)
def test_the_stream_argument_names_where_the_buffer_is_zeroed(make):
    f, s = make(3), torch.cuda.Stream()
    want = f().clone()
    torch.cuda.synchronize()
    busy = torch.empty(1 << 28, dtype=torch.uint8, device=dev())
    for _ in range(20):
        busy.zero_()  # the current stream is behind
    got = f(stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    torch.cuda.synchronize()
    assert sv.check_device_status() == 0


@pytest.mark.parametrize("make,larger", [(CALLS[0], lambda: _attention(9, 2, 64, 16, 2, (900, 700))),
                                         (CALLS[1], lambda: _logprobs(9, 500, 120000))])
def test_a_graph_has_its_own(make, larger):
    """The first call ever on a stream is a captured one; eager calls follow on
    that stream, one of them with more to keep; the graph goes on giving the same."""
    f, g, s = make(4), make(5), torch.cuda.Stream()
    want_f, want_g = f().clone(), g().clone()  # (loads the kernels, on the current stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out_f, out_g = f(), g()  # one after the other, in one buffer
        both = api._stream_ws[(0, s.cuda_stream, "kv8_attention" if make is CALLS[0] else "logprobs", True)][1]
    for _ in range(3):
        out_f.fill_(-1.0), out_g.fill_(-1.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out_f, want_f) and torch.equal(out_g, want_g)
        with torch.cuda.stream(s):
            assert torch.equal(f(), want_f)
            larger()()
            assert torch.equal(g(), want_g)
        torch.cuda.synchronize()
    # a second capture on the same stream has another buffer
    second = torch.cuda.CUDAGraph()
    with torch.cuda.graph(second, stream=s):
        out_2 = f()
        assert api._stream_ws[(0, s.cuda_stream, "kv8_attention" if make is CALLS[0] else "logprobs",
                               True)][1].data_ptr() != both.data_ptr()
    second.replay(), graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out_2, want_f) and torch.equal(out_f, want_f) and torch.equal(out_g, want_g)
    assert sv.check_device_status() == 0


@pytest.mark.parametrize("make", CALLS)
def test_a_workspace_that_is_not_on_the_device_is_refused(make):
    f = make(6)
    f()
    with pytest.raises(ValueError):
        f(ws=torch.zeros(1 << 26, dtype=torch.uint8))
    with pytest.raises(sv.W4A16Error) as e:
        f(ws=torch.zeros(256, dtype=torch.uint8, device=dev()))
    assert e.value.status == 6  # W4A16_ERR_WORKSPACE
    torch.cuda.synchronize()
    assert sv.check_device_status() == 0
