"""Host-side checks of the paged 8-bit cache and log-probability entry points
(no GPU needed): bad arguments are refused before any launch; the plain
implementations the GPU tests compare with keep their own invariants."""
import ctypes
import math

import numpy as np
import pytest
import torch

import __graft_entry__  # noqa: F401  (puts the repo root on sys.path)
import kv8_reference as ref
from speculative_decode_verify_w4a16_gb300 import _lib
from speculative_decode_verify_w4a16_gb300 import build as sv_build

P, ODD, WS = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10002), ctypes.c_void_p(0x20000)
OTHER = ctypes.c_void_p(0x30000)
BAD, UNSUPPORTED, WORKSPACE = _lib.ERR_INVALID_ARG, _lib.ERR_UNSUPPORTED, _lib.ERR_WORKSPACE


@pytest.fixture(scope="module")
def L():
    sv_build.build()
    return _lib.lib()


def test_plan_refuses(L):
    def plan(lens=P, row_start=None, parents=None, node=P, B=4, n=5, rows=20, max_blocks=8, cap=64, table=P,
             new_lens=OTHER, new_tails=OTHER, new_queue=OTHER, src=P, slots=P):
        return L.kv_block_plan(lens, P, row_start, parents, node, None, B, n, rows, max_blocks, cap, table, P, P,
                               new_lens, new_tails, P, new_queue, src, slots, None)
    assert plan(lens=None) == BAD and plan(table=None) == BAD and plan(src=None) == BAD and plan(slots=None) == BAD
    assert plan(node=None) == BAD and plan(row_start=P) == BAD             # one of the two modes
    assert plan(node=None, row_start=P, parents=P) == BAD
    assert plan(B=0) == BAD and plan(rows=19) == BAD and plan(n=0, rows=0) == BAD and plan(rows=-1) == BAD
    assert plan(max_blocks=0) == BAD and plan(cap=0) == BAD
    assert plan(new_lens=P) == BAD and plan(new_tails=P) == BAD and plan(new_queue=P) == BAD  # no aliases
    assert plan(lens=ODD) == BAD and plan(slots=ODD) == BAD
    assert plan(B=5000, rows=25000) == UNSUPPORTED and plan(n=65, rows=260) == UNSUPPORTED
    assert plan(cap=(1 << 25) + 1) == UNSUPPORTED and plan(max_blocks=1 << 30) == UNSUPPORTED
    assert plan(node=None, row_start=P, rows=(1 << 30) + 1) == UNSUPPORTED


def test_append_refuses(L):
    def append(k_new=P, stride=1024, layer=0, B=4, rows=20, Hkv=8, D=128, layers=1, pages=10, tail_pages=8, fmt=0,
               k=P, scale=P, tail=P, slots=P):
        return L.kv8_append(k_new, P, stride, layer, P, P, P, P, slots, B, rows, Hkv, D, layers, pages, tail_pages, fmt,
                            k, P, scale, P, tail, P, None)
    for name in ("k_new", "k", "scale", "tail", "slots"):
        assert append(**{name: None}) == BAD
        assert append(**{name: ODD}) == BAD
    assert append(stride=1016) == BAD and append(stride=1028) == BAD and append(layer=4) == BAD and append(layer=-8) == BAD
    assert append(B=0) == BAD and append(rows=0) == BAD and append(layers=0) == BAD and append(Hkv=0) == BAD
    assert append(pages=0) == BAD and append(tail_pages=0) == BAD and append(fmt=2) == BAD and append(fmt=-1) == BAD
    assert append(D=64, stride=512) == UNSUPPORTED and append(B=5000) == UNSUPPORTED


def test_attention_refuses(L):
    def attn(q=P, q_stride=8192, kv_stride=1024, k=P, lens=P, parents=None, B=4, n=5, H=64, Hkv=8, D=128, max_blocks=16,
             pages=10, tail_pages=8, max_len=1000, fmt=0, scale=0.1, out=P):
        return L.kv8_tree_attention(q, P, P, q_stride, kv_stride, k, P, P, P, P, P, P, lens, P, parents, B, n, H, Hkv, D,
                                    max_blocks, pages, tail_pages, max_len, fmt, scale, out, None, 0, None)
    for name in ("q", "k", "lens", "out"):
        assert attn(**{name: None}) == BAD
        assert attn(**{name: ODD}) == BAD
    assert attn(parents=ODD) == BAD
    assert attn(q_stride=8184) == BAD and attn(q_stride=8196) == BAD and attn(kv_stride=1016) == BAD
    assert attn(B=0) == BAD and attn(n=0) == BAD and attn(H=60) == BAD and attn(Hkv=0) == BAD
    assert attn(max_len=-1) == BAD and attn(max_len=17 * 64) == BAD and attn(max_blocks=0) == BAD
    assert attn(fmt=3) == BAD and attn(scale=0.0) == BAD and attn(scale=math.inf) == BAD and attn(scale=math.nan) == BAD
    assert attn(pages=0) == BAD and attn(tail_pages=0) == BAD
    assert attn(n=65) == UNSUPPORTED and attn(D=64) == UNSUPPORTED
    f = L.kv8_tree_attention_workspace_bytes
    assert f(0, 5, 64, 8, 128, 100) == 0 and f(4, 65, 64, 8, 128, 100) == 0 and f(4, 5, 60, 8, 128, 100) == 0


def test_logprobs_refuses(L):
    def lp(x=P, bf16=0, ids=P, R=4, V=1000, m=1, top=5, logp=P, ent=P, ti=P, tl=P, ws=WS, size=1 << 20):
        return L.token_logprobs(x, bf16, ids, R, V, m, top, logp, ent, ti, tl, ws, size, None)
    assert lp(x=None) == BAD and lp(ids=None) == BAD and lp(logp=None) == BAD and lp(ti=None) == BAD and lp(tl=None) == BAD
    assert lp(x=ODD) == BAD and lp(ids=ODD) == BAD and lp(ent=ODD) == BAD and lp(bf16=2) == BAD
    assert lp(x=ctypes.c_void_p(0x10001), bf16=1) == BAD
    assert lp(R=0) == BAD and lp(V=0) == BAD and lp(m=-1) == BAD and lp(m=65) == BAD and lp(top=65) == BAD
    assert lp(V=4, top=5) == BAD and lp(V=(1 << 20) + 1) == BAD
    assert lp(ws=None) == WORKSPACE and lp(ws=ODD) == WORKSPACE and lp(size=16) == WORKSPACE
    f = L.token_logprobs_workspace_bytes
    assert f(4, 1000, 5) > 0 and f(0, 1000, 5) == 0 and f(4, 3, 5) == 0


# ------------------------------------------- the plain implementations

@pytest.mark.parametrize("dtype", [torch.float8_e4m3fn, torch.float8_e5m2])
def test_reference_scale_is_the_smallest_power_of_two(dtype):
    rng = np.random.default_rng(1)
    for mag in (1e-20, 1e-3, 1.0, 1e5, 3e38):
        x = torch.from_numpy(rng.standard_normal((64, 128)) * mag).bfloat16()
        codes, s = ref.quantize(x, dtype)
        top = float(x.double().abs()[x.isfinite()].max())
        assert math.frexp(s)[0] == 0.5 and top / s <= ref.LARGEST[dtype] and top / (s / 2) > ref.LARGEST[dtype]
        step = 2.0 ** (-4 if dtype == torch.float8_e4m3fn else -3)  # half a step of the type
        low = 2.0 ** (-10 if dtype == torch.float8_e4m3fn else -17) * s
        err = (codes.double() * s - x.double()).abs()[x.isfinite()]
        assert (err <= step * x.double().abs()[x.isfinite()] + low).all()


def test_reference_plan_by_hand():
    """Request 0 keeps rows 0 1 and completes block 1; request 1 ended; request 2 keeps nothing."""
    table, ring, p = ref.plan([126, 64, 5], [0, 3, 4], np.array([[9, -1, -1], [7, -1, -1], [-1, -1, -1]]),
                              np.array([5, 6, 0, 0]), [0, 2, 0], 4, [[0, 1], [2], []], [0, 1, 0])
    assert table.tolist() == [[9, 5, -1], [7, -1, -1], [-1, -1, -1]]
    assert ring.tolist() == [5, 6, 7, 0]
    assert p["new_lens"].tolist() == [128, 0, 5] and p["new_tails"].tolist() == [1, 3, 4]
    assert p["slots"].tolist() == [5 * 64 + 62, 5 * 64 + 63, ref.SKIP, ref.SKIP]
    assert p["src_rows"].tolist() == [0, 1, -1, -1] and p["queue"].tolist() == [1, 2, 0]


def test_reference_attention_by_hand():
    """Equal scores average the values that a node sees: the prefix, its ancestors and itself."""
    values = [torch.zeros(1, 2, 4, dtype=torch.float64), torch.tensor([[[1.0] * 4, [3.0] * 4]], dtype=torch.float64)]
    v = torch.tensor([[[5.0] * 4], [[7.0] * 4], [[11.0] * 4]])
    out, mag = ref.attention(values, torch.ones(3, 2, 4), torch.zeros(3, 1, 4), v, [-1, 0, 0])
    assert out[:, 0, 0].tolist() == [3.0, 4.0, 5.0] and torch.equal(out, mag)


def test_the_verify_loop_refuses_what_it_cannot_run():
    from speculative_decode_verify_w4a16_gb300 import verify_step

    with pytest.raises(ValueError):
        verify_step.decode(None, [], 1, 1, None)
    with pytest.raises(ValueError):
        verify_step.decode(None, [[1], []], 1, 1, None)
    with pytest.raises(ValueError):
        verify_step.decode(None, [[1]] * 17, 1, 4, None)
