"""Host-side checks of rotary positions and the paged 16-bit cache (no GPU
needed): bad arguments are refused before any launch; the frequencies and the
plain implementations the GPU tests compare with keep their own invariants."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import __graft_entry__  # noqa: F401  (puts the repo root on sys.path)
import kv16_reference as ref
import speculative_decode_verify_w4a16_gb300 as sv
from speculative_decode_verify_w4a16_gb300 import _lib
from speculative_decode_verify_w4a16_gb300 import build as sv_build

P, ODD = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10002)
OTHER = ctypes.c_void_p(0x30000)
BAD, UNSUPPORTED = _lib.ERR_INVALID_ARG, _lib.ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    sv_build.build()
    return _lib.lib()


def test_rope_refuses(L):
    def rope(x=P, xs=1024, pos=P, turns=P, T=4, heads=8, D=128, rot=128, factor=1.0, kind=0, y=OTHER, ys=1024):
        return L.rope_rotate(x, xs, pos, turns, T, heads, D, rot, 0, factor, 0, kind, y, ys, None)
    for name in ("x", "pos", "turns", "y"):
        assert rope(**{name: None}) == BAD and rope(**{name: ODD}) == BAD
    assert rope(T=0) == BAD and rope(heads=0) == BAD and rope(D=0) == BAD and rope(rot=0) == BAD and rope(rot=144) == BAD
    assert rope(xs=1016) == BAD and rope(xs=1028) == BAD and rope(ys=1016) == BAD and rope(y=P, ys=2048) == BAD
    assert rope(kind=3) == BAD and rope(kind=-1) == BAD
    assert rope(factor=0.0) == BAD and rope(factor=math.inf) == BAD and rope(factor=math.nan) == BAD
    assert rope(rot=24) == UNSUPPORTED and rope(D=132, xs=2048, ys=2048) == UNSUPPORTED
    assert rope(D=1032, xs=8256, ys=8256) == UNSUPPORTED


def test_append_refuses(L):
    def append(k_new=P, v_new=P, ks=256, vs=256, q=P, qs=1024, turns=P, rot=128, factor=1.0, table=P, lens=P, start=P,
               T=6, B=2, H=8, Hkv=2, D=128, max_blocks=4, pages=9, kind=0, k=P, v=P, q_out=OTHER, os=1024):
        return L.kv16_append(k_new, v_new, ks, vs, q, qs, turns, rot, 0, factor, table, lens, start, T, B, H, Hkv, D,
                             max_blocks, pages, kind, k, v, q_out, os, None)
    for name in ("k_new", "v_new", "table", "lens", "k", "v"):
        assert append(**{name: None}) == BAD and append(**{name: ODD}) == BAD
    assert append(q=None) == BAD and append(q_out=None) == BAD and append(q=ODD) == BAD and append(q_out=ODD) == BAD
    assert append(start=ODD) == BAD and append(turns=ODD) == BAD and append(turns=None) == BAD
    assert append(ks=248) == BAD and append(vs=260) == BAD and append(qs=1016) == BAD and append(os=1020) == BAD
    assert append(q_out=P, os=2048) == BAD
    assert append(T=0) == BAD and append(B=0) == BAD and append(H=0) == BAD and append(Hkv=0) == BAD
    assert append(max_blocks=0) == BAD and append(pages=0) == BAD and append(pages=1 << 25) == BAD
    assert append(B=1 << 20, max_blocks=1 << 12) == BAD and append(rot=-16) == BAD and append(rot=144) == BAD
    assert append(start=None, T=7) == BAD and append(kind=2) == BAD and append(factor=-1.0) == BAD
    assert append(D=80, rot=80) == UNSUPPORTED and append(rot=24) == UNSUPPORTED and append(B=5000) == UNSUPPORTED
    assert append(T=(1 << 24) + 2) == UNSUPPORTED


def test_attention_refuses(L):
    def attn(q=P, qs=1024, k=P, v=P, table=P, lens=P, start=P, T=6, B=2, H=8, Hkv=2, D=128, max_blocks=4, pages=9,
             window=0, scale=0.1, kind=0, out=P):
        return L.kv16_attention(q, qs, k, v, table, lens, start, T, B, H, Hkv, D, max_blocks, pages, window, scale, kind,
                                out, None, 0, None)
    for name in ("q", "k", "v", "table", "lens", "out"):
        assert attn(**{name: None}) == BAD and attn(**{name: ODD}) == BAD
    assert attn(start=ODD) == BAD and attn(start=None, T=7) == BAD
    assert attn(qs=1016) == BAD and attn(qs=1028) == BAD
    assert attn(T=0) == BAD and attn(B=0) == BAD and attn(H=7) == BAD and attn(Hkv=0) == BAD and attn(H=0) == BAD
    assert attn(max_blocks=0) == BAD and attn(pages=0) == BAD and attn(pages=1 << 25) == BAD and attn(window=-1) == BAD
    assert attn(scale=0.0) == BAD and attn(scale=math.inf) == BAD and attn(scale=math.nan) == BAD and attn(kind=2) == BAD
    assert attn(D=80) == UNSUPPORTED and attn(D=256, qs=2048) == UNSUPPORTED and attn(B=5000) == UNSUPPORTED
    assert attn(T=(1 << 24) + 2, qs=1024) == UNSUPPORTED
    f = L.kv16_attention_workspace_bytes
    assert f(0, 8, 2, 128) == 0 and f(4, 7, 2, 128) == 0 and f(4, 8, 2, 80) == 0


# ------------------------------------------------------------- frequencies

def test_frequencies_by_hand():
    f, a = sv.rope_angles(4, 100.0)
    assert f == pytest.approx([1.0, 0.1]) and a == 1.0
    assert sv.rope_angles(4, 100.0, {"kind": "linear", "factor": 4})[0] == pytest.approx([0.25, 0.025])
    assert sv.rope_angles(4, 100.0, {"kind": "ntk", "factor": 3})[0] == pytest.approx([1.0, (100 * 9) ** -0.5])
    # bands: over 100 positions the pairs turn 15.9 and 1.59 times: kept above 10, divided below 1, a blend between
    f, a = sv.rope_angles(4, 100.0, {"kind": "bands", "factor": 5, "low": 1, "high": 10, "trained": 100})
    keep = (10 / (2 * math.pi) - 1) / 9
    assert f == pytest.approx([1.0, 0.1 * keep + 0.02 * (1 - keep)]) and a == 1.0
    # yarn: 8 pairs; the ramp runs from the pair that turns 32 times to the one that turns once
    f, a = sv.rope_angles(16, 10000.0, {"kind": "yarn", "factor": 16, "trained": 4096})
    plain = sv.rope_angles(16, 10000.0)[0]
    at = [16 * math.log(4096 / (n * 2 * math.pi)) / (2 * math.log(10000.0)) for n in (32, 1)]
    lo, hi = math.floor(at[0]), math.ceil(at[1])
    assert (lo, hi) == (2, 6) and a == pytest.approx(0.1 * math.log(16) + 1)
    for i in range(8):
        r = min(max((i - lo) / (hi - lo), 0), 1)
        assert f[i] == pytest.approx(plain[i] * (1 - r) + plain[i] / 16 * r)
    assert sv.rope_angles(16, 10000.0, {"kind": "yarn", "factor": 16, "trained": 4096, "attention": 1.0})[1] == 1.0


def test_turns_are_the_angles():
    r = sv.rope_frequencies(128, 500000.0, device="cpu")
    assert r.rot == 128 and not r.interleaved and r.factor == 1.0
    for t, a in zip(r.turns.tolist(), sv.rope_angles(128, 500000.0)[0]):
        assert abs(Fraction(t % 2 ** 64, 2 ** 64) - Fraction(a) / (2 * ref.PI)) <= Fraction(1, 2 ** 65)


def test_frequencies_refuse():
    for args, kw in (((0,), {}), ((24,), {}), ((8,), {}), ((64, -1.0), {}), ((64, math.inf), {}),
                     ((64,), dict(scaling={"kind": "other"})), ((64,), dict(scaling={"kind": "linear"})),
                     ((64,), dict(scaling={"kind": "linear", "factor": 0})), ((64,), dict(scaling={"factor": 2})),
                     ((64,), dict(scaling={"kind": "linear", "factor": 2, "low": 1})),
                     ((64,), dict(scaling={"kind": "bands", "factor": 2, "low": 4, "high": 4, "trained": 100})),
                     ((64,), dict(scaling={"kind": "yarn", "factor": 2, "trained": 100, "fast": 1, "slow": 2}))):
        with pytest.raises(ValueError):
            sv.rope_frequencies(*args, device="cpu", **kw)
    with pytest.raises(ValueError):
        sv.rope_angles(3)


def test_cpu_tensors_are_refused():
    x, p = torch.zeros(2, 3, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    c = sv.KV16Cache(*(torch.zeros(1, 2, 1, 64, 64, dtype=torch.bfloat16) for _ in range(2)))
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        sv.rope(x, p, sv.rope_frequencies(64, device="cpu"))
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        sv.kv16_attention(x, c, 0, p[:, None], p)


# ------------------------------------------- the plain implementations

def test_reference_rotation_by_hand():
    cos, sin = ref.cos_sin([1, 3], [math.pi / 2, math.pi])
    assert cos.numpy() == pytest.approx(np.array([[0, -1], [0, -1]]), abs=1e-12)
    assert sin.numpy() == pytest.approx(np.array([[1, 0], [-1, 0]]), abs=1e-12)
    x = torch.tensor([[[1.0, 2.0, 3.0, 4.0, 5.0]]] * 2)
    half, _ = ref.rotate(x, cos, sin, False)  # pairs (1, 3) and (2, 4)
    assert half[0, 0].tolist() == pytest.approx([-3, -2, 1, -4, 5], abs=1e-12)
    adjacent, _ = ref.rotate(x, cos, sin, True, 2.0)  # pairs (1, 2) and (3, 4)
    assert adjacent[1, 0].tolist() == pytest.approx([4, -2, -6, -8, 5], abs=1e-12)
    back, _ = ref.rotate(adjacent, cos, sin, True, 0.5, inverse=True)
    assert back[1, 0].tolist() == pytest.approx([1, 2, 3, 4, 5], abs=1e-12)


def test_reference_far_positions_keep_their_turns():
    cos, sin = ref.cos_sin([10 ** 9], [2 * math.pi * 0.25])
    exact = float((10 ** 9 * Fraction(2 * math.pi * 0.25) / (2 * ref.PI)) % 1)
    assert abs(cos[0, 0] - math.cos(2 * math.pi * exact)) < 1e-12 and abs(sin[0, 0] - math.sin(2 * math.pi * exact)) < 1e-12


def test_reference_attention_by_hand():
    """Equal scores average the values that a row sees."""
    k = torch.zeros(1, 5, 4)
    v = torch.tensor([1.0, 3.0, 5.0, 7.0, 11.0])[None, :, None].expand(1, 5, 4).clone()
    out, mag = ref.attention(torch.ones(3, 2, 4), k, v, 2)
    assert out[:, 0, 0].tolist() == pytest.approx([3, 4, 5.4]) and torch.equal(out, mag)
    out, _ = ref.attention(torch.ones(3, 2, 4), k, v, 2, window=2)
    assert out[:, 1, 3].tolist() == pytest.approx([4, 6, 9])
    v[0, 4, 0] = torch.nan  # the last row alone sees it
    out, _ = ref.attention(torch.ones(3, 2, 4), k, v, 2)
    assert out[:2].isfinite().all() and out[2, :, 0].isnan().all() and out[2, :, 1].isfinite().all()


def test_reference_pages():
    table, pages = ref.paged(np.random.default_rng(0), [0, 64, 10], [1, 1, 0])
    assert pages == 1 + 2 + 1 + 2 and (table >= 0).sum(1).tolist() == [1, 2, 1]
    cache = torch.arange(pages * 64.0).view(pages, 1, 64, 1)
    rows = ref.rows_of(table, 1, cache, 62, 66)[0, :, 0].tolist()
    a, b = table[1, 0].item() * 64, table[1, 1].item() * 64
    assert rows == [a + 62, a + 63, b, b + 1]
