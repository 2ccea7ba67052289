"""Rotation and paged 16-bit cache: a size beyond what the header states is refused
with the code that the header gives it (no GPU needed)."""
import pytest

from speculative_decode_verify_w4a16_gb300 import _lib
from speculative_decode_verify_w4a16_gb300 import build as sv_build
from test_kv16_host import BAD, OTHER, P, UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    sv_build.build()
    return _lib.lib()


@pytest.mark.parametrize("kw,status", [
    (dict(T=1 << 20, H=2048, Hkv=2), UNSUPPORTED), (dict(T=1 << 24, H=128, Hkv=1), UNSUPPORTED),  # T * H = 2^31
    (dict(T=1 << 24, H=256, Hkv=1), UNSUPPORTED), (dict(T=2, H=2 ** 30, Hkv=1 << 15), UNSUPPORTED),
    (dict(T=(1 << 24) + 4), UNSUPPORTED), (dict(B=4097), UNSUPPORTED), (dict(max_blocks=(1 << 21) + 1), UNSUPPORTED),
    (dict(H=65536, Hkv=65536), BAD), (dict(max_blocks=1 << 25), BAD), (dict(B=1 << 11, max_blocks=1 << 20), BAD),
    (dict(pages=1 << 24, Hkv=4), BAD),
])
def test_attention(L, kw, status):
    a = dict(T=4, B=2, H=8, Hkv=2, D=128, max_blocks=4, pages=9)
    a.update(kw)
    T, B, H, Hkv, D = (a[x] for x in ("T", "B", "H", "Hkv", "D"))
    assert L.kv16_attention(P, H * D, P, P, P, P, P, T, B, H, Hkv, D, a["max_blocks"], a["pages"], 0, 0.1, 0, P, None, 0,
                            None) == status
    if not {"B", "max_blocks", "pages"} & set(kw):
        assert L.kv16_attention_workspace_bytes(T, H, Hkv, D) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(heads=(1 << 20) + 1), UNSUPPORTED), (dict(D=1032), UNSUPPORTED), (dict(D=132), UNSUPPORTED),
    (dict(rot=24), UNSUPPORTED), (dict(rot=0), BAD), (dict(rot=144), BAD), (dict(T=-1), BAD),
])
def test_rotation(L, kw, status):
    a = dict(T=4, heads=8, D=128, rot=128)
    a.update(kw)
    stride = -(-a["heads"] * a["D"] // 8) * 8
    assert L.rope_rotate(P, stride, P, P, a["T"], a["heads"], a["D"], a["rot"], 0, 1.0, 0, 0, OTHER, stride, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(H=(1 << 20) + 1), UNSUPPORTED), (dict(T=(1 << 24) + 2), UNSUPPORTED), (dict(B=4097), UNSUPPORTED),
    (dict(D=80), UNSUPPORTED), (dict(rot=24), UNSUPPORTED), (dict(Hkv=65536), BAD), (dict(pages=1 << 25), BAD),
    (dict(max_blocks=1 << 25), BAD),
])
def test_append(L, kw, status):
    a = dict(T=6, B=2, H=8, Hkv=2, D=128, max_blocks=4, pages=9, rot=64)
    a.update(kw)
    T, B, H, Hkv, D = (a[x] for x in ("T", "B", "H", "Hkv", "D"))
    assert L.kv16_append(P, P, Hkv * D, Hkv * D, P, H * D, P, a["rot"], 0, 1.0, P, P, P, T, B, H, Hkv, D, a["max_blocks"],
                         a["pages"], 0, P, P, OTHER, H * D, None) == status


@pytest.mark.parametrize("scale,status", [(3e38, BAD), (2.4e38, BAD), (1e38, UNSUPPORTED), (1e-30, UNSUPPORTED), (0.0, BAD),
                                          (-1.0, BAD), (float("inf"), BAD), (float("nan"), BAD)])
def test_scales(L, scale, status):
    """Scales whose product with log2(e) fp32 does not hold would give NaN (4097 requests, so that no good call launches)."""
    assert L.kv16_attention(P, 1024, P, P, P, P, P, 8, 4097, 8, 2, 128, 4, 9, 0, scale, 0, P, None, 0, None) == status


def test_out_in_place_of_queries_that_are_not_dense(L):
    """The output is dense: over a slice of a fused projection its rows would lie on queries that are still to be read.
    (Nothing launches: the calls that are not refused for that have no workspace, where there is a GPU, or no device.)"""
    def attn(q, stride, out, T=6):
        return L.kv16_attention(q, stride, P, P, P, P, P, T, 2, 8, 2, 128, 4, 9, 0, 0.1, 0, out, None, 0, None)
    assert attn(P, 1536, P) == BAD
    for q, stride, out, T in ((P, 1024, P, 6), (P, 1536, OTHER, 6), (P, 1536, P, 1)):
        assert attn(q, stride, out, T) in (_lib.ERR_WORKSPACE, _lib.ERR_CUDA)
