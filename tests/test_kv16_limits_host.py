"""The sizes that the paged 16-bit attention refuses because its split could not count them (no GPU needed)."""
import pytest

from speculative_decode_verify_w4a16_gb300 import _lib
from speculative_decode_verify_w4a16_gb300 import build as sv_build
from test_kv16_host import P, UNSUPPORTED


@pytest.mark.parametrize("T,B,H,Hkv,max_blocks", [
    (4, 1, 1025, 1, 4),               # a group of more than 1024 heads
    (4, 1, 8, 1, (1 << 21) + 1),      # more blocks than that
    (1 << 20, 16, 1024, 1, 1 << 21),  # 2^22 units of 1024 heads over 2^27 keys, times their weight 8: 2^62
])
def test_what_the_split_cannot_count(T, B, H, Hkv, max_blocks):
    sv_build.build()
    L = _lib.lib()
    assert L.kv16_attention(P, H * 128, P, P, P, P, P, T, B, H, Hkv, 128, max_blocks, 9, 0, 0.1, 0, P, None, 0,
                            None) == UNSUPPORTED
