"""Values and keys that are not finite, where some rows see them and others do not:
every infinity with its sign, every NaN, in whole units, cut ones and with windows."""
import pytest
import torch

import kv16_reference as ref
import speculative_decode_verify_w4a16_gb300 as sv
from helpers import dev
from test_kv16_gpu import BF16, F16, Case, _starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decode_verify_w4a16_gb300 import build
    build.build()


def _check(c, out, window=0):
    """As Case.check, and what is not finite by what it is."""
    c.check(out, window)
    at = _starts(c.counts)
    for b, (k, v) in enumerate(c.kv):
        want, _ = ref.attention(c.q[at[b]:at[b + 1]], k, v, c.lens[b], window)
        got = out[at[b]:at[b + 1]]
        for what in (torch.isnan, torch.isposinf, torch.isneginf):
            assert torch.equal(what(got), what(want)), (b, what)
    return out


def _run(c, **kw):
    for b in range(len(c.lens)):
        c.put(b)
    out = c.run(**kw)
    torch.cuda.synchronize()
    assert sv.check_device_status() == 0
    return out


# whole units of both kinds, pieces, many units
SHAPES = [(70, 9), (0, 200), (40, 300), (20000, 5), (9000, 300), (30000, 40)]


@pytest.mark.parametrize("dtype,D,H,Hkv", [(BF16, 128, 8, 2), (F16, 64, 4, 4), (F16, 128, 3, 1)])
@pytest.mark.parametrize("past,n", SHAPES)
def test_values_among_the_step_s_own(dtype, D, H, Hkv, past, n):
    """In tiles that the first rows do not see whole: an infinity, the other one, both of them, and NaN."""
    c = Case(n, dtype, D, H, Hkv, [past], [n])
    k, v = c.kv[0]
    for at, col, x in ((0, 1, torch.inf), (n // 3, 2, -torch.inf), (n // 3, 33, torch.inf), (n // 2, 33, -torch.inf),
                       (n // 2, 5, torch.nan), (n - 1, 60, torch.inf), (n - 2, 63, -torch.inf)):
        v[0, past + at, col] = x
    v[Hkv - 1, past + 2 * n // 3, 7] = -torch.inf
    _check(c, _run(c))


@pytest.mark.parametrize("window", [64, 100, 1000])
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F16, 64)])
@pytest.mark.parametrize("past,n", [(0, 200), (1000, 300), (300, 40), (5000, 5)])
def test_values_where_a_window_ends(window, dtype, D, past, n):
    """Seen by the first rows and no longer by the last."""
    c = Case(window, dtype, D, 6, 2, [past], [n])
    k, v = c.kv[0]
    for at, col, x in ((past - window + n // 3, 1, torch.inf), (past - window + n // 2, 2, -torch.inf),
                       (past - window + n // 2, 3, torch.nan), (past + n // 4, 4, torch.inf), (past - window, 5, -torch.inf)):
        if at >= 0:
            v[0, at, col] = x
    _check(c, _run(c, window=window), window)


@pytest.mark.parametrize("H,Hkv,n", [(8, 2, 300), (4, 1, 9), (6, 3, 40)])
def test_a_key_that_is_not_a_number(H, Hkv, n):
    """Rows from it on, of its head's group, are NaN, and no others."""
    c = Case(n, BF16, 128, H, Hkv, [70], [n])
    c.kv[0][0][0, 70 + n // 2, 3] = torch.nan
    out = _run(c)
    group = H // Hkv
    assert out[n // 2:, :group].isnan().all()
    assert out[:n // 2].isfinite().all() and out[:, group:].isfinite().all()
    _check(c, out)


@pytest.mark.parametrize("past,n", [(70, 9), (20000, 5), (9000, 300)])
def test_infinite_keys(past, n):
    """A key whose scores are infinite: of weight zero to rows that they are negative for, NaN to the others."""
    c = Case(n, BF16, 128, 4, 1, [past], [n])
    k, v = c.kv[0]
    k[0, past + n // 2, 9] = torch.inf
    c.q[..., 9] = torch.where(torch.arange(n, device=dev())[:, None] % 2 == 0, -1.0, 1.0).to(BF16)
    out = _run(c)
    odd = torch.arange(n, device=dev()) % 2 == 1
    assert out[n // 2:][odd[n // 2:]].isnan().all() and out[~odd].isfinite().all()
    _check(c, out)
