"""Sizes that do not fit the C interface's int: the binding refuses them (no GPU
needed: stand-ins with the shapes and strides of such tensors)."""
import types

import pytest
import torch

from speculative_decode_verify_w4a16_gb300 import _lib, api
from speculative_decode_verify_w4a16_gb300 import build as sv_build

BIG = 2 ** 32 + 4


def stand_in(*shape, dtype=torch.bfloat16):
    strides = [1]
    for n in reversed(shape[1:]):
        strides.insert(0, strides[0] * n)
    return types.SimpleNamespace(shape=shape, stride=lambda: tuple(strides), dtype=dtype, is_cuda=True, device="cuda:0",
                                 get_device=lambda: 0, is_contiguous=lambda: True, dim=lambda: len(shape),
                                 numel=lambda: shape[0] * strides[0])


@pytest.mark.parametrize("shape", [(4, 2, 64), (2 ** 31 - 1, 1, 8), (1, 2, 64), (2, 2, 2, 64), (3, 1, 2, 64), (0, 2, 64)])
def test_rows_that_fit(shape):
    rows = shape[0] * shape[1] if len(shape) == 4 else shape[0]
    assert api._rows(stand_in(*shape), "x", 0) == (rows, shape[-2], shape[-1], shape[-2] * shape[-1])


@pytest.mark.parametrize("shape", [(BIG, 2, 64), (2 ** 31, 1, 8), (2, BIG, 8), (2, 1, BIG), (1, BIG, 8), (2 ** 16, 2 ** 16 + 1, 1, 8),
                                   (2 ** 32, 1, 1, 8)])
def test_rows_that_do_not(shape):
    with pytest.raises(ValueError):
        api._rows(stand_in(*shape), "x", 0)


def test_tables_that_do_not():
    i32 = torch.int32
    assert api._need_step(stand_in(2, 70, dtype=i32), stand_in(2, dtype=i32), None, 4, 0) == (2, 70)
    for B, blocks in ((1, BIG), (BIG, 1), (2, 2 ** 31)):
        with pytest.raises(ValueError):
            api._need_step(stand_in(B, blocks, dtype=i32), stand_in(B, dtype=i32), None, B, 0)


def test_workspace_of_no_call():
    sv_build.build()
    for sizes in ((BIG, 8, 2, 128), (4, BIG, 1, 128), (4, 8, 2, 2 ** 32 + 128)):
        assert api.kv16_attention_workspace_bytes(*sizes) == 0


@pytest.mark.parametrize("window,passed", [(0, 0), (5, 5), (2 ** 31 - 1, 2 ** 31 - 1), (-1, -1), (BIG, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1),
                                           (-2 ** 32 + 5, -1), (-2 ** 31 - 1, -1)])
def test_windows(monkeypatch, window, passed):
    """A window that no int holds is past every position, not its lower bits."""
    got = []
    monkeypatch.setattr(api, "_device", lambda: 0)
    monkeypatch.setattr(api, "lib", lambda: types.SimpleNamespace(kv16_attention=lambda *a: got.append(a[14]) or _lib.OK))
    tensors = {}
    for name, t in (("q", stand_in(2, 4, 64)), ("k", stand_in(1, 3, 2, 64, 64)), ("table", stand_in(2, 1, dtype=torch.int32)),
                    ("lens", stand_in(2, dtype=torch.int32)), ("ws", stand_in(256, dtype=torch.uint8))):
        t.data_ptr = lambda: 256
        tensors[name] = t
    c = types.SimpleNamespace(k=tensors["k"], v=tensors["k"])
    api.kv16_attention(tensors["q"], c, 0, tensors["table"], tensors["lens"], window=window, out=tensors["q"],
                       ws=tensors["ws"], stream=types.SimpleNamespace(cuda_stream=0))
    assert got == [passed]


@pytest.mark.parametrize("scaling", [{"kind": "ntk", "factor": 1e305}, {"kind": "ntk", "factor": 1e306},
                                     {"kind": "linear", "factor": 1e-320},
                                     {"kind": "bands", "factor": 1e-320, "low": 1, "high": 4, "trained": 10},
                                     {"kind": "yarn", "factor": 1e-320, "trained": 4096}])
def test_frequencies_that_no_number_holds(scaling):
    for f in (api.rope_angles, lambda *a, **k: api.rope_frequencies(*a, device="cpu", **k)):
        with pytest.raises(ValueError):
            f(64, 10000.0, scaling=scaling)


@pytest.mark.parametrize("scaling", [{"kind": "ntk", "factor": 1e200}, {"kind": "linear", "factor": 1e-200}])
def test_frequencies_of_any_size(scaling):
    assert api.rope_frequencies(64, 10000.0, scaling=scaling, device="cpu").rot == 64
