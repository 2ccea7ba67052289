"""Rotary positions against the definition in 64 bits: layouts, parts of a head,
far positions, types, strides, both directions."""
import numpy as np
import pytest
import torch

import kv16_reference as ref
import speculative_decode_verify_w4a16_gb300 as sv
from helpers import dev

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
BANDS = {"kind": "bands", "factor": 8.0, "low": 1.0, "high": 4.0, "trained": 8192}
YARN = {"kind": "yarn", "factor": 16.0, "trained": 4096}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decode_verify_w4a16_gb300 import build
    build.build()


def _positions(rng, T):
    far = [0, 1, 131071, 2 ** 31 - 1, -1, -2 ** 31, 2 ** 24 + 1, 65536]
    p = rng.integers(0, 200000, T).astype(np.int32)
    p[:min(T, len(far))] = far[:T]
    return p


def _check(got, x, positions, angles, factor, interleaved, inverse=False):
    cos, sin = ref.cos_sin(positions, angles)
    y, mag = ref.rotate(x.reshape(len(positions), *x.shape[-2:]).cpu(), cos, sin, interleaved, factor, inverse)
    err = (got.cpu().double().reshape(y.shape) - y).abs()
    bound = ref.rotation_bound(y, mag, x.dtype)
    assert (err <= bound).all(), float((err / bound.clamp(min=1e-300)).max())
    rot = 2 * len(angles)
    assert torch.equal(got.cpu().reshape(y.shape)[..., rot:], x.cpu().reshape(y.shape)[..., rot:])


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,heads,D,rot,scaling", [
    (1, 1, 128, 128, None), (1, 72, 128, 128, BANDS), (17, 9, 64, 64, YARN), (80, 72, 128, 128, BANDS),
    (5, 3, 128, 32, None), (33, 40, 96, 48, YARN), (7, 2, 80, 80, None), (3, 5, 256, 64, BANDS), (65, 1, 16, 16, None),
    (9, 3, 24, 16, {"kind": "linear", "factor": 4}), (301, 11, 128, 64, {"kind": "ntk", "factor": 8}),
    (2, 3, 1024, 1024, None)])
def test_against_the_definition(dtype, interleaved, T, heads, D, rot, scaling):
    rng = np.random.default_rng(T + heads)
    x = torch.from_numpy(rng.standard_normal((T, heads, D)) * np.exp(rng.standard_normal(D))).to(dtype)
    positions = _positions(rng, T)
    angles, factor = sv.rope_angles(rot, 500000.0, scaling)
    freqs = sv.rope_frequencies(rot, 500000.0, scaling=scaling, interleaved=interleaved)
    p = torch.from_numpy(positions).to(dev())
    for inverse in (False, True):
        got = sv.rope(x.to(dev()), p, freqs, inverse=inverse)
        _check(got, x, positions, angles, factor, interleaved, inverse)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_slices_of_a_projection_in_place_and_apart(dtype):
    """q and k of a fused projection turned in one call; v, and the rows' other parts, stay."""
    rng = np.random.default_rng(4)
    B, n, H, Hkv, D = 3, 5, 8, 2, 128
    qkv = torch.from_numpy(rng.standard_normal((B, n, H + 2 * Hkv, D))).to(dtype)
    positions = rng.integers(0, 9999, (B, n)).astype(np.int32)
    angles, _ = sv.rope_angles(D)
    freqs = sv.rope_frequencies(D)
    p = torch.from_numpy(positions).to(dev())
    d = qkv.to(dev())
    x = d[:, :, 1:H + Hkv]
    apart = sv.rope(x, p, freqs)
    assert torch.equal(d.cpu(), qkv) and apart.is_contiguous() and apart.shape == x.shape
    _check(apart, qkv[:, :, 1:H + Hkv], positions.ravel(), angles, 1.0, False)
    into = torch.full((B, n, H + Hkv + 3, D), 7.0, dtype=dtype, device=dev())
    assert sv.rope(x, p, freqs, out=into[:, :, 2:H + Hkv + 1]).data_ptr() == into[:, :, 2:].data_ptr()
    assert torch.equal(into[:, :, 2:H + Hkv + 1], apart)
    assert (into[:, :, :2] == 7).all() and (into[:, :, H + Hkv + 1:] == 7).all()
    assert sv.rope(x, p, freqs, out=x) is x
    assert torch.equal(x, apart)
    assert torch.equal(d[:, :, :1].cpu(), qkv[:, :, :1]) and torch.equal(d[:, :, H + Hkv:].cpu(), qkv[:, :, H + Hkv:])


def test_relative_positions_alone_count():
    """q . k after the rotation depends on the positions' difference."""
    rng = np.random.default_rng(5)
    D = 128
    q, k = (torch.from_numpy(rng.standard_normal((1, 1, D))).float().to(dev()) for _ in range(2))
    freqs = sv.rope_frequencies(D, 500000.0)
    at = lambda x, p: sv.rope(x, torch.tensor([p], dtype=torch.int32, device=dev()), freqs).double()  # noqa: E731
    size = float(q.double().norm() * k.double().norm())
    want = float((at(q, 57) * at(k, 0)).sum())
    for p in (1, 1000, 131071, 10 ** 9):
        got = float((at(q, p + 57) * at(k, p)).sum())
        assert abs(got - want) <= 2 * 3e-7 * 2 * 1.42 * size  # both rows' errors, of both dot products


def test_gradient():
    """The rotation is linear: its gradient is the inverse rotation of the
    result's; against the formula and against differences."""
    rng = np.random.default_rng(6)
    T, heads, D, rot = 7, 3, 64, 32
    x, dy = (torch.from_numpy(rng.standard_normal((T, heads, D))).float() for _ in range(2))
    positions = rng.integers(0, 100000, T).astype(np.int32)
    p = torch.from_numpy(positions).to(dev())
    for interleaved in (False, True):
        freqs = sv.rope_frequencies(rot, scaling=YARN, interleaved=interleaved)
        angles, factor = sv.rope_angles(rot, scaling=YARN)
        cos, sin = ref.cos_sin(positions, angles)
        leaf = x.double().requires_grad_()
        c, s = cos[:, None] * factor, sin[:, None] * factor
        u, v = (leaf[..., 0:rot:2], leaf[..., 1:rot:2]) if interleaved else (leaf[..., :rot // 2], leaf[..., rot // 2:rot])
        a, b = u * c - v * s, v * c + u * s
        y = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
        torch.cat([y, leaf[..., rot:]], -1).backward(dy.double())
        got = sv.rope(dy.to(dev()), p, freqs, inverse=True)
        _, mag = ref.rotate(dy, cos, sin, interleaved, factor, True)
        assert ((got.cpu().double() - leaf.grad).abs() <= ref.rotation_bound(leaf.grad, mag, F32)).all()
        # <R x1 - R x0, dy> = <x1 - x0, R' dy>, exactly so for a linear map
        x1 = x + torch.from_numpy(rng.standard_normal(x.shape)).float()
        moved = sv.rope(x1.to(dev()), p, freqs).cpu().double() - sv.rope(x.to(dev()), p, freqs).cpu().double()
        left, right = float((moved * dy).sum()), float(((x1 - x).double() * got.cpu().double()).sum())
        assert abs(left - right) <= 4e-7 * factor * float((x1.abs() + x.abs()).double().norm() * dy.double().norm()) * 2
        back = sv.rope(sv.rope(x.to(dev()), p, freqs), p, freqs, inverse=True).cpu().double() / 1.0
        scale = torch.ones(D, dtype=torch.float64)
        scale[:rot] = factor ** 2
        assert (back - x.double() * scale).abs().max() <= 1e-5


def test_no_rows():
    freqs = sv.rope_frequencies(64)
    x = torch.empty(0, 4, 64, dtype=BF16, device=dev())
    assert sv.rope(x, torch.empty(0, dtype=torch.int32, device=dev()), freqs).shape == (0, 4, 64)


def test_a_stream_and_a_graph():
    rng = np.random.default_rng(8)
    x = torch.from_numpy(rng.standard_normal((64, 8, 128))).to(BF16).to(dev())
    p = torch.arange(64, dtype=torch.int32, device=dev())
    freqs = sv.rope_frequencies(128)
    want = sv.rope(x, p, freqs)
    s, out = torch.cuda.Stream(), torch.zeros_like(x)
    torch.cuda.synchronize()
    sv.rope(x, p, freqs, out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = sv.rope(x, p, freqs)
    x.neg_()
    p.add_(3)
    g.replay()
    assert torch.equal(y, sv.rope(x, p, freqs)) and not torch.equal(y, want)


def test_refusals():
    x = torch.zeros(4, 3, 64, dtype=BF16, device=dev())
    p = torch.zeros(4, dtype=torch.int32, device=dev())
    f = sv.rope_frequencies(64)
    for bad in (lambda: sv.rope(x.double(), p, f), lambda: sv.rope(x, p.long(), f), lambda: sv.rope(x, p[:3], f),
                lambda: sv.rope(x.cpu(), p, f), lambda: sv.rope(x, p.cpu(), f), lambda: sv.rope(x[0], p, f),
                lambda: sv.rope(x, p, sv.rope_frequencies(128)), lambda: sv.rope(x.transpose(1, 2), p, f),
                lambda: sv.rope(x[:1].expand(4, 3, 64), p, f), lambda: sv.rope(x, p, f, out=x.float()),
                lambda: sv.rope(x, p, f, out=x[:2]), lambda: sv.rope(x, p, sv.rope_frequencies(64, device="cpu")),
                lambda: sv.rope(x.view(2, 2, 3, 64)[:, :1], p[:2], f)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(sv.W4A16Error):  # not 16-byte aligned
        sv.rope(torch.zeros(4 * 3 * 64 + 1, dtype=BF16, device=dev())[1:].view(4, 3, 64), p, f)
    with pytest.raises(sv.W4A16Error):  # a width that is not a multiple of 8
        sv.rope(torch.zeros(1, 3, 68, dtype=BF16, device=dev()), p[:1], f)
