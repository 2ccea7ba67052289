"""Python binding of libw4a16sv: argument marshalling from torch tensors to the
C ABI (include/w4a16sv.h). PyTorch supplies device memory and the current
CUDA stream; every step of the computation runs in the library's kernels.
"""
from __future__ import annotations

import contextlib
from dataclasses import dataclass
from functools import lru_cache
from typing import Optional

import torch

from ._lib import W4A16Error, check, lib

GROUP = 128

# the current device's index, its current stream's handle, and whether that is
# being captured, without the lookups that the public functions add (a torch
# without CUDA has none of them)
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: True)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda i: torch.cuda.current_stream(i).cuda_stream)


def _stream(stream: Optional[torch.cuda.Stream] = None) -> int:
    if stream is not None:
        return int(stream.cuda_stream)
    return _raw_stream(_device())


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, shape=None):
    if (t.dtype is dtype and t.is_contiguous() and t.is_cuda and t.get_device() == _device()
            and (shape is None or t.shape == shape)):
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device.index != torch.cuda.current_device():
        # the library launches on, and keeps its state for, the current device
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{torch.cuda.current_device()}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


# --------------------------------------------------------------- workspace
_ws_cache: dict = {}


def workspace(nbytes: int, device: Optional[torch.device] = None, key: str = "default") -> torch.Tensor:
    """A zero-filled scratch buffer of at least nbytes on `device`, cached per
    (device, key). The kernels leave it zeroed after every call. The linears,
    the accept step and tree_attention take theirs from here by default: calls
    that may overlap, on several streams, need a `ws` each."""
    index = None if device is None else (device if isinstance(device, torch.device) else torch.device(device)).index
    k = (_device() if index is None else index, key)
    buf = _ws_cache.get(k)
    if buf is None or buf.numel() < nbytes:
        dev = torch.device("cuda", k[0])
        buf = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=dev)
        _ws_cache[k] = buf
    return buf


_stream_ws: dict = {}


def _stream_workspace(nbytes: int, key: str, stream=None) -> torch.Tensor:
    """The default workspace of a call on `stream` (default: the current one):
    zero-filled on that stream, and kept for it, so that calls on several
    streams share nothing. Within a graph capture it is the capture's own,
    zeroed by the graph: a captured graph holds no address of a buffer that a
    later call might replace, and an eager call none that only a graph zeroes."""
    raw = _stream(stream)
    capture = lib().w4a16_stream_capture_id(raw) if stream is not None or _capturing() else 0
    k = (_device(), raw, key, capture != 0)
    kept = _stream_ws.get(k)
    if kept is not None and kept[0] == capture and kept[1].numel() >= nbytes:
        return kept[1]
    with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
        buf = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=torch.device("cuda", k[0]))
    _stream_ws[k] = (capture, buf)
    return buf


# ------------------------------------------------------------------ format

def packed_weight_bytes(N: int, K: int) -> int:
    return int(lib().w4a16_packed_weight_bytes(N, K))


def packed_scale_bytes(N: int, K: int) -> int:
    return int(lib().w4a16_packed_scale_bytes(N, K))


def quantize(w: torch.Tensor, stream=None):
    """w fp32 [N, K] (CUDA) -> canonical (qweight int32 [N, K/8] holding the
    uint32 words, scales fp16 [N, K/128])."""
    _need(w, "w", torch.float32)
    N, K = w.shape
    qw = torch.empty((N, K // 8), dtype=torch.int32, device=w.device)
    sc = torch.empty((N, K // GROUP), dtype=torch.float16, device=w.device)
    check(lib().w4a16_quantize(_ptr(w), N, K, _ptr(qw), _ptr(sc), _stream(stream)), "w4a16_quantize")
    return qw, sc


@dataclass
class PackedWeight:
    """A prepacked W4A16 weight (N x K) ready for linear()."""
    N: int
    K: int
    qweight: torch.Tensor  # uint8 [N*K/2], streaming layout
    scales: torch.Tensor   # uint8 [N*K/64], streaming layout

    @property
    def nbytes(self) -> int:
        return self.qweight.numel() + self.scales.numel()


def prepack(qweight: torch.Tensor, scales: torch.Tensor, stream=None) -> PackedWeight:
    """Canonical (qweight int32/uint32 [N, K/8], scales fp16 [N, K/128]) -> PackedWeight."""
    if qweight.dtype not in (torch.int32, torch.uint32):
        raise ValueError("qweight must hold 32-bit words")
    _need(qweight, "qweight", qweight.dtype)
    _need(scales, "scales", torch.float16)
    N, K8 = qweight.shape
    K = K8 * 8
    if tuple(scales.shape) != (N, K // GROUP):
        raise ValueError("scales shape mismatch")
    qp = torch.empty(packed_weight_bytes(N, K), dtype=torch.uint8, device=qweight.device)
    sp = torch.empty(packed_scale_bytes(N, K), dtype=torch.uint8, device=qweight.device)
    if qp.numel() == 0:
        raise W4A16Error(1, "w4a16_prepack: N and K must be positive multiples of 128")
    check(lib().w4a16_prepack(_ptr(qweight), _ptr(scales), N, K, _ptr(qp), _ptr(sp), _stream(stream)),
          "w4a16_prepack")
    return PackedWeight(N, K, qp, sp)


# ------------------------------------------------------------------ linear

def linear_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib().w4a16_linear_workspace_bytes(M, N, K))


def linear(x: torch.Tensor, w: PackedWeight, out: Optional[torch.Tensor] = None,
           ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out[M, N] = bf16(x[M, K] . W^T) with W the dequantised int4 weight."""
    _need(x, "x", torch.bfloat16)
    M, K = x.shape
    if K != w.K:
        raise ValueError(f"x has K={K}, weight has K={w.K}")
    if out is None:
        out = torch.empty((M, w.N), dtype=torch.bfloat16, device=x.device)
    _need(out, "out", torch.bfloat16, (M, w.N))
    if ws is None:
        ws = workspace(linear_workspace_bytes(M, w.N, K), x.device, "linear")
    check(lib().w4a16_linear(_ptr(x), M, K, _ptr(w.qweight), _ptr(w.scales), w.N, _ptr(out), _ptr(ws),
                             ws.numel(), _stream(stream)), "w4a16_linear")
    return out


def linear_noalloc(x: torch.Tensor, w: PackedWeight, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """linear() without a workspace: the library uses its static device scratch
    (see w4a16_linear_noalloc in the header for the rules on sharing it)."""
    _need(x, "x", torch.bfloat16)
    M, K = x.shape
    if K != w.K:
        raise ValueError(f"x has K={K}, weight has K={w.K}")
    if out is None:
        out = torch.empty((M, w.N), dtype=torch.bfloat16, device=x.device)
    _need(out, "out", torch.bfloat16, (M, w.N))
    check(lib().w4a16_linear_noalloc(_ptr(x), M, K, _ptr(w.qweight), _ptr(w.scales), w.N, _ptr(out),
                                     _stream(stream)), "w4a16_linear_noalloc")
    return out


def linear_logits_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib().w4a16_linear_logits_workspace_bytes(M, N, K))


def linear_logits(x: torch.Tensor, w: PackedWeight, logits: Optional[torch.Tensor] = None,
                  stats: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None):
    """The lm_head of the verify pass with fused softmax statistics:
    returns (logits fp32 [M, N], stats fp32 [M, N/32, 2] = (max, sum exp(l - max))
    per 32-logit slice)."""
    _need(x, "x", torch.bfloat16)
    M, K = x.shape
    if K != w.K:
        raise ValueError(f"x has K={K}, weight has K={w.K}")
    if logits is None:
        logits = torch.empty((M, w.N), dtype=torch.float32, device=x.device)
    if stats is None:
        stats = torch.empty((M, w.N // 32, 2), dtype=torch.float32, device=x.device)
    _need(logits, "logits", torch.float32, (M, w.N))
    _need(stats, "stats", torch.float32, (M, w.N // 32, 2))
    if ws is None:
        ws = workspace(linear_logits_workspace_bytes(M, w.N, K), x.device, "linear")
    check(lib().w4a16_linear_logits(_ptr(x), M, K, _ptr(w.qweight), _ptr(w.scales), w.N, _ptr(logits), _ptr(stats),
                                    _ptr(ws), ws.numel(), _stream(stream)), "w4a16_linear_logits")
    return logits, stats


# ------------------------------------------------------------------ accept

def accept_workspace_bytes(B: int, n: int, V: int) -> int:
    return int(lib().spec_accept_workspace_bytes(B, n, V))


def spec_accept(p_logits: torch.Tensor, draft_ids: torch.Tensor, q_logits: Optional[torch.Tensor] = None,
                tree_parents: Optional[torch.Tensor] = None, uniforms: Optional[torch.Tensor] = None,
                accepted_len: Optional[torch.Tensor] = None, next_token: Optional[torch.Tensor] = None,
                ws: Optional[torch.Tensor] = None, stream=None):
    """Speculative accept step; see the header for the three modes.
    Returns (accepted_len int32 [B], next_token int32 [B])."""
    _need(p_logits, "p_logits", torch.float32)
    _need(draft_ids, "draft_ids", torch.int32)
    B, rows, V = p_logits.shape
    if tree_parents is not None:
        n = rows
        _need(tree_parents, "tree_parents", torch.int32, (B, n))
        _need(draft_ids, "draft_ids", torch.int32, (B, n))
    else:
        n = rows - 1
        _need(draft_ids, "draft_ids", torch.int32, (B, n))
    if q_logits is not None:
        _need(q_logits, "q_logits", torch.float32, (B, n, V))
    if uniforms is not None:  # stochastic tree: [B, n] (u_0 draws); sequence: [B, n + 1]
        _need(uniforms, "uniforms", torch.float32, (B, n) if tree_parents is not None else (B, n + 1))
    if accepted_len is None:
        accepted_len = torch.empty(B, dtype=torch.int32, device=p_logits.device)
    if next_token is None:
        next_token = torch.empty(B, dtype=torch.int32, device=p_logits.device)
    if ws is None:
        ws = workspace(accept_workspace_bytes(B, n, V), p_logits.device, "accept")
    check(lib().spec_accept(_ptr(p_logits), _ptr(q_logits), _ptr(draft_ids), _ptr(tree_parents), _ptr(uniforms),
                            B, n, V, _ptr(accepted_len), _ptr(next_token), _ptr(ws), ws.numel(),
                            _stream(stream)), "spec_accept")
    return accepted_len, next_token


def spec_accept_prestat(p_logits: torch.Tensor, p_stats: torch.Tensor, draft_ids: torch.Tensor,
                        q_logits: torch.Tensor, uniforms: torch.Tensor, accepted_len: Optional[torch.Tensor] = None,
                        next_token: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None):
    """Stochastic sequence accept with the target rows' statistics supplied
    (p_stats [B, n+1, V/32, 2] from linear_logits). Returns (accepted_len, next_token)."""
    _need(p_logits, "p_logits", torch.float32)
    B, n1, V = p_logits.shape
    n = n1 - 1
    _need(p_stats, "p_stats", torch.float32, (B, n1, V // 32, 2))
    _need(draft_ids, "draft_ids", torch.int32, (B, n))
    _need(q_logits, "q_logits", torch.float32, (B, n, V))
    _need(uniforms, "uniforms", torch.float32, (B, n + 1))
    if accepted_len is None:
        accepted_len = torch.empty(B, dtype=torch.int32, device=p_logits.device)
    if next_token is None:
        next_token = torch.empty(B, dtype=torch.int32, device=p_logits.device)
    if ws is None:
        ws = workspace(accept_workspace_bytes(B, n, V), p_logits.device, "accept")
    check(lib().spec_accept_prestat(_ptr(p_logits), _ptr(p_stats), _ptr(q_logits), _ptr(draft_ids), _ptr(uniforms),
                                    B, n, V, _ptr(accepted_len), _ptr(next_token), _ptr(ws), ws.numel(),
                                    _stream(stream)), "spec_accept_prestat")
    return accepted_len, next_token


def spec_accept_node(p_logits: torch.Tensor, draft_ids: torch.Tensor, q_logits: Optional[torch.Tensor] = None,
                     tree_parents: Optional[torch.Tensor] = None, uniforms: Optional[torch.Tensor] = None,
                     ws: Optional[torch.Tensor] = None, stream=None):
    """spec_accept that also returns the accepted node:
    (accepted_len, next_token, accepted_node), int32 [B] each."""
    _need(p_logits, "p_logits", torch.float32)
    B, rows, V = p_logits.shape
    n = rows if tree_parents is not None else rows - 1
    _need(draft_ids, "draft_ids", torch.int32, (B, n))
    if tree_parents is not None:
        _need(tree_parents, "tree_parents", torch.int32, (B, n))
    if q_logits is not None:
        _need(q_logits, "q_logits", torch.float32, (B, n, V))
    if uniforms is not None:
        _need(uniforms, "uniforms", torch.float32, (B, n) if tree_parents is not None else (B, n + 1))
    acc, nxt, node = (torch.empty(B, dtype=torch.int32, device=p_logits.device) for _ in range(3))
    if ws is None:
        ws = workspace(accept_workspace_bytes(B, n, V), p_logits.device, "accept")
    check(lib().spec_accept_node(_ptr(p_logits), _ptr(q_logits), _ptr(draft_ids), _ptr(tree_parents),
                                 _ptr(uniforms), B, n, V, _ptr(acc), _ptr(nxt), _ptr(node), _ptr(ws), ws.numel(),
                                 _stream(stream)), "spec_accept_node")
    return acc, nxt, node


# ------------------------------------------------------ verify attention

def tree_attention_workspace_bytes(B: int, n: int, H: int, Hkv: int, D: int, Lcap: int, max_len: int) -> int:
    return int(lib().tree_attention_workspace_bytes(B, n, H, Hkv, D, Lcap, max_len))


def tree_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, lens: torch.Tensor,
                   tree_parents: Optional[torch.Tensor] = None, max_len: Optional[int] = None,
                   scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                   ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Tree-masked verify attention. q bf16 [B, n, H, D]; caches bf16
    [B, Hkv, Lcap, D] (prefix at 0..lens-1, the tree nodes at lens..lens+n-1);
    lens int32 [B]; tree_parents int32 [B, n] or None (chain); max_len: an
    upper bound of lens (default Lcap - n). Returns bf16 [B, n, H, D]."""
    _need(q, "q", torch.bfloat16)
    B, n, H, D = q.shape
    _need(k_cache, "k_cache", torch.bfloat16)
    Hkv, Lcap = k_cache.shape[1], k_cache.shape[2]
    _need(k_cache, "k_cache", torch.bfloat16, (B, Hkv, Lcap, D))
    _need(v_cache, "v_cache", torch.bfloat16, (B, Hkv, Lcap, D))
    _need(lens, "lens", torch.int32, (B,))
    if tree_parents is not None:
        _need(tree_parents, "tree_parents", torch.int32, (B, n))
    max_len = Lcap - n if max_len is None else int(max_len)
    scale = D ** -0.5 if scale is None else float(scale)
    if out is None:
        out = torch.empty((B, n, H, D), dtype=torch.bfloat16, device=q.device)
    _need(out, "out", torch.bfloat16, (B, n, H, D))
    nbytes = tree_attention_workspace_bytes(B, n, H, Hkv, D, Lcap, max_len)
    if ws is None and nbytes > 0:
        ws = workspace(nbytes, q.device, "attention")
    check(lib().tree_attention(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(lens), _ptr(tree_parents), B, n, H, Hkv,
                               D, Lcap, max_len, scale, _ptr(out), _ptr(ws), 0 if ws is None else ws.numel(),
                               _stream(stream)), "tree_attention")
    return out


def kv_compact(k_cache: torch.Tensor, v_cache: torch.Tensor, lens: torch.Tensor, accepted_node: torch.Tensor,
               tree_parents: Optional[torch.Tensor] = None, n: Optional[int] = None,
               new_lens: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Moves the accepted root path's keys/values to lens..lens+depth in
    place. Caches bf16 [layers, B, Hkv, Lcap, D] (or [B, Hkv, Lcap, D]);
    tree_parents [B, n] or None (chain, then n is required). Returns new_lens."""
    _need(k_cache, "k_cache", torch.bfloat16)
    kc, vc = (k_cache, v_cache) if k_cache.dim() == 5 else (k_cache.unsqueeze(0), v_cache.unsqueeze(0))
    layers, B, Hkv, Lcap, D = kc.shape
    _need(vc, "v_cache", torch.bfloat16, (layers, B, Hkv, Lcap, D))
    _need(lens, "lens", torch.int32, (B,))
    _need(accepted_node, "accepted_node", torch.int32, (B,))
    if tree_parents is not None:
        n = tree_parents.shape[1]
        _need(tree_parents, "tree_parents", torch.int32, (B, n))
    elif n is None:
        raise ValueError("n is required for a sequence draft")
    if new_lens is None:
        new_lens = torch.empty(B, dtype=torch.int32, device=lens.device)
    check(lib().kv_compact(_ptr(kc), _ptr(vc), _ptr(lens), _ptr(tree_parents), _ptr(accepted_node), B, int(n), Hkv,
                           D, Lcap, layers, _ptr(new_lens), _stream(stream)), "kv_compact")
    return new_lens


def check_device_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device error status."""
    return int(lib().w4a16_check_device_status(_stream(stream)))


# ------------------------------------------------------ paged 8-bit cache

KV_BLOCK = 64  # tokens per block (a page, a scale)
_KV8_FORMATS = {torch.float8_e4m3fn: 0, torch.float8_e5m2: 1}


@dataclass
class KV8Cache:
    """Keys and values of full 64-token blocks in 8 bits, code * scale with a
    scale per (block, head), and the blocks being filled in bf16 tail pages
    (in pairs; see the header). The leading dimension is the layer."""
    k: torch.Tensor        # float8_e4m3fn or float8_e5m2 [layers, pages, Hkv, 64, D]
    v: torch.Tensor
    k_scale: torch.Tensor  # fp32 [layers, pages, Hkv]
    v_scale: torch.Tensor
    k_tail: torch.Tensor   # bf16 [layers, tail_pages, Hkv, 64, D]
    v_tail: torch.Tensor

    @property
    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size()
                   for t in (self.k, self.v, self.k_scale, self.v_scale, self.k_tail, self.v_tail))


@dataclass
class BlockPlan:
    """What kv_block_plan leaves for kv8_append and for the next step."""
    new_lens: torch.Tensor   # int32 [B]
    new_tails: torch.Tensor  # int32 [B]
    new_start: torch.Tensor  # int32 [B + 1]: kept rows before each request
    queue: torch.Tensor      # int32 [3]: ring head, free pages, pages missing
    src_rows: torch.Tensor   # int32 [rows]: source row of each kept row, -1 behind
    slots: torch.Tensor      # int32 [rows]: its place (page * 64 + offset, or -1 - tail row)


def kv8_cache(layers: int, pages: int, B: int, Hkv: int, D: int = 128, dtype: torch.dtype = torch.float8_e4m3fn,
              device=None) -> KV8Cache:
    """An empty cache of `pages` pages, with a pair of tail pages for each of B requests."""
    if dtype not in _KV8_FORMATS:
        raise ValueError("dtype must be torch.float8_e4m3fn or torch.float8_e5m2")
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    codes = [torch.zeros((layers, pages, Hkv, KV_BLOCK, D), dtype=torch.uint8, device=dev).view(dtype)
             for _ in range(2)]
    scales = [torch.ones((layers, pages, Hkv), dtype=torch.float32, device=dev) for _ in range(2)]
    tails = [torch.zeros((layers, 2 * B, Hkv, KV_BLOCK, D), dtype=torch.bfloat16, device=dev) for _ in range(2)]
    return KV8Cache(*codes, *scales, *tails)


def _is(t: torch.Tensor, dtype: torch.dtype, dev: int, shape) -> bool:
    """What _need accepts, for the calls of a decode step: _need says what is
    wrong with the rest."""
    return t.dtype is dtype and t.get_device() == dev and t.shape == shape and t.is_contiguous()


def _need_ws(ws: torch.Tensor, dev: int):
    if ws.get_device() != dev:
        raise ValueError(f"ws is on {ws.device}, the current device is cuda:{dev}")


def _need_cache(c: KV8Cache, dev: int):
    k, k_tail = c.k, c.k_tail
    shape = k.shape
    layers, pages, Hkv, block, D = shape
    dtype = k.dtype
    if dtype not in _KV8_FORMATS:
        raise ValueError("the cache's codes must be torch.float8_e4m3fn or torch.float8_e5m2")
    if block != KV_BLOCK:
        raise ValueError(f"a page holds {KV_BLOCK} tokens, the cache has {block}")
    tail_pages = k_tail.shape[1]
    f32, bf16 = torch.float32, torch.bfloat16
    heads, tail = (layers, pages, Hkv), (layers, tail_pages, Hkv, KV_BLOCK, D)
    if not (_is(k, dtype, dev, shape) and _is(c.v, dtype, dev, shape) and _is(c.k_scale, f32, dev, heads)
            and _is(c.v_scale, f32, dev, heads) and _is(k_tail, bf16, dev, tail) and _is(c.v_tail, bf16, dev, tail)):
        for name, dt, sh in (("k", dtype, shape), ("v", dtype, shape), ("k_scale", f32, heads),
                             ("v_scale", f32, heads), ("k_tail", bf16, tail), ("v_tail", bf16, tail)):
            _need(getattr(c, name), f"cache.{name}", dt, sh)
    return layers, pages, tail_pages, Hkv, D


def _need_rows(t: torch.Tensor, name: str, shape, dev: int) -> int:
    """A bf16 tensor [.., tokens, heads, D] whose heads are dense and whose
    tokens are evenly apart, over all leading dimensions but a layer's (a
    slice of a fused projection); returns the tokens' stride."""
    if t.dtype is not torch.bfloat16 or t.get_device() != dev or t.shape != shape:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.get_device() != dev:
            raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")
        if t.dtype is not torch.bfloat16:
            raise ValueError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    outer, tokens, H, D = shape
    if tokens == 0:
        return H * D
    so, stride, sh, sd = t.stride()
    if tokens == 1:
        stride = so if outer > 1 else H * D
    if (D > 1 and sd != 1) or (H > 1 and sh != D):
        raise ValueError(f"{name}: a token's heads must be contiguous")
    if stride < H * D or stride % 8 != 0:
        raise ValueError(f"{name}: tokens must be a multiple of 8 elements apart and not overlap")
    return stride


def kv_block_plan(lens: torch.Tensor, tails: torch.Tensor, block_table: torch.Tensor, free_ring: torch.Tensor,
                  queue: torch.Tensor, *, row_start: Optional[torch.Tensor] = None, rows: Optional[int] = None,
                  accepted_node: Optional[torch.Tensor] = None, n: Optional[int] = None,
                  tree_parents: Optional[torch.Tensor] = None, release: Optional[torch.Tensor] = None,
                  plan: Optional[BlockPlan] = None, stream=None) -> BlockPlan:
    """Block tables, slot maps and free list of one step, on the GPU. Either
    ragged rows (row_start int32 [B + 1], rows = row_start[B] or more) or a
    draft's accepted path (accepted_node int32 [B], n nodes a request,
    tree_parents int32 [B, n] or None for the chain). block_table int32
    [B, max_blocks] and free_ring int32 [cap] are updated in place; lens,
    tails and queue are not (the plan holds their next values)."""
    i32, dev = torch.int32, _device()
    B = lens.shape[0] if lens.dim() == 1 else lens.numel()
    vec, cap = (B,), free_ring.numel()
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError(f"block_table must have shape ({B}, max_blocks), got {tuple(block_table.shape)}")
    if (row_start is None) == (accepted_node is None):
        raise ValueError("give row_start (ragged rows) or accepted_node (a draft's accepted path)")
    if row_start is not None:
        if not _is(row_start, i32, dev, (B + 1,)):
            _need(row_start, "row_start", i32, (B + 1,))
        if rows is None:
            raise ValueError("rows (an upper bound of row_start[B]) is required with row_start")
        if tree_parents is not None:
            raise ValueError("tree_parents goes with accepted_node")
        rows, n = int(rows), 0
    else:
        if not _is(accepted_node, i32, dev, vec):
            _need(accepted_node, "accepted_node", i32, vec)
        if tree_parents is not None:
            n = tree_parents.shape[-1] if n is None else n
            _need(tree_parents, "tree_parents", i32, (B, n))
        if n is None:
            raise ValueError("n is required for a sequence draft")
        n = int(n)
        rows = B * n
    if release is not None:
        _need(release, "release", i32, vec)
    if plan is None:
        sizes = (B, B, B + 1, 3, max(rows, 1), max(rows, 1))
        plan = BlockPlan(*(torch.empty(s, dtype=i32, device=lens.device) for s in sizes))
    if not (_is(lens, i32, dev, vec) and _is(tails, i32, dev, vec) and _is(block_table, i32, dev, block_table.shape)
            and _is(free_ring, i32, dev, (cap,)) and _is(queue, i32, dev, (3,)) and _is(plan.new_lens, i32, dev, vec)
            and _is(plan.new_tails, i32, dev, vec) and _is(plan.new_start, i32, dev, (B + 1,))
            and _is(plan.queue, i32, dev, (3,))):
        for t, name, shape in ((lens, "lens", vec), (tails, "tails", vec), (block_table, "block_table", None),
                               (free_ring, "free_ring", (cap,)), (queue, "queue", (3,)),
                               (plan.new_lens, "plan.new_lens", vec), (plan.new_tails, "plan.new_tails", vec),
                               (plan.new_start, "plan.new_start", (B + 1,)), (plan.queue, "plan.queue", (3,))):
            _need(t, name, i32, shape)
    _need_plan_rows(plan, rows, dev)
    check(lib().kv_block_plan(lens.data_ptr(), tails.data_ptr(), _ptr(row_start), _ptr(tree_parents),
                              _ptr(accepted_node), _ptr(release), B, n, rows, block_table.shape[1], cap,
                              block_table.data_ptr(), free_ring.data_ptr(), queue.data_ptr(),
                              plan.new_lens.data_ptr(), plan.new_tails.data_ptr(), plan.new_start.data_ptr(),
                              plan.queue.data_ptr(), plan.src_rows.data_ptr(), plan.slots.data_ptr(),
                              _stream(stream)), "kv_block_plan")
    return plan


def _need_plan_rows(plan: BlockPlan, rows: int, dev: int):
    for t, name in ((plan.src_rows, "plan.src_rows"), (plan.slots, "plan.slots")):
        if not _is(t, torch.int32, dev, t.shape):
            _need(t, name, torch.int32)
        if t.numel() < rows:
            raise ValueError(f"{name} must hold {rows} rows, has {t.numel()}")


def kv8_append(cache: KV8Cache, k_new: torch.Tensor, v_new: torch.Tensor, tails: torch.Tensor, plan: BlockPlan,
               stream=None) -> None:
    """The step's kept rows into the cache, every layer at once. k_new, v_new
    bf16 [layers, rows, Hkv, D] (rows evenly apart, heads dense; [rows, Hkv, D]
    for one layer; no rows: nothing to do); tails: the tail pages before the step."""
    dev, i32 = _device(), torch.int32
    layers, pages, tail_pages, Hkv, D = _need_cache(cache, dev)
    if k_new.dim() == 3:
        k_new, v_new = k_new.unsqueeze(0), v_new.unsqueeze(0)
    rows = k_new.shape[1]
    shape = (layers, rows, Hkv, D)
    stride = _need_rows(k_new, "k_new", shape, dev)
    v_stride = _need_rows(v_new, "v_new", shape, dev)
    layer_stride, v_layer = (k_new.stride(0), v_new.stride(0)) if layers > 1 else (0, 0)
    if rows > 0 and (layer_stride != v_layer or (rows > 1 and stride != v_stride)):
        raise ValueError("k_new and v_new must have the same strides")
    B = tails.numel()
    if not (_is(tails, i32, dev, (B,)) and _is(plan.new_tails, i32, dev, (B,))
            and _is(plan.new_start, i32, dev, (B + 1,))):
        _need(tails, "tails", i32, (B,))
        _need(plan.new_tails, "plan.new_tails", i32, (B,))
        _need(plan.new_start, "plan.new_start", i32, (B + 1,))
    _need_plan_rows(plan, rows, dev)
    if rows == 0:  # a step that keeps nothing, as kv_block_plan has it
        return
    check(lib().kv8_append(k_new.data_ptr(), v_new.data_ptr(), stride, layer_stride, tails.data_ptr(),
                           plan.new_tails.data_ptr(), plan.new_start.data_ptr(), plan.src_rows.data_ptr(),
                           plan.slots.data_ptr(), B, rows, Hkv, D, layers, pages, tail_pages,
                           _KV8_FORMATS[cache.k.dtype], cache.k.data_ptr(), cache.v.data_ptr(),
                           cache.k_scale.data_ptr(), cache.v_scale.data_ptr(), cache.k_tail.data_ptr(),
                           cache.v_tail.data_ptr(), _stream(stream)), "kv8_append")


@lru_cache(maxsize=256)
def _attention_ws(device: int, B: int, n: int, H: int, Hkv: int, D: int, max_len: int) -> int:
    return kv8_tree_attention_workspace_bytes(B, n, H, Hkv, D, max_len)


@lru_cache(maxsize=256)
def _logprobs_ws(R: int, V: int, top: int) -> int:
    return token_logprobs_workspace_bytes(R, V, top)


def kv8_tree_attention_workspace_bytes(B: int, n: int, H: int, Hkv: int, D: int, max_len: int) -> int:
    return int(lib().kv8_tree_attention_workspace_bytes(B, n, H, Hkv, D, max_len))


def kv8_tree_attention(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, cache: KV8Cache, layer: int,
                       block_table: torch.Tensor, lens: torch.Tensor, tails: torch.Tensor,
                       tree_parents: Optional[torch.Tensor] = None, max_len: Optional[int] = None,
                       scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                       ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Tree-masked verify attention over the 8-bit cache of one layer. q bf16
    [B, n, H, D] and the tree's own k_new, v_new bf16 [B, n, Hkv, D] may be
    slices of one fused projection (heads dense, tokens evenly apart); lens,
    tails int32 [B]; block_table int32 [B, max_blocks]; max_len: an upper bound
    of lens (default: what the table holds); ws: zeroed before its first use, and
    used by no two calls at once (default: one for each stream and capture).
    Returns bf16 [B, n, H, D]."""
    dev, i32 = _device(), torch.int32
    layers, pages, tail_pages, Hkv, D = _need_cache(cache, dev)
    if not 0 <= layer < layers:
        raise ValueError(f"layer {layer} is not one of the cache's {layers}")
    if q.dim() != 4:
        raise ValueError(f"q must have 4 dimensions, got {tuple(q.shape)}")
    B, n, H, _ = q.shape
    q_stride = _need_rows(q, "q", (B, n, H, D), dev)
    new = (B, n, Hkv, D)
    kv_stride = _need_rows(k_new, "k_new", new, dev)
    v_stride = _need_rows(v_new, "v_new", new, dev)
    if B > 1 and n > 1:
        for t, name, s in ((q, "q", q_stride), (k_new, "k_new", kv_stride), (v_new, "v_new", v_stride)):
            if t.stride(0) != n * s:
                raise ValueError(f"{name}: the tokens of all requests must be evenly apart")
    if B * n > 1 and kv_stride != v_stride:
        raise ValueError("k_new and v_new must have the same strides")
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError(f"block_table must have shape ({B}, max_blocks), got {tuple(block_table.shape)}")
    if not (_is(lens, i32, dev, (B,)) and _is(tails, i32, dev, (B,)) and _is(block_table, i32, dev, block_table.shape)):
        _need(lens, "lens", i32, (B,))
        _need(tails, "tails", i32, (B,))
        _need(block_table, "block_table", i32)
    if tree_parents is not None and not _is(tree_parents, i32, dev, (B, n)):
        _need(tree_parents, "tree_parents", i32, (B, n))
    max_blocks = block_table.shape[1]
    max_len = max_blocks * KV_BLOCK + KV_BLOCK - 1 if max_len is None else int(max_len)
    scale = D ** -0.5 if scale is None else float(scale)
    if out is None:
        out = torch.empty((B, n, H, D), dtype=torch.bfloat16, device=q.device)
    else:
        _need(out, "out", torch.bfloat16, (B, n, H, D))
    if ws is None:
        ws = _stream_workspace(_attention_ws(dev, B, n, H, Hkv, D, max_len), "kv8_attention", stream)
    else:
        _need_ws(ws, dev)
    codes, heads = pages * Hkv * KV_BLOCK * D * layer, pages * Hkv * layer * 4
    tail = tail_pages * Hkv * KV_BLOCK * D * layer * 2
    check(lib().kv8_tree_attention(
        q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), q_stride, kv_stride, cache.k.data_ptr() + codes,
        cache.v.data_ptr() + codes, cache.k_scale.data_ptr() + heads, cache.v_scale.data_ptr() + heads,
        cache.k_tail.data_ptr() + tail, cache.v_tail.data_ptr() + tail, block_table.data_ptr(), lens.data_ptr(),
        tails.data_ptr(), _ptr(tree_parents), B, n, H, Hkv, D, max_blocks, pages, tail_pages, max_len,
        _KV8_FORMATS[cache.k.dtype], scale, out.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream)),
        "kv8_tree_attention")
    return out


# ------------------------------------------------------ log probabilities

@dataclass
class TokenLogprobs:
    logp: torch.Tensor      # fp32 [R, m] (or [R]): of the given tokens
    entropy: torch.Tensor   # fp32 [R]
    top_ids: torch.Tensor   # int32 [R, top]
    top_logp: torch.Tensor  # fp32 [R, top]


def token_logprobs_workspace_bytes(R: int, V: int, top: int) -> int:
    return int(lib().token_logprobs_workspace_bytes(R, V, top))


def token_logprobs(logits: torch.Tensor, ids: torch.Tensor, top: int = 0, ws: Optional[torch.Tensor] = None,
                   stream=None) -> TokenLogprobs:
    """Log probabilities of given tokens under logit rows (fp32 or bf16 [R, V];
    ids int32 [R, m] or [R], -1 for none), each row's entropy, and its `top`
    most probable tokens (ties to the lower index). ws: used by no two calls at
    once (default: one for each stream and capture)."""
    if logits.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"logits must be {torch.float32} or {torch.bfloat16}, got {logits.dtype}")
    _need(logits, "logits", logits.dtype)
    if logits.dim() != 2:
        raise ValueError(f"logits must have shape (R, V), got {tuple(logits.shape)}")
    R, V = logits.shape
    _need(ids, "ids", torch.int32)
    if ids.dim() not in (1, 2) or ids.shape[0] != R:
        raise ValueError(f"ids must have shape ({R}, m) or ({R},), got {tuple(ids.shape)}")
    m, dev = (ids.shape[1] if ids.dim() == 2 else 1), logits.device
    f32 = torch.float32
    out = TokenLogprobs(torch.empty(ids.shape, dtype=f32, device=dev), torch.empty(R, dtype=f32, device=dev),
                        torch.empty((R, top), dtype=torch.int32, device=dev),
                        torch.empty((R, top), dtype=f32, device=dev))
    if ws is None:
        ws = _stream_workspace(_logprobs_ws(R, V, top), "logprobs", stream)
    else:
        _need_ws(ws, _device())
    check(lib().token_logprobs(logits.data_ptr(), int(logits.dtype is torch.bfloat16), ids.data_ptr(), R, V, m, top,
                               out.logp.data_ptr(), out.entropy.data_ptr(), out.top_ids.data_ptr(),
                               out.top_logp.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream)),
          "token_logprobs")
    return out
