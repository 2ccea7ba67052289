"""A speculative-verify decode loop over a paged cache, in 8 or in 16 bits.

One step, for every request of a batch at once: the target's forward over a
draft (the last emitted token and the drafted ones), each layer attending to
the committed tokens in pages and to the draft's own keys and values where the
fused projection left them; acceptance; the log probabilities of the emitted
tokens; the block plan for the accepted path; and the accepted rows into every
layer's cache. Nothing of a step goes through the host.

With the 16-bit cache a step's keys and values, rejected ones too, go into the
pages before the layer's attention, which reads nothing else; the length then
moves on by the accepted rows, and the next step writes over what was rejected.
Its requests hold their pages from the start.

The weights are random and the layers bare (no norms' weights): what is shown is
how the entry points go together. Queries and keys are rotated by their
positions where the target has a rotation.

Drafts change how many tokens a step emits, not which ones, up to rounding: a
row of a longer draft adds its keys in another order, and reads a block in bf16
until the step that completes it has put it into 8 bits. Its logits so differ in
the last bf16 places, and where the best two lie that close together either may
be emitted.

    python -m speculative_decode_verify_w4a16_gb300.verify_step [--requests B] [--layers L] [--draft K] [--steps N]
        [--cache kv8|kv16] [--rope BASE]
"""
from __future__ import annotations

import argparse
from dataclasses import dataclass
from typing import List, Optional, Union

import torch

from . import api
from ._lib import check

D = 128
MAX_ROWS = 80  # of one linear


def _weight(N: int, K: int, gen: torch.Generator) -> api.PackedWeight:
    w = torch.randn(N, K, generator=gen, device="cuda") * K ** -0.5
    return api.prepack(*api.quantize(w))


def _norm(x: torch.Tensor) -> torch.Tensor:
    y = x.float()
    return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()


class Target:
    """A small random W4A16 target model."""

    def __init__(self, layers: int = 2, heads: int = 8, kv_heads: int = 2, hidden: int = 1024, inner: int = 2048,
                 vocab: int = 4096, seed: int = 0, rope: Optional[api.Rope] = None):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.heads, self.kv_heads, self.hidden, self.inner, self.vocab = heads, kv_heads, hidden, inner, vocab
        self.rope = rope
        self.embed = torch.randn(vocab, hidden, generator=gen, device="cuda").bfloat16()
        shapes = ((heads + 2 * kv_heads) * D, hidden), (hidden, heads * D), (2 * inner, hidden), (hidden, inner)
        self.layers = [[_weight(N, K, gen) for N, K in shapes] for _ in range(layers)]
        self.lm_head = _weight(vocab, hidden, gen)

    def forward(self, ids: torch.Tensor, cache: Union[api.KV8Cache, api.KV16Cache], state: "Requests", max_len: int,
                row_start: Optional[torch.Tensor] = None):
        """ids int32 [B, n], a chain from each request's last token: fp32
        logits [B, n, vocab] and the layers' own keys and values
        [layers, B * n, kv_heads, D], None with the 16-bit cache, which has them.
        With that cache also ids int32 [T, 1] with row_start: chains of
        different lengths."""
        B, n = ids.shape
        h = self.embed[ids.long().view(-1)]
        paged = isinstance(cache, api.KV16Cache)
        if self.rope is not None and not paged:
            pos = state.lens[:, None] + torch.arange(n, dtype=torch.int32, device=ids.device)
        new_k, new_v = [], []
        for i, (qkv_w, o_w, gate_up, down) in enumerate(self.layers):
            qkv = api.linear(_norm(h), qkv_w).view(B, n, self.heads + 2 * self.kv_heads, D)
            q, k, v = qkv.split((self.heads, self.kv_heads, self.kv_heads), 2)
            if paged:
                at = dict(row_start=row_start)
                if self.rope is None:
                    api.kv16_append(cache, i, k, v, state.table, state.lens, **at)
                else:
                    q = api.kv16_append(cache, i, k, v, state.table, state.lens, rope=self.rope, q=q, q_out=q, **at)
                a = api.kv16_attention(q, cache, i, state.table, state.lens, **at)
            else:
                if self.rope is not None:
                    qk = qkv[:, :, :self.heads + self.kv_heads]
                    api.rope(qk, pos, self.rope, out=qk)
                new_k.append(k.reshape(B * n, self.kv_heads, D))
                new_v.append(v.reshape(B * n, self.kv_heads, D))
                a = api.kv8_tree_attention(q, k, v, cache, i, state.table, state.lens, state.tails, max_len=max_len)
            h = h + api.linear(a.view(B * n, self.heads * D), o_w)
            gate, up = api.linear(_norm(h), gate_up).chunk(2, 1)
            h = h + api.linear((torch.nn.functional.silu(gate.float()) * up.float()).bfloat16(), down)
        logits, _ = api.linear_logits(_norm(h), self.lm_head)
        kv = (None, None) if paged else (torch.stack(new_k), torch.stack(new_v))
        return (logits.view(B, n, self.vocab), *kv)


@dataclass
class Requests:
    """The batch's place in the cache."""
    lens: torch.Tensor   # committed tokens
    tails: torch.Tensor  # tail pages
    table: torch.Tensor  # block table
    ring: torch.Tensor   # free pages
    queue: torch.Tensor  # their head and count

    @classmethod
    def empty(cls, B: int, max_blocks: int, pages: int) -> "Requests":
        z = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        return cls(z([0] * B), z([2 * b for b in range(B)]),
                   torch.full((B, max_blocks), -1, dtype=torch.int32, device="cuda"),
                   torch.arange(pages, dtype=torch.int32, device="cuda"), z([0, pages, 0]))

    @classmethod
    def resident(cls, B: int, max_blocks: int) -> "Requests":
        """For the 16-bit cache: every request holds all its pages, dealt out in turn."""
        state = cls.empty(B, max_blocks, 0)
        state.table.copy_(torch.arange(B * max_blocks, dtype=torch.int32, device="cuda").view(max_blocks, B).T)
        return state

    def advance(self, plan: api.BlockPlan):
        self.lens, self.tails, self.queue = plan.new_lens, plan.new_tails, plan.queue


@dataclass
class Emitted:
    tokens: torch.Tensor  # int32 [B, n]: accepted drafts, then the target's own; -1 behind
    logp: torch.Tensor    # fp32 [B, n]: their log probabilities (0 behind)
    top_ids: torch.Tensor
    top_logp: torch.Tensor


def verify_step(target: Target, cache: Union[api.KV8Cache, api.KV16Cache], state: Requests, last: torch.Tensor, draft: torch.Tensor,
                max_len: int, top: int = 3) -> Emitted:
    """One greedy step: `last` int32 [B], the last emitted token of each
    request (not yet in the cache), and its draft int32 [B, K], K = 0 for plain
    decoding. The state and the cache move on."""
    B, K = draft.shape
    ids = torch.cat([last[:, None], draft], 1)  # row i gives the token after draft i - 1
    logits, k, v = target.forward(ids, cache, state, max_len)
    if K:
        accepted, token, node = api.spec_accept_node(logits, draft)
    else:  # nothing to accept: the most probable token
        token = api.token_logprobs(logits.view(B, -1), ids[:, :0], top=1).top_ids[:, 0]
        accepted = node = torch.zeros_like(token)
    # the emitted tokens, row by row: drafts as far as they were accepted, then the target's
    row = torch.arange(K + 1, device=ids.device)[None]
    tokens = torch.where(row < accepted[:, None], torch.cat([draft, token[:, None]], 1), token[:, None])
    tokens = torch.where(row <= accepted[:, None], tokens, -1).int()
    report = api.token_logprobs(logits.view(B * (K + 1), -1), tokens.view(-1), top=top)
    # rows 0 .. accepted (the last token and the accepted drafts) go into the cache, or are kept there
    if isinstance(cache, api.KV16Cache):
        state.lens = state.lens + accepted + 1
        return Emitted(tokens, report.logp.view(B, K + 1), report.top_ids, report.top_logp)
    plan = api.kv_block_plan(state.lens, state.tails, state.table, state.ring, state.queue, accepted_node=node, n=K + 1)
    api.kv8_append(cache, k, v, state.tails, plan)
    state.advance(plan)
    return Emitted(tokens, report.logp.view(B, K + 1), report.top_ids, report.top_logp)


def decode(target: Target, prompts: List[List[int]], steps: int, K: int, draft_of, cache: str = "kv8") -> List[list]:
    """Greedy decoding with drafts: draft_of(b, tokens, K) gives K token ids to
    try after request b's tokens (a drafter's place). cache: "kv8" or "kv16",
    the paged cache in 8 or in 16 bits. Returns each request's
    (token, log probability) pairs; raises W4A16Error for whatever the kernels
    reported in the device error word."""
    B = len(prompts)
    if not B or not all(prompts):
        raise ValueError("decode needs prompts of at least one token")
    if B * (K + 1) > MAX_ROWS:
        raise ValueError(f"{B} requests with drafts of {K} are more than the linear's {MAX_ROWS} rows")
    if cache not in ("kv8", "kv16"):
        raise ValueError(f"cache must be kv8 or kv16, got {cache!r}")
    longest = max(map(len, prompts)) + steps * (K + 1)
    blocks = longest // api.KV_BLOCK + 1
    pages = B * blocks  # no request is ever refused one
    if cache == "kv16":
        state, kv = Requests.resident(B, blocks), api.kv16_cache(len(target.layers), pages, target.kv_heads)
    else:
        state, kv = Requests.empty(B, blocks, pages), api.kv8_cache(len(target.layers), pages, B, target.kv_heads)
    # the prompts, all but their last tokens, chains of as many rows as the linear takes
    done, at_once = [0] * B, min(MAX_ROWS // B, 64)
    while any(done[b] < len(p) - 1 for b, p in enumerate(prompts)):
        rows = [p[done[b]:min(done[b] + at_once, len(p) - 1)] for b, p in enumerate(prompts)]
        start = torch.tensor([0] + [len(r) for r in rows]).cumsum(0).int().cuda()
        if cache == "kv16":
            ids = torch.tensor(sum(rows, []), dtype=torch.int32, device="cuda")
            target.forward(ids[:, None], kv, state, longest, row_start=start)
            state.lens = state.lens + start.diff()
        else:
            n = max(map(len, rows))
            ids = torch.tensor([r + [0] * (n - len(r)) for r in rows], dtype=torch.int32, device="cuda")
            _, k, v = target.forward(ids, kv, state, longest)
            # a request's rows are the first of its n: kept as ragged rows
            keep = torch.cat([torch.arange(len(r)) + b * n for b, r in enumerate(rows)]).cuda()
            plan = api.kv_block_plan(state.lens, state.tails, state.table, state.ring, state.queue, row_start=start,
                                     rows=int(keep.numel()))
            api.kv8_append(kv, k[:, keep], v[:, keep], state.tails, plan)
            state.advance(plan)
        done = [d + len(r) for d, r in zip(done, rows)]
    tokens = [list(p) for p in prompts]
    out: List[list] = [[] for _ in prompts]
    for _ in range(steps):
        draft = torch.tensor([draft_of(b, t, K) for b, t in enumerate(tokens)], dtype=torch.int32, device="cuda").view(B, K)
        last = torch.tensor([t[-1] for t in tokens], dtype=torch.int32, device="cuda")
        e = verify_step(target, kv, state, last, draft, longest)
        for b, (ids, lps) in enumerate(zip(e.tokens.tolist(), e.logp.tolist())):
            new = [(t, lp) for t, lp in zip(ids, lps) if t >= 0]
            out[b] += new
            tokens[b] += [t for t, _ in new]
    check(api.check_device_status(), "decode")
    return out


def main():
    a = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    a.add_argument("--requests", type=int, default=4)
    a.add_argument("--layers", type=int, default=2)
    a.add_argument("--draft", type=int, default=4)
    a.add_argument("--steps", type=int, default=8)
    a.add_argument("--cache", choices=("kv8", "kv16"), default="kv8")
    a.add_argument("--rope", type=float, metavar="BASE", help="rotate queries and keys")
    a = a.parse_args()
    target = Target(layers=a.layers, rope=None if a.rope is None else api.rope_frequencies(D, a.rope))
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, target.vocab, (20 + 37 * b,), generator=g).tolist() for b in range(a.requests)]
    # plain greedy decoding first; its tokens, every third one wrong, then serve as drafts
    need = a.steps * (a.draft + 1)
    plain = decode(target, prompts, need, 0, lambda b, t, K: [], cache=a.cache)
    known = [p + [t for t, _ in o] for p, o in zip(prompts, plain)]

    def draft_of(b, tokens, K):
        at = len(tokens)
        return [known[b][at + i] if at + i < len(known[b]) and (at + i) % 3 else 1 for i in range(K)]

    out = decode(target, prompts, a.steps, a.draft, draft_of, cache=a.cache)
    for b, o in enumerate(out):
        same = 0
        while same < len(o) and o[same][0] == plain[b][same][0]:
            same += 1
        print(f"request {b}: {len(o)} tokens in {a.steps} steps ({len(o) / a.steps:.2f} a step), "
              f"mean log probability {sum(lp for _, lp in o) / len(o):.3f}, "
              + ("all as without drafts" if same == len(o) else f"the first {same} as without drafts, then a near tie: "
                 f"{o[same][1]:.4f} and {plain[b][same][1]:.4f}"))


if __name__ == "__main__":
    main()
