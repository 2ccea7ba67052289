"""GPU parity of the paged 8-bit cache operators (block plan, append, tree
attention) against plain 64-bit implementations (kv8_reference).

The plan is whole numbers and the append rounds once from bf16 with exact
scaling, so both are compared bit for bit. Attention: each softmax weight is
rounded once for the weighted sum (fp16, half a step 2^-11; for the tail and
the tree's own rows bf16, half a step 2^-8), against a normaliser of fp32
weights, so the weighted sum moves by at most 2^-8 A, A = sum w |v|; the output
is rounded to bf16 (2^-8 |out|). Scores: fp32 sums over 128 products and the
exponential's approximation move a weight by some 1e-5 of itself, 2 % of 2^-8
beyond which nothing is left over: bound = 1.05 * 2^-8 (A + |out|) + 1e-7 max|v|."""
import numpy as np
import pytest
import torch

import kv8_reference as ref
import speculative_decode_verify_w4a16_gb300 as sv
from helpers import dev

pytestmark = pytest.mark.gpu
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decode_verify_w4a16_gb300 import build
    build.build()


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev())


def _status(want=0):
    torch.cuda.synchronize()
    assert sv.check_device_status() == want


# ------------------------------------------------------------------- plan

def _plan_case(B, hi, rng, spare_pages, max_blocks):
    lens = rng.integers(0, hi + 1, B).astype(np.int32)
    full = lens // 64
    pages = int(full.sum()) + spare_pages
    perm = rng.permutation(pages)
    table = np.full((B, max_blocks), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :full[b]] = perm[at:at + full[b]]
        at += full[b]
    ring = np.full(pages, -7, np.int32)
    head = int(rng.integers(0, pages))
    ring[(head + np.arange(spare_pages)) % pages] = perm[at:]
    tails = (2 * np.arange(B) + rng.integers(0, 2, B)).astype(np.int32)
    return lens, tails, table, ring, np.array([head, spare_pages, 0], np.int32)


def _check_plan(case, kept, total, release, **kw):
    lens, tails, table, ring, queue = case
    want_table, want_ring, want = ref.plan(lens, tails, table, ring, queue, total, kept, release)
    t, r = _i32(table), _i32(ring)
    args = (_i32(lens), _i32(tails), t, r, _i32(queue))
    for _ in range(2):  # the same call again gives the same
        got = sv.kv_block_plan(*args, release=None if release is None else _i32(release), **kw)
        _status()
        assert np.array_equal(t.cpu().numpy(), want_table) and np.array_equal(r.cpu().numpy(), want_ring)
        for name, w in want.items():
            g = getattr(got, name).cpu().numpy()
            assert np.array_equal(g[:len(w)], w), name


@pytest.mark.parametrize("B,n,tree", [(1, 1, False), (16, 5, False), (7, 64, False), (33, 64, True), (300, 17, True)])
@pytest.mark.parametrize("ended", [False, True])
def test_plan_of_a_draft(B, n, tree, ended):
    rng = np.random.default_rng(100 * B + n)
    case = _plan_case(B, 500, rng, B + 2, 10)
    parents = np.stack([ref.random_tree(n, rng) if tree else ref.chain(n) for _ in range(B)])
    node = rng.integers(0, n, B)
    release = (rng.random(B) < 0.3).astype(np.int32) if ended else None
    kept = [[b * n + j for j in ref.root_path(parents[b], node[b])] for b in range(B)]
    _check_plan(case, kept, B * n, release, accepted_node=_i32(node), n=n, tree_parents=_i32(parents) if tree else None)


@pytest.mark.parametrize("B,per,hi", [(1, 200, 0), (3, 0, 200), (7, 700, 300), (1500, 40, 130), (4096, 3, 64)])
def test_plan_of_ragged_rows(B, per, hi):
    rng = np.random.default_rng(B)
    cnt = rng.integers(0, 2 * per + 1, B)
    cnt[rng.random(B) < 0.2] = 0
    start = np.concatenate([[0], np.cumsum(cnt)])
    rows = int(start[-1]) + 5  # an upper bound, as a captured step has it
    case = _plan_case(B, hi, rng, int((cnt // 64 + 1).sum()), (hi + 2 * per) // 64 + 1)
    release = (np.arange(B) % 11 == 3).astype(np.int32)
    kept = [list(range(start[b], start[b + 1])) for b in range(B)]
    _check_plan(case, kept, rows, release, row_start=_i32(start), rows=rows)


@pytest.mark.parametrize("free", [0, 1, 5, 9])
def test_plan_when_pages_run_out(free):
    rng = np.random.default_rng(free)
    B = 12
    cnt = np.array([70, 3, 0, 64, 130, 1, 200, 5, 64, 64, 2, 0])
    start = np.concatenate([[0], np.cumsum(cnt)])
    case = _plan_case(B, 100, rng, free, 6)
    kept = [list(range(start[b], start[b + 1])) for b in range(B)]
    _check_plan(case, kept, int(start[-1]), None, row_start=_i32(start), rows=int(start[-1]))


def test_plan_reports_bad_input():
    rng = np.random.default_rng(3)
    B, n = 6, 5
    lens, tails, table, ring, queue = _plan_case(B, 200, rng, 8, 5)
    good = np.zeros(B, np.int64)

    def run(lens=lens, node=good, queue=queue, ring=ring, parents=None):
        p = sv.kv_block_plan(_i32(lens), _i32(tails), _i32(table), _i32(ring), _i32(queue), accepted_node=_i32(node),
                             n=n, tree_parents=None if parents is None else _i32(parents))
        torch.cuda.synchronize()
        status = sv.check_device_status()
        return status, {k: getattr(p, k).cpu().numpy() for k in ("new_lens", "new_start", "queue", "slots", "src_rows")}

    assert run()[0] == 0
    bad = lens.copy()
    bad[2], bad[4] = -1, 10 ** 6
    s, p = run(lens=bad)
    assert s == 5 and p["new_lens"][2] == -1 and p["new_lens"][4] == 10 ** 6
    assert p["new_start"][3] == p["new_start"][2] and p["new_start"][5] == p["new_start"][4]
    s, p = run(node=np.array([0, 5, 0, -1, 4, 0]))
    assert s == 5 and list(np.diff(p["new_start"])) == [1, 1, 1, 1, 5, 1]  # the root alone
    par = np.stack([ref.chain(n)] * B)
    par[1, 3], par[3, 0] = 4, 2
    s, p = run(node=np.full(B, 4), parents=par)
    assert s == 5 and list(np.diff(p["new_start"])) == [5, 1, 5, 1, 5, 5]
    for q in ([-1, 3, 0], [len(ring), 3, 0], [0, len(ring) + 1, 0], [0, -1, 0]):
        assert run(queue=np.array(q))[0] == 5
    full = lens.copy()
    full[:] = 63
    s, p = run(lens=full, ring=np.full_like(ring, -3))
    assert s == 5 and set(p["slots"][:B]) == {ref.SKIP}


@pytest.mark.parametrize("start,rows", [([0, 5, 3, 9], 9), ([0, 4, 12, 12], 9), ([-2, 4, 6, 9], 9), ([0, 9, 0, 9], 9),
                                        ([0, 4, 6, 10], 9)])
def test_plan_with_bad_row_ranges_keeps_nothing(start, rows):
    """And leaves nothing of an earlier plan in its outputs."""
    rng = np.random.default_rng(4)
    lens, tails, table, ring, queue = _plan_case(3, 200, rng, 8, 5)
    args = [_i32(x) for x in (lens, tails, table, ring, queue)]
    plan = sv.kv_block_plan(*args, row_start=_i32([0, 3, 6, 9]), rows=rows)
    assert sv.check_device_status() == 0
    args = [_i32(x) for x in (lens, tails, table, ring, queue)]
    plan = sv.kv_block_plan(*args, row_start=_i32(start), rows=rows, plan=plan)
    torch.cuda.synchronize()
    assert sv.check_device_status() == 5
    assert np.array_equal(plan.new_lens.cpu(), lens) and np.array_equal(plan.new_tails.cpu(), tails)
    assert not plan.new_start.any() and (plan.src_rows[:rows] == -1).all() and (plan.slots[:rows] == ref.SKIP).all()
    assert plan.queue[:2].tolist() == list(queue[:2]) and np.array_equal(args[2].cpu(), table)


# ----------------------------------------------------------------- append

def _history(rng, Hkv, tokens, D=128, scale=1.0):
    k = torch.from_numpy(rng.standard_normal((Hkv, tokens, D)) * np.exp(rng.standard_normal(D)) * scale).bfloat16()
    v = torch.from_numpy(rng.standard_normal((Hkv, tokens, D)) * scale).bfloat16()
    return k, v


@pytest.mark.parametrize("dtype", [E4M3, E5M2])
@pytest.mark.parametrize("Hkv,layers,chunks,extra", [
    (1, 1, [[1, 62, 1, 1]], 0),                      # one token at a time over a block's end
    (8, 2, [[200, 5, 64, 1], [0, 63, 1, 64]], 0),    # blocks filled by prompts and by one token
    (3, 3, [[17, 300, 0], [64, 64, 65], [1, 1, 190]], 64),  # rows of a wider projection
])
def test_append_builds_the_cache_whatever_the_steps(dtype, Hkv, layers, chunks, extra):
    """Requests whose tokens arrive in chunks: after each step the pages and
    tails hold what the whole history gives, bit for bit."""
    rng = np.random.default_rng(7 * Hkv + layers)
    B, D = len(chunks), 128
    hist = [[_history(rng, Hkv, sum(c)) for c in chunks] for _ in range(layers)]
    pages = sum(sum(c) // 64 for c in chunks) + 2
    cache = sv.kv8_cache(layers, pages, B, Hkv, dtype=dtype, device=dev())
    table = _i32(np.full((B, 8), -1))
    ring, queue = _i32(rng.permutation(pages)), _i32([0, pages, 0])
    lens, tails = _i32(np.zeros(B)), _i32(2 * np.arange(B))
    done = np.zeros(B, int)
    for step in range(max(map(len, chunks))):
        cnt = [c[step] if step < len(c) else 0 for c in chunks]
        start = np.concatenate([[0], np.cumsum(cnt)])
        rows = max(1, int(start[-1]))
        new = [torch.zeros(layers, rows, Hkv * D + extra, dtype=torch.bfloat16) for _ in range(2)]
        for l in range(layers):
            for b in range(B):
                for c in range(2):
                    x = hist[l][b][c][:, done[b]:done[b] + cnt[b]]
                    new[c][l, start[b]:start[b + 1], :Hkv * D] = x.transpose(0, 1).reshape(cnt[b], Hkv * D)
        dn = [x.to(dev())[:, :, :Hkv * D].unflatten(2, (Hkv, D)) for x in new]
        plan = sv.kv_block_plan(lens, tails, table, ring, queue, row_start=_i32(start), rows=rows)
        sv.kv8_append(cache, dn[0], dn[1], tails, plan)
        sv.kv8_append(cache, dn[0], dn[1], tails, plan)  # again: nothing it reads was overwritten
        _status()
        lens, tails, queue = plan.new_lens, plan.new_tails, plan.queue
        done += np.array(cnt)
        assert np.array_equal(lens.cpu().numpy(), done)
    tb, tl = table.cpu().numpy(), tails.cpu().numpy()
    for c, (codes, scales, tail) in enumerate(((cache.k, cache.k_scale, cache.k_tail),
                                               (cache.v, cache.v_scale, cache.v_tail))):
        codes, scales, tail = codes.cpu().view(torch.uint8), scales.cpu(), tail.cpu()
        for l in range(layers):
            for b in range(B):
                x = hist[l][b][c]
                for j in range(done[b] // 64):
                    for h in range(Hkv):
                        q, s = ref.quantize(x[h, 64 * j:64 * j + 64], dtype)
                        assert float(scales[l, tb[b, j], h]) == s
                        assert torch.equal(codes[l, tb[b, j], h], q.view(torch.uint8))
                rest = done[b] % 64
                assert torch.equal(tail[l, tl[b], :, :rest], x[:, done[b] - rest:])


@pytest.mark.parametrize("dtype", [E4M3, E5M2])
def test_append_of_unusual_values(dtype):
    """Zero blocks, denormals, infinities, NaN, values at the scale's edges."""
    D = 128
    x = torch.zeros(64 * 6, 1, D, dtype=torch.bfloat16)
    rng = np.random.default_rng(5)
    x[64:128] = torch.from_numpy(rng.standard_normal((64, 1, D)) * 1e-39).bfloat16()   # below the smallest scale
    x[128:192] = torch.from_numpy(rng.standard_normal((64, 1, D)) * 1e38).bfloat16()
    x[130, 0, 3], x[131, 0, 4] = float("inf"), float("-inf")
    x[192:256, 0, :] = 1.75  # the largest code exactly
    x[256:320, 0, 7] = 1.7578125  # one step above: the next power of two
    x[320:384] = torch.from_numpy(rng.standard_normal((64, 1, D))).bfloat16()
    x[333, 0, 9] = float("nan")
    cache = sv.kv8_cache(1, 6, 1, 1, dtype=dtype, device=dev())
    tails = _i32([0])
    plan = sv.kv_block_plan(_i32([0]), tails, _i32(np.full((1, 6), -1)), _i32(np.arange(6)), _i32([0, 6, 0]),
                            row_start=_i32([0, 384]), rows=384)
    sv.kv8_append(cache, x.to(dev()), (-x).to(dev()), tails, plan)
    _status()
    for j in range(6):
        for sign, codes, scales in ((1, cache.k, cache.k_scale), (-1, cache.v, cache.v_scale)):
            q, s = ref.quantize(sign * x[64 * j:64 * j + 64, 0], dtype)
            assert float(scales[0, j, 0]) == s, j
            got = codes[0, j, 0].cpu().float()
            assert torch.equal(got.isnan(), q.float().isnan())
            assert torch.equal(got.nan_to_num(0.0), q.float().nan_to_num(0.0)), j


def test_append_skips_and_reports_what_fits_no_plan():
    D, Hkv = 128, 2
    k = torch.ones(70, Hkv, D, dtype=torch.bfloat16, device=dev())
    tails = _i32([0, 2])

    def run(**change):
        cache = sv.kv8_cache(1, 3, 2, Hkv, device=dev())
        plan = sv.kv_block_plan(_i32([0, 0]), tails, _i32(np.full((2, 4), -1)), _i32(np.arange(3)), _i32([0, 3, 0]),
                                row_start=_i32([0, 3, 70]), rows=70)
        for name, (i, value) in change.items():
            getattr(plan, name)[i] = value
        sv.kv8_append(cache, k, k, tails, plan)
        torch.cuda.synchronize()
        return sv.check_device_status(), float(cache.k_tail.float().sum()), float(cache.k.float().sum())

    one = Hkv * D
    assert run() == (0, 6 * one, 64 * one * 256.0)  # 1 = 256 * 2^-8
    assert run(src_rows=(1, 70)) == (5, 3 * one, 64 * one * 256.0)     # request 0: a row that is not there
    assert run(src_rows=(10, -1)) == (5, 6 * one, 0.0)                  # a row of the page
    assert run(slots=(20, 5)) == (5, 6 * one, 0.0)
    assert run(slots=(3, ref.SKIP)) == (5, 3 * one, 0.0)                # request 1's first slot: all of it
    assert run(new_tails=(0, 4)) == (5, 3 * one, 64 * one * 256.0)
    assert run(new_tails=(0, -1)) == (5, 3 * one, 64 * one * 256.0)
    assert run(new_start=(1, 80))[0] == 5
    assert run(new_start=(1, -5))[0] == 5


# -------------------------------------------------------------- attention

def _attn_inputs(rng, B, n, H, Hkv, wide=0, D=128):
    qkv = torch.from_numpy(rng.standard_normal((B, n, (H + 2 * Hkv) * D + wide))).bfloat16()
    return qkv, (slice(0, H * D), slice(H * D, (H + Hkv) * D), slice((H + Hkv) * D, (H + 2 * Hkv) * D))


def _attend(rng, B, n, H, Hkv, lens, tree, dtype, hist=None, max_len=None, wide=0, layers=1, layer=0, stale=None,
            qkv=None, parents=None, status=0, scale=None):
    D = 128
    hist = hist or [_history(rng, Hkv, L) for L in lens]
    cap = max(lens) if max_len is None else max_len
    cache = ref.Cache(hist, dtype, rng, cap, stale=stale)
    made, cols = _attn_inputs(rng, B, n, H, Hkv, wide)
    qkv = made if qkv is None else qkv
    q, k, v = (qkv[:, :, c].unflatten(2, (-1, D)) for c in cols)
    if parents is None:
        parents = np.stack([ref.random_tree(n, rng) if tree else ref.chain(n) for _ in range(B)])
    c, table, dl, dt = cache.to(sv, dev(), layers, layer)
    dq = qkv.to(dev())
    out = sv.kv8_tree_attention(*(dq[:, :, s].unflatten(2, (-1, D)) for s in cols), c, layer, table, dl, dt,
                                tree_parents=_i32(parents) if tree else None, max_len=cap, scale=scale)
    torch.cuda.synchronize()
    assert sv.check_device_status() == status
    return out.cpu().double(), cache, (q, k, v), parents


def _check(got, cache, qkv, parents, what="", rows=None, scale=None):
    q, k, v = qkv
    worst = 0.0
    for b in range(q.shape[0]):
        want, mag = ref.attention(cache.values[b], q[b], k[b], v[b], parents[b], scale)
        top = max(float(x.abs().max()) if x.numel() else 0.0 for x in (cache.values[b][1], v[b].double()))
        bound = 1.05 * 2.0 ** -8 * (mag + want.abs()) + 1e-7 * top
        ratio = (got[b] - want).abs() / bound
        assert not ratio.isnan().any(), f"{what}: NaN in request {b}"
        worst = max(worst, float(ratio.max()))
    print(f"{what}: max |err| / bound = {worst:.3f}")
    assert worst <= 1.0, what


ATTN = [  # B, n, H, Hkv, lens, tree, dtype
    (1, 1, 8, 8, [1], False, E4M3),
    (1, 1, 8, 1, [0], False, E4M3),                      # nothing cached: the token itself
    (9, 1, 8, 2, [63, 64, 65, 127, 128, 129, 191, 192, 700], False, E5M2),  # block and tile edges
    (4, 5, 64, 8, [0, 63, 64, 2000], False, E4M3),       # sequence draft, 40 rows a head
    (3, 9, 16, 2, [0, 37, 300], True, E4M3),
    (2, 17, 12, 4, [129, 1007], True, E5M2),              # three query heads a head: 51 rows
    (2, 64, 8, 8, [100, 513], True, E4M3),                # 64 rows
    (2, 33, 8, 2, [511, 64], True, E4M3),                 # 132 rows: row blocks, the last one with 4
    (1, 64, 64, 8, [1000], True, E5M2),                   # 512 rows
    (2, 24, 48, 3, [300, 77], True, E4M3),                # 16 query heads a head
    (70, 2, 4, 2, [(i * 37) % 261 for i in range(70)], False, E4M3),
    (900, 1, 1, 1, [(i * 61) % 331 for i in range(900)], False, E5M2),  # more requests than a CTA has threads
]


@pytest.mark.parametrize("B,n,H,Hkv,lens,tree,dtype", ATTN)
def test_attention(B, n, H, Hkv, lens, tree, dtype):
    rng = np.random.default_rng(B * 1000 + n)
    got, cache, qkv, parents = _attend(rng, B, n, H, Hkv, lens, tree, dtype)
    _check(got, cache, qkv, parents, f"B={B} n={n} H={H}/{Hkv}")


def test_attention_of_a_long_request():
    rng = np.random.default_rng(1)
    got, cache, qkv, parents = _attend(rng, 2, 3, 4, 1, [30011, 640], False, E4M3)
    _check(got, cache, qkv, parents, "long")


def test_attention_in_a_layer_of_a_wider_projection_with_room():
    """Another layer than the first, rows of a projection with more columns, a
    bound of the lengths far above them."""
    rng = np.random.default_rng(2)
    got, cache, qkv, parents = _attend(rng, 3, 4, 8, 2, [200, 0, 70], True, E4M3, max_len=9000, wide=72, layers=3,
                                       layer=2)
    _check(got, cache, qkv, parents, "layer 2")


@pytest.mark.parametrize("scale", [0.02, 0.5])
def test_attention_with_rising_scores(scale):
    """Keys that grow along the request: the running maximum is raised again
    and again, by little and by much."""
    rng = np.random.default_rng(3)
    hist = []
    for L in (700, 1500):
        k, v = _history(rng, 2, L)
        grow = torch.linspace(0.05, 3.0, L)[None, :, None]
        hist.append(((k * grow).bfloat16(), v))
    got, cache, qkv, parents = _attend(rng, 2, 5, 8, 2, [700, 1500], False, E4M3, hist=hist, scale=scale)
    _check(got, cache, qkv, parents, "rising", scale=scale)


def test_attention_with_scales_far_apart():
    """Blocks whose values differ by many powers of two, a block of zeros, and
    a first token that takes almost all the weight and brings no value."""
    rng = np.random.default_rng(4)
    k, v = _history(rng, 1, 64 * 5 + 9)
    mult = torch.ones(64 * 5 + 9)
    mult[:64], mult[64:128], mult[128:192], mult[192:256] = 2.0 ** -40, 2.0 ** 20, 0.0, 2.0 ** -8
    tiny = (v * mult[None, :, None]).bfloat16()
    got, cache, qkv, parents = _attend(rng, 1, 4, 8, 1, [329], True, E4M3, hist=[(k, tiny)])
    _check(got, cache, qkv, parents, "scales")
    k, v = _history(rng, 1, 500)
    qkv, cols = _attn_inputs(rng, 1, 3, 4, 1)
    qkv = (qkv * 0.1 + 1.0).bfloat16()  # queries that agree with the first key
    k = (k * 0.05).bfloat16()
    k[0, 0], v[0, 0] = 1.0, 0.0
    got, cache, qkv, parents = _attend(rng, 1, 3, 4, 1, [500], False, E4M3, hist=[(k, v)], qkv=qkv)
    _check(got, cache, qkv, parents, "sink")


@pytest.mark.parametrize("junk", [float("nan"), float("inf")])
def test_attention_does_not_read_stale_rows(junk):
    """Tail rows past the length and unused pages hold NaN or infinities."""
    rng = np.random.default_rng(5)
    got, cache, qkv, parents = _attend(rng, 4, 6, 16, 2, [5, 64, 200, 0], True, E5M2, stale=junk)
    _check(got, cache, qkv, parents, "stale")


@pytest.mark.parametrize("junk", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("where", ["k", "v"])
def test_attention_keeps_a_bad_node_to_its_descendants(junk, where):
    """A NaN or infinity in one node's key or value reaches the rows that see
    the node, and no other."""
    rng = np.random.default_rng(6)
    n, H, Hkv = 12, 8, 2
    parents = np.stack([np.array([-1, 0, 0, 1, 2, 1, 3, 4, 4, 5, 6, 0], np.int32)] * 2)
    qkv, cols = _attn_inputs(rng, 2, n, H, Hkv)
    col = cols[1 if where == "k" else 2].start + 128 + 5  # head 1, column 5
    qkv[1, 3, col] = junk
    got, cache, qkv, parents = _attend(rng, 2, n, H, Hkv, [100, 70], True, E4M3, qkv=qkv, parents=parents)
    q, k, v = qkv
    sees = [3 in ref.root_path(parents[1], j) for j in range(n)]
    clean_k, clean_v = k.clone(), v.clone()
    clean_k[1, 3, 1, 5], clean_v[1, 3, 1, 5] = 0.0, 0.0
    for b in range(2):
        want, mag = ref.attention(cache.values[b], q[b], clean_k[b], clean_v[b], parents[b])
        for j in range(n):
            for h in range(H):
                hit = b == 1 and sees[j] and h // 4 == 1
                g = got[b, j, h]
                ok = (g - want[j, h]).abs() <= 1.05 * 2.0 ** -8 * (mag[j, h] + want[j, h].abs()) + 1e-6
                if not hit:
                    assert ok.all(), (b, j, h)
                elif where == "v":
                    ok[5] = True
                    assert ok.all() and (g[5].isnan() if junk != junk else g[5] == junk), (j, h)
                elif junk != junk:
                    assert g.isnan().all()


def test_attention_of_a_row_with_nan():
    """A query row with a NaN or an infinity is NaN; the others are not touched."""
    rng = np.random.default_rng(8)
    n, H, Hkv = 5, 8, 2
    qkv, cols = _attn_inputs(rng, 1, n, H, Hkv)
    qkv[0, 2, 3 * 128 + 7] = float("nan")
    qkv[0, 4, 6 * 128 + 1] = float("inf")
    got, cache, (q, k, v), parents = _attend(rng, 1, n, H, Hkv, [150], False, E4M3, qkv=qkv)
    assert got[0, 2, 3].isnan().all() and got[0, 4, 6].isnan().all()
    got[0, 2, 3], got[0, 4, 6] = 0.0, 0.0
    q = q.nan_to_num(0.0, 0.0, 0.0)
    want, mag = ref.attention(cache.values[0], q[0], k[0], v[0], parents[0])
    want[2, 3], want[4, 6] = 0.0, 0.0
    assert ((got[0] - want).abs() <= 1.05 * 2.0 ** -8 * (mag + want.abs()) + 1e-6).all()


def test_attention_reports_bad_input():
    rng = np.random.default_rng(9)
    B, n, H, Hkv, D = 3, 3, 8, 2, 128
    hist = [_history(rng, Hkv, L) for L in (130, 300, 20)]
    cache = ref.Cache(hist, E4M3, rng, 320)
    c, table, lens, tails = cache.to(sv, dev())
    qkv, cols = _attn_inputs(rng, B, n, H, Hkv)
    dq = [qkv.to(dev())[:, :, s].unflatten(2, (-1, D)) for s in cols]
    par = np.stack([ref.chain(n)] * B)

    def run(table=table, lens=lens, tails=tails, parents=None, max_len=320):
        out = sv.kv8_tree_attention(*dq, c, 0, table, lens, tails, max_len=max_len,
                                    tree_parents=None if parents is None else _i32(parents))
        torch.cuda.synchronize()
        return out.cpu(), sv.check_device_status()

    good, status = run()
    assert status == 0
    for b, j, value in ((1, 2, -1), (1, 0, 1 << 24)):
        t = table.clone()
        t[b, j] = value
        out, status = run(table=t)
        assert status == 5 and torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
    t = tails.clone()
    t[0] = 6
    out, status = run(tails=t)
    assert status == 5 and torch.equal(out[1:], good[1:])
    assert torch.isfinite(out).all()
    for value in (-4, 321):
        l = lens.clone()
        l[2] = value
        out, status = run(lens=l)  # the split of the work may change with the lengths: equal to rounding
        assert status == 5 and (out[:2].float() - good[:2].float()).abs().max() <= 2.0 ** -6 * good.float().abs().max()
    p = par.copy()
    p[1, 2], p[2, 1] = 2, -1
    out, status = run(parents=p)
    assert status == 5 and torch.equal(out[0], good[0]) and torch.isfinite(out).all()


def test_attention_is_the_same_each_time_and_on_another_stream():
    rng = np.random.default_rng(10)
    B, n, H, Hkv = 5, 5, 64, 8
    hist = [_history(rng, Hkv, L) for L in (900, 1, 64, 3000, 127)]
    cache = ref.Cache(hist, E4M3, rng, 3000)
    c, table, lens, tails = cache.to(sv, dev())
    qkv, cols = _attn_inputs(rng, B, n, H, Hkv)
    dq = [qkv.to(dev())[:, :, s].unflatten(2, (-1, 128)) for s in cols]
    run = lambda **kw: sv.kv8_tree_attention(*dq, c, 0, table, lens, tails, max_len=3000, **kw)
    first = run().cpu()
    s = torch.cuda.Stream()
    ws = torch.zeros(sv.kv8_tree_attention_workspace_bytes(B, n, H, Hkv, 128, 3000) + 256, dtype=torch.uint8, device=dev())
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        assert torch.equal(run().cpu(), first)
        out = run(stream=s, ws=ws)
        s.synchronize()
        assert torch.equal(out.cpu(), first)
    _status()


# ------------------------------------------------------ a step, in a graph

def test_a_step_replayed_from_a_graph():
    """Attention, plan and append of a draft step captured once and replayed
    with the lengths, tails and free list moving on the device."""
    rng = np.random.default_rng(11)
    B, n, H, Hkv, D = 3, 4, 8, 2, 128
    hist = [list(_history(rng, Hkv, L)) for L in (60, 0, 125)]
    steps = 6
    pages = 12
    cache = sv.kv8_cache(1, pages, B, Hkv, device=dev())
    table = _i32(np.full((B, 4), -1))
    ring, queue = _i32(rng.permutation(pages)), _i32([3, pages, 0])
    lens, tails = _i32(np.zeros(B)), _i32(2 * np.arange(B))
    start = np.concatenate([[0], np.cumsum([60, 0, 125])])
    rows = [torch.cat([hist[b][c].transpose(0, 1) for b in range(B)]).to(dev()) for c in range(2)]
    plan = sv.kv_block_plan(lens, tails, table, ring, queue, row_start=_i32(start), rows=185)
    sv.kv8_append(cache, rows[0], rows[1], tails, plan)
    lens.copy_(plan.new_lens), tails.copy_(plan.new_tails), queue.copy_(plan.queue)
    q = torch.zeros(B, n, H, D, dtype=torch.bfloat16, device=dev())
    k, v = (torch.zeros(B, n, Hkv, D, dtype=torch.bfloat16, device=dev()) for _ in range(2))
    node, out = _i32(np.zeros(B)), torch.empty_like(q)
    plan = sv.kv_block_plan(lens, tails, table, ring, queue, accepted_node=node, n=n)
    ws = torch.zeros(sv.kv8_tree_attention_workspace_bytes(B, n, H, Hkv, D, 250) + 256, dtype=torch.uint8, device=dev())

    def step():
        sv.kv8_tree_attention(q, k, v, cache, 0, table, lens, tails, max_len=250, out=out, ws=ws)
        sv.kv_block_plan(lens, tails, table, ring, queue, accepted_node=node, n=n, plan=plan)
        sv.kv8_append(cache, k.flatten(0, 1), v.flatten(0, 1), tails, plan)
        lens.copy_(plan.new_lens), tails.copy_(plan.new_tails), queue.copy_(plan.queue)

    sv.kv8_tree_attention(q, k, v, cache, 0, table, lens, tails, max_len=250, out=out, ws=ws)  # loads the kernel
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        graph.capture_begin()
        step()
        graph.capture_end()
    torch.cuda.synchronize()
    for i in range(steps):
        hq, hk, hv = (torch.from_numpy(rng.standard_normal(t.shape)).bfloat16() for t in (q, k, v))
        hn = rng.integers(0, n, B)
        q.copy_(hq), k.copy_(hk), v.copy_(hv), node.copy_(_i32(hn))
        ref_cache = ref.Cache(hist, E4M3, rng, 256)
        torch.cuda.synchronize()
        graph.replay()
        _status()
        _check(out.cpu().double(), ref_cache, (hq, hk, hv), [ref.chain(n)] * B, f"step {i}")
        for b in range(B):
            for c, new in enumerate((hk, hv)):
                hist[b][c] = torch.cat([hist[b][c], new[b, :hn[b] + 1].transpose(0, 1)], 1)
        assert np.array_equal(lens.cpu().numpy(), [h[0].shape[1] for h in hist])
