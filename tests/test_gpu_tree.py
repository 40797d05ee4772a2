"""GPU: attention of drafted tokens over a cache, against the fp64 oracle on the cache's values.

Tolerances are counted, per element, from the magnitudes the oracle returns (A = sum p|v|,
E = scale sum |q||k|): each weight p is rounded to bf16 for its product (2^-8 A), the result
once more (2^-8 |O| <= 2^-8 A); a score is a sum of D products accumulated in fp32, off by at
most D 2^-23 E (twice the half-step bound, for a truncating adder), and enters a weight and
the weights' sum (2 D 2^-23 E A); 2^x is good to 2^-22, sums and rescales to a few 2^-23 (the
2^-16 covers them at these lengths). A microscaled cache may be read with the weights in fp16
(11 bits, better than bf16's 8) scaled so that its smallest step is 2^-33: a weight below 2^-23 is
off by at most 2^-34 of the row's largest, which adds 2^-34 |v| per key, whatever A is.
"""
import numpy as np
import pytest
import torch

import oracle
from sequence_exact_attention_ring_b200 import (KVCache, RingAttnError, binding, cache_read, cache_write, merge, status,
                                                tree_attention, tree_workspace, window_attention)

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check(out, lse, ref, D, what="", floor=0.0):
    O, L, A, E = ref
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    seen = np.isfinite(L)
    assert (np.isneginf(l) == ~seen).all(), what
    assert (o[~seen] == 0).all(), what
    es = D * 2.0 ** -23 * E + 2.0 ** -16
    tol = A * (2.0 ** -8 + 2.0 ** -8 + 2 * es[..., None]) + 2.0 ** -126 + floor
    assert np.isfinite(o).all(), what
    worst = (np.abs(o - O) / tol).max()
    assert worst <= 1, f"{what}: out off by {worst:.2f} of its tolerance"
    d = np.abs(l[seen] - L[seen])
    t = (es + 2.0 ** -22 * (np.abs(np.where(seen, L, 0)) + 4))[seen]
    assert (d <= t).all(), f"{what}: lse off by {(d / t).max():.2f} of its tolerance"


def make(B, Hq, Hkv, D, T, lengths, fmt, seed, cap=None, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    cap = cap or (max(lengths) + T + 15) // 16 * 16
    cache = KVCache.allocate(B, Hkv, cap, D, fmt)
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        if t is not None:
            t.view(torch.uint8).fill_(0xff)  # rows that are never written read as NaN
    k = torch.randn(B, Hkv, cap, D, generator=g)
    v = torch.randn(B, Hkv, cap, D, generator=g) + 0.5
    k[..., 3::29] *= 4
    k, v = k.bfloat16().cuda(), v.bfloat16().cuda()
    for b in range(B):  # committed rows and drafts
        n = lengths[b] + T
        one = KVCache(fmt, *(None if t is None else t[b:b + 1] for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)))
        cache_write(one, k[b:b + 1, :, :n], v[b:b + 1, :, :n], i32([0]))
    q = (spread * torch.randn(B, T, Hq, D, generator=g)).bfloat16().cuda().transpose(1, 2)
    vals = [t.double().cpu().numpy() for t in cache_read(cache, i32([0] * B), cap)]
    return q, cache, vals


def random_tree(B, T, seed):
    r = np.random.default_rng(seed)
    return [[-1 if i == 0 else int(r.integers(-1, i)) for i in range(T)] for _ in range(B)]


def weight_floor(cache, vals, lengths, T):
    """2^-34 sum |v| over a sequence's keys, at most (0 for bf16 rows)."""
    if cache.format == "bf16":
        return 0.0
    top = max(np.abs(vals[1][b, :, :n + T]).max(initial=0, where=np.isfinite(vals[1][b, :, :n + T])) * (n + T)
              for b, n in enumerate(lengths))
    return 2.0 ** -34 * top


def run(q, cache, vals, lengths, parents=None, counts=None, window=0, sinks=0, scale=None, what="", floor=None):
    D = q.shape[-1]
    ws = tree_workspace(q, cache)
    out, lse = tree_attention(q, cache, i32(lengths), None if parents is None else i32(parents),
                              None if counts is None else i32(counts), window, sinks, scale, workspace=ws)
    assert status(ws) == 0
    ref = oracle.tree_reference(q.double().cpu().numpy(), *vals, lengths, parents, counts, window, sinks,
                                1 / np.sqrt(D) if scale is None else scale)
    check(out, lse, ref, D, what, weight_floor(cache, vals, lengths, q.shape[2]) if floor is None else floor)
    return out, lse


FORMATS = ["bf16", "mxfp8", "mxfp4"]
SHAPES = [
    # B, Hq, Hkv, T, lengths
    (1, 1, 1, 1, [0]),                     # the drafted token alone
    (1, 2, 2, 1, [1]),
    (3, 4, 2, 1, [15, 16, 17]),            # around a step's end
    (2, 8, 1, 1, [700, 0]),                # grouped heads, an empty cache in the batch
    (2, 4, 4, 3, [64, 63]),
    (1, 32, 1, 5, [333]),                  # 160 rows: ten row groups
    (2, 6, 2, 33, [129, 260]),             # 99 rows per kv head: a ragged last group
    (1, 4, 1, 64, [500]),
]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s[:4])))
def test_trees_against_oracle(cuda_lib, fmt, D, shape):
    B, Hq, Hkv, T, lengths = shape
    q, cache, vals = make(B, Hq, Hkv, D, T, lengths, fmt, 11)
    run(q, cache, vals, lengths, random_tree(B, T, 5), what="tree")
    run(q, cache, vals, lengths, what="chain")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 3), (16, 0), (17, 5), (100, 1), (100, 40), (5000, 3),
                                          (130, 1000)])
def test_window_and_sinks(cuda_lib, fmt, window, sinks):
    """Windows from one position to past the start, also shorter than the drafted tree is deep."""
    B, T = 3, 21
    lengths = [401, 3, 96]
    q, cache, vals = make(B, 4, 2, 128, T, lengths, fmt, 21)
    run(q, cache, vals, lengths, random_tree(B, T, 6), window=window, sinks=sinks, what="tree")
    run(q, cache, vals, lengths, window=window, sinks=sinks, what="chain")
    q1, cache, vals = make(B, 4, 2, 64, 1, lengths, fmt, 22)
    run(q1, cache, vals, lengths, window=window, sinks=sinks, what="token")


@pytest.mark.parametrize("fmt", FORMATS)
def test_counts_and_dead_rows(cuda_lib, fmt):
    """Dead nodes give 0 and -inf; rows behind the last node and rows that fell out of every window hold NaN."""
    B, T, lengths, counts = 4, 9, [300, 40, 0, 200], [9, 1, 4, 0]
    q, cache, vals = make(B, 4, 2, 128, T, lengths, fmt, 31, cap=512)
    for b in range(B):
        for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
            if t is not None:
                t[b, :, lengths[b] + counts[b]:].view(torch.uint8).fill_(0xff)
    run(q, cache, vals, lengths, random_tree(B, T, 7), counts, what="counts")
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        if t is not None:
            t[0, :, 3:300 - 50 + 1].view(torch.uint8).fill_(0xff)
    run(q, cache, vals, lengths, random_tree(B, T, 7), counts, window=50, sinks=3, what="evicted rows")


def test_large_scores_and_far_scales(cuda_lib):
    """Scores far apart (one key wins), rising maxima, tiny and large block scales."""
    for fmt in FORMATS:
        q, cache, vals = make(2, 4, 2, 128, 4, [600, 77], fmt, 41, spread=40.0)
        run(q, cache, vals, [600, 77], what="spread " + fmt)
    g = torch.Generator().manual_seed(9)
    for fmt in ("mxfp8", "mxfp4"):
        for e in (-100, -40, 40, 60):
            cache = KVCache.allocate(1, 1, 64, 64, fmt)
            k = torch.randn(1, 1, 64, 64, generator=g) * 2.0 ** e
            v = torch.randn(1, 1, 64, 64, generator=g) * 2.0 ** -e
            cache_write(cache, k.cuda(), v.cuda(), i32([0]))
            vals = [t.double().cpu().numpy() for t in cache_read(cache, i32([0]), 64, dtype=torch.float32)]
            q = (torch.randn(1, 2, 1, 64, generator=g) * (2.0 ** -e if e > -100 else 1.0)).bfloat16().cuda()
            run(q, cache, vals, [63], what=f"{fmt} 2^{e}")
    # scales of one step far apart: rows and blocks 2^-40 .. 2^40 of one another, the largest values with small weights
    for fmt in ("mxfp8", "mxfp4"):
        cache = KVCache.allocate(1, 1, 96, 128, fmt)
        k, v = torch.randn(1, 1, 96, 128, generator=g), torch.randn(1, 1, 96, 128, generator=g)
        v[0, 0, 5] *= 2.0 ** 40
        k[0, 0, 5] = 0.0
        v[0, 0, 40:] *= torch.exp2(torch.arange(56.0) - 40)[:, None]
        v[0, 0, 20, 32:64] *= 2.0 ** -30
        k[0, 0, 21, 64:] *= 2.0 ** -40
        k[0, 0, 50:52] *= 2.0 ** -20
        cache_write(cache, k.cuda(), v.cuda(), i32([0]))
        vals = [t.double().cpu().numpy() for t in cache_read(cache, i32([0]), 96, dtype=torch.float32)]
        q = (8 * torch.randn(1, 4, 2, 128, generator=g)).bfloat16().cuda()
        run(q, cache, vals, [90], what=f"{fmt} mixed scales", floor=0.0)
        run(q, cache, vals, [4], what=f"{fmt} mixed scales, short", floor=0.0)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("D", [64, 128])
def test_many_rows_and_far_scales(cuda_lib, fmt, D):
    """Tiles of every mix: ordinary, blocks of zeros, K or V scales past fp16's range, 2^-40 to 2^40 in one tile,
    scores that rise from tile to tile."""
    g = torch.Generator().manual_seed(43)
    n, T = 900, 20
    cache = KVCache.allocate(1, 1, n + T + 12, D, fmt)
    k, v = torch.randn(1, 1, n + T, D, generator=g), torch.randn(1, 1, n + T, D, generator=g)
    k[0, 0, 130:250], v[0, 0, 140:384] = 0.0, 0.0                  # zero blocks, a V tile of zeros alone
    k[0, 0, 260:270] *= 2.0 ** -30                                  # a K tile below the range
    v[0, 0, 400:405] *= 2.0 ** 20                                   # a V tile above it, weights small
    k[0, 0, 400:405] = 0.0
    v[0, 0, 520:640] *= torch.exp2(torch.arange(120.0) / 3 - 40)[:, None]
    k[0, 0, 530, 32:] *= 2.0 ** -60
    k[0, 0, 640:] *= torch.linspace(0.5, 4, n + T - 640)[:, None]   # rising maxima
    cache_write(cache, k.cuda(), v.cuda(), i32([0]))
    vals = [t.double().cpu().numpy() for t in cache_read(cache, i32([0]), cache.capacity, dtype=torch.float32)]
    q = (3 * torch.randn(1, 6, T, D, generator=g)).bfloat16().cuda()
    run(q, cache, vals, [n], random_tree(1, T, 8), what="tree")
    run(q, cache, vals, [n], window=300, sinks=150, what="window")
    run(q, cache, vals, [0], what="drafts alone")
    run(q[:, :, :1].expand(1, 6, 1, D)[:, :2], cache, vals, [n + T - 1], what="one token")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128])
def test_references_that_move_at_every_tile(cuda_lib, fmt, D):
    """Scores that rise by more than a reference holds from tile to tile, for rows of the tiled form:
    the output is rescaled at every tile, behind every product so far; the same bits every time."""
    g = torch.Generator().manual_seed(44)
    n, T = 3000, 33
    q = torch.randn(1, 4, T, D, generator=g).abs().bfloat16().cuda()
    k = torch.rand(1, 1, n + T, D, generator=g) * torch.linspace(0.02, 8, n + T)[:, None] * (128 / D)
    v = torch.randn(1, 1, n + T, D, generator=g)
    cache = KVCache.allocate(1, 1, n + T, D, fmt)
    cache_write(cache, k.cuda(), v.cuda(), i32([0]))
    vals = [t.double().cpu().numpy() for t in cache_read(cache, i32([0]), cache.capacity, dtype=torch.float32)]
    o, l = run(q, cache, vals, [n], what="rising")
    for _ in range(20):
        o2, l2 = tree_attention(q, cache, i32([n]))
        assert torch.equal(o, o2) and torch.equal(l, l2)


def test_window_prefill_then_decode(cuda_lib):
    """A windowed layer's prompt, its rows written to a cache, and its last tokens again as a chain over
    the cache: the rows of the whole prompt's attention."""
    B, Hq, Hkv, D, S, W, sinks = 2, 8, 2, 128, 700, 200, 5
    g = torch.Generator().manual_seed(97)
    q, k, v = (torch.randn(B, h, S, D, generator=g).bfloat16().cuda() for h in (Hq, Hkv, Hkv))
    out, lse = window_attention(q, k, v, W, sinks)
    O, L, A, E = oracle.window_reference(*(x.double().cpu().numpy() for x in (q, k, v)), W, sinks, D ** -0.5)
    check(out, lse, (O, L, A, E), D, "prompt")
    cache = KVCache.allocate(B, Hkv, S, D, "bf16")
    cache_write(cache, k, v, i32([0] * B))
    for T in (1, 3, 64):
        o, l = tree_attention(q[:, :, S - T:], cache, i32([S - T] * B), window=W, sinks=sinks)
        check(o, l, tuple(x[:, :, S - T:] for x in (O, L, A, E)), D, f"last {T}")


def test_other_streams_and_two_at_once(cuda_lib):
    """Calls follow the stream they are given, and two of them with their own workspaces do not meet."""
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for T, rep in ((1, 4), (9, 8)):
        q, cache, vals = make(2, 2 * rep, 2, 128, T, [5000, 300], "mxfp8", 45)
        n = i32([5000, 300])
        want = tree_attention(q, cache, n)
        got = []
        torch.cuda.synchronize()
        for s in (a, b):
            ws = tree_workspace(q, cache)
            late, len_late = torch.zeros_like(q), torch.zeros_like(n)
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                torch.cuda._sleep(2_000_000)  # the inputs come late on the call's own stream
                late.copy_(q)
                len_late.copy_(n)
            got += [tree_attention(late, cache, len_late, workspace=ws, stream=s, out=torch.empty_like(want[0]),
                                   lse=torch.empty_like(want[1])) for _ in range(3)]
        torch.cuda.synchronize()
        for o, l in got:
            assert torch.equal(o, want[0]) and torch.equal(l, want[1])


def test_two_graphs_with_one_workspace(cuda_lib):
    """Captured calls of different shapes that share a workspace, replayed in any order on one stream."""
    s = torch.cuda.Stream()
    cases, ws = [], None
    for T, rep, fmt in ((1, 4, "mxfp8"), (30, 8, "mxfp4")):
        q, cache, vals = make(2, 2 * rep, 2, 64, T, [3000, 1700], fmt, 46)
        n = i32([3000, 1700])
        x = tree_workspace(q, cache)
        ws = x if ws is None or x.nbytes > ws.nbytes else ws
        cases.append([q, cache, n, tree_attention(q, cache, n)])
    torch.cuda.synchronize()
    for c in cases:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
            got = tree_attention(c[0], c[1], c[2], workspace=ws)
        c += [graph, got]
    for i in (0, 1, 1, 0, 1, 0, 0):
        for t in cases[i][5]:
            t.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            cases[i][4].replay()
        torch.cuda.synchronize()
        assert torch.equal(cases[i][5][0], cases[i][3][0]) and torch.equal(cases[i][5][1], cases[i][3][1])


def test_windows_past_every_int(cuda_lib):
    """A window or sinks too large for the sequence, or for a C int, hold all of it."""
    for T in (1, 20):
        q, cache, vals = make(1, 4, 2, 64, T, [200], "mxfp8", 47)
        for kw in (dict(window=2 ** 31 - 1), dict(window=2 ** 32), dict(window=2 ** 40 + 1, sinks=2 ** 33),
                   dict(window=1, sinks=2 ** 31 - 1)):
            got = tree_attention(q, cache, i32([200]), **kw)
            ref = oracle.tree_reference(q.double().cpu().numpy(), *vals, [200], None, None, kw["window"],
                                        kw.get("sinks", 0), 1 / 8)
            check(*got, ref, 64, str(kw), weight_floor(cache, vals, [200], T))


@pytest.mark.parametrize("fmt", FORMATS)
def test_long_cache_splits_and_repeats(cuda_lib, fmt):
    """Long enough that every unit is split over many CTAs; ragged; the same bits twice."""
    lengths = [20011, 333, 8192]
    q, cache, vals = make(3, 4, 1, 128, 2, lengths, fmt, 51)
    o1, l1 = run(q, cache, vals, lengths, what="long")
    o2, l2 = tree_attention(q, cache, i32(lengths))
    assert torch.equal(o1, o2) and torch.equal(l1, l2)


def test_offsets_past_32_bits(cuda_lib):
    """A cache of more than 2^32 bytes per tensor: the last sequence's rows lie past a 32-bit offset."""
    B, Hkv, cap, D = 5, 8, 1 << 20, 128
    cache = KVCache("mxfp8", *(torch.empty(B, Hkv, cap, D, dtype=torch.uint8, device="cuda") for _ in range(2)),
                    *(torch.empty(B, Hkv, cap, D // 32, dtype=torch.uint8, device="cuda") for _ in range(2)))
    g = torch.Generator(device="cuda").manual_seed(3)
    new = torch.randn(B, Hkv, 80, D, generator=g, device="cuda").bfloat16()
    start = [0, 0, 0, 0, cap - 80]
    cache_write(cache, new, -new, i32(start))
    ko, vo = cache_read(cache, i32(start), 80)
    assert torch.equal(ko, -vo)
    want = oracle.quantise(new[4, 7].double().cpu().numpy(), "mxfp8")[2]
    np.testing.assert_array_equal(ko[4, 7].double().cpu().numpy(), want)
    # a window over the end of the last sequence's full cache
    q = torch.randn(B, 8, 1, D, generator=g, device="cuda").bfloat16()
    lengths = [79, 79, 79, 79, cap - 1]
    out, lse = tree_attention(q, cache, i32(lengths), window=80)
    vals = [t.double().cpu().numpy() for t in (ko, vo)]
    ref = oracle.tree_reference(q.double().cpu().numpy(), *vals, [79] * 5, None, None, 80, 0, 1 / np.sqrt(D))
    check(out, lse, ref, D)


def test_draft_verify_accept(cuda_lib):
    """The operators as they are used: a prompt's rows, a drafted tree behind them, its attention, the
    accepted path written over the drafts, the next token; equal to attention over the plain sequence."""
    B, Hq, Hkv, D, n, T = 2, 4, 2, 128, 200, 6
    g = torch.Generator().manual_seed(61)
    for fmt in FORMATS:
        cache = KVCache.allocate(B, Hkv, 512, D, fmt)
        prompt = torch.randn(2, B, Hkv, n, D, generator=g).bfloat16().cuda()
        cache_write(cache, prompt[0], prompt[1], i32([0, 0]))
        draft = torch.randn(2, B, Hkv, T, D, generator=g).bfloat16().cuda()
        cache_write(cache, draft[0], draft[1], i32([n, n]))
        parents = [[-1, 0, 0, 1, 2, 4], [-1, -1, 1, 1, 3, 0]]
        q = torch.randn(B, Hq, T, D, generator=g).bfloat16().cuda()
        out, lse = tree_attention(q, cache, i32([n, n]), i32(parents))
        path, count = [[0, 2, 4], [1, 3, 0]], [3, 2]  # accepted nodes, root first
        cache_write(cache, draft[0], draft[1], i32([n, n]), count=i32(count), index=i32(path))
        # each accepted node's row equals plain attention over prompt + path up to it
        vals = [t.double().cpu().numpy() for t in cache_read(cache, i32([0, 0]), 512)]
        for b in range(B):
            for i in range(count[b]):
                o1, l1, A, E = oracle.tree_reference(q[b:b + 1, :, path[b][i]:path[b][i] + 1].double().cpu().numpy(),
                                                     *(x[b:b + 1] for x in vals), [n + i], None, None, 0, 0, D ** -0.5)
                check(out[b:b + 1, :, path[b][i]:path[b][i] + 1], lse[b:b + 1, :, path[b][i]:path[b][i] + 1],
                      (o1, l1, A, E), D, f"{fmt} {b} {i}")
        new = torch.randn(2, B, Hkv, 1, D, generator=g).bfloat16().cuda()
        lengths = [n + c for c in count]
        cache_write(cache, new[0], new[1], i32(lengths))
        vals = [t.double().cpu().numpy() for t in cache_read(cache, i32([0, 0]), 512)]
        run(q[:, :, :1], cache, vals, lengths, what="next token")


def test_split_cache_merges(cuda_lib):
    """Two caches over two halves of the keys: their (out, lse) merge to attention over both."""
    q, cache, vals = make(1, 4, 2, 128, 1, [300], "mxfp8", 71)
    whole, lse = tree_attention(q, cache, i32([300]))
    parts = []
    for lo, hi in ((0, 160), (160, 301)):
        half = KVCache.allocate(1, 2, 512, 128, "mxfp8")
        for a, b in ((half.k, cache.k), (half.v, cache.v), (half.k_scale, cache.k_scale), (half.v_scale, cache.v_scale)):
            a[:, :, :hi - lo] = b[:, :, lo:hi]
        parts.append(tree_attention(q, half, i32([hi - lo - 1])))
    o, l = merge(torch.stack([p[0].float() for p in parts]), torch.stack([p[1] for p in parts]), torch.float32)
    ref = oracle.tree_reference(q.double().cpu().numpy(), *vals, [300], None, None, 0, 0, 128 ** -0.5)
    # the halves' outputs were rounded to bf16 once more on the way
    assert (np.abs(o.double().cpu().numpy() - ref[0]) <= 3 * 2.0 ** -8 * ref[2] + 2.0 ** -12).all()
    assert (l - lse).abs().max().item() <= 1e-4


def test_bad_sequences_and_parents_are_reported(cuda_lib):
    q, cache, vals = make(3, 2, 2, 64, 2, [40, 40, 40], "mxfp8", 81, cap=48)
    ws = tree_workspace(q, cache)
    out, lse = tree_attention(q, cache, i32([40, -1, 47]), workspace=ws)  # 47 + 2 rows do not fit in 48
    assert status(ws) == binding.EINVAL
    ref = oracle.tree_reference(q.double().cpu().numpy(), *vals, [40, 0, 0], None, [2, 0, 0], 0, 0, 1 / 8)
    check(out, lse, ref, 64)
    out, lse = tree_attention(q, cache, i32([40, 40, 40]), i32([[-1, 1], [5, 0], [-7, -1]]), workspace=ws)
    assert status(ws) == binding.EINVAL
    ref = oracle.tree_reference(q.double().cpu().numpy(), *vals, [40] * 3, [[-1, -1], [-1, 0], [-1, -1]], None, 0, 0, 1 / 8)
    check(out, lse, ref, 64)
    tree_attention(q, cache, i32([40, 40, 40]), workspace=ws)
    assert status(ws) == 0
    tree_attention(q, cache, i32([40, 40, 40]), counts=i32([2, 3, -1]), workspace=ws)
    assert status(ws) == binding.EINVAL


def test_refusals(cuda_lib):
    q, cache, _ = make(1, 2, 2, 64, 2, [10], "mxfp8", 91)
    for bad in (dict(lengths=torch.tensor([10], device="cuda")), dict(parents=i32([[0]])), dict(counts=i32([1, 1]))):
        a = dict(lengths=i32([10])) | bad
        with pytest.raises(ValueError):
            tree_attention(q, cache, **a)
    for x in (q.float(), q[0], q[..., :32], q.transpose(2, 3).contiguous().transpose(2, 3)):
        with pytest.raises(ValueError):
            tree_attention(x, cache, i32([10]))
    with pytest.raises(RingAttnError) as e:
        tree_attention(q, cache, i32([10]), workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.code == binding.EWORKSPACE
    for kw in (dict(window=-1), dict(sinks=-1), dict(scale=0.0), dict(scale=float("nan"))):
        with pytest.raises(RingAttnError) as e:
            tree_attention(q, cache, i32([10]), **kw)
        assert e.value.code == binding.EINVAL
    with pytest.raises(RingAttnError):
        tree_attention(torch.empty(1, 2, 65, 64, dtype=torch.bfloat16, device="cuda"), cache, i32([10]))
    with pytest.raises(RingAttnError):
        tree_attention(torch.empty(1, 3, 1, 64, dtype=torch.bfloat16, device="cuda"), cache, i32([10]))
    with pytest.raises(RingAttnError) as e:
        flat = torch.empty(1 * 2 * 2 * 64 + 8, dtype=torch.bfloat16, device="cuda")
        tree_attention(flat[4:260].view(1, 2, 2, 64), cache, i32([10]))
    assert e.value.code == binding.EALIGN


def test_graph_replay_follows_the_lengths(cuda_lib):
    """One captured call replayed as the sequences grow; lengths, counts and parents are read on the device."""
    B, T = 2, 3
    q, cache, vals = make(B, 4, 2, 128, T, [3000, 2000], "mxfp4", 95, cap=4096)
    lengths, par = i32([1, 1]), i32(random_tree(B, T, 1))
    ws = tree_workspace(q, cache)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        tree_attention(q, cache, lengths, par, workspace=ws)
        with torch.cuda.graph(graph, stream=s):
            out, lse = tree_attention(q, cache, lengths, par, workspace=ws)
    for n, seed in (([0, 17], 2), ([3000, 2000], 3)):
        tree = random_tree(B, T, seed)
        lengths.copy_(i32(n))
        par.copy_(i32(tree))
        graph.replay()
        torch.cuda.synchronize()
        ref = oracle.tree_reference(q.double().cpu().numpy(), *vals, n, tree, None, 0, 0, 128 ** -0.5)
        check(out, lse, ref, 128, str(n))
