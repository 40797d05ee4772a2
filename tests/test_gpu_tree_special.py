"""GPU: attention of drafted tokens where a query, a key or a value is not finite.

What a row sees decides: a score that is NaN makes the row's out and lse NaN, in both forms of
the kernel, however the keys are divided among warps and CTAs; rows that do not see it keep
what they have without it. The reference is the fp64 oracle on the cache's values with the
rows in question left out, and the tolerances are test_gpu_tree.py's.
"""
import numpy as np
import pytest
import torch

import oracle
from sequence_exact_attention_ring_b200 import cache_read, cache_write, status, tree_attention, tree_workspace
from test_gpu_tree import FORMATS, check, i32, make, weight_floor

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
# (T, query heads per kv head): one token and a short chain (at most 16 rows), a tree of 80 rows
FORMS = [(1, 4), (3, 4), (20, 4)]


def poison(cache, b, h, row, what, value=NAN, block=1):
    """Put `value` into one 32-value block of cache row `row` of K or V (a block that is not finite)."""
    t, s = (cache.k, cache.k_scale) if what == "k" else (cache.v, cache.v_scale)
    if cache.format == "bf16":
        t[b, h, row, 32 * block + 5] = value
    else:
        s[b, h, row, block] = 255
        per = 32 if cache.format == "mxfp8" else 16
        t[b, h, row, per * block:per * (block + 1)] = 0


def attend(q, cache, lengths, parents=None, **kw):
    ws = tree_workspace(q, cache)
    out, lse = tree_attention(q, cache, i32(lengths), None if parents is None else i32(parents), workspace=ws, **kw)
    assert status(ws) == 0
    return out, lse


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [0, 15, 16, 31, 32, 33, 63, 64, 127, 128, 255, 256, 700])
def test_new_token_whose_key_is_not_finite(cuda_lib, fmt, D, n):
    """The new token's key, alone in its step, tile or part at some of these lengths: every node of the
    chain sees it. The other kv head's rows are untouched."""
    for T, rep in FORMS:
        q, cache, _ = make(1, 2 * rep, 2, D, T, [n], fmt, 301)
        want = tree_attention(q, cache, i32([n]))
        poison(cache, 0, 1, n, "k")
        out, lse = attend(q, cache, [n])
        assert torch.isnan(lse[:, rep:]).all(), (T, rep)
        assert torch.isnan(out[:, rep:]).all(), (T, rep)
        assert torch.equal(out[:, :rep], want[0][:, :rep]) and torch.equal(lse[:, :rep], want[1][:, :rep])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128])
def test_written_nan_and_infinity(cuda_lib, fmt, D):
    """A row whose keys were NaN or infinite when they were written, committed long ago."""
    for T, rep in FORMS:
        for value in (NAN, INF):
            q, cache, _ = make(2, 2 * rep, 2, D, T, [300, 40], fmt, 302)
            new = torch.ones(2, 2, 1, D, device="cuda")
            new[1, 0, 0, 3] = value
            cache_write(cache, new, torch.ones_like(new), i32([17, 17]))
            out, lse = attend(q, cache, [300, 40])
            # (an infinite key in a bf16 row gives a score of plus or minus infinity: the latter weighs nothing)
            if fmt == "bf16" and value == INF:
                up = (q[1, :rep, :, 3] > 0)
                assert torch.isnan(lse[1, :rep][up]).all() and torch.isnan(out[1, :rep][up]).all()
                assert torch.isfinite(lse[1, :rep][~up]).all()
            else:
                assert torch.isnan(lse[1, :rep]).all() and torch.isnan(out[1, :rep]).all()
            assert torch.isfinite(out[0]).all() and torch.isfinite(out[1, rep:]).all()
            assert torch.isfinite(lse[0]).all() and torch.isfinite(lse[1, rep:]).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [0, 10, 300, 5000])
def test_query_row_that_is_nan(cuda_lib, fmt, D, n):
    """One query row is NaN: its row of out and lse is NaN, every other is what it is without it. (Not bit by
    bit: a row's reference moves, to its own maximum, whenever that of any row of its warp passes its own by
    the margin, so the rounding of a row's weights depends on its neighbours; the tolerance covers any
    reference.)"""
    for T, rep in FORMS:
        q, cache, vals = make(2, 2 * rep, 2, D, T, [n, n // 2], fmt, 303)
        want = oracle.tree_reference(q.double().cpu().numpy(), *vals, [n, n // 2], None, None, 0, 0, D ** -0.5)
        bad = q.clone()
        bad[1, rep + 1, T - 1, 7] = NAN
        out, lse = attend(bad, cache, [n, n // 2])
        assert torch.isnan(out[1, rep + 1, T - 1]).all() and torch.isnan(lse[1, rep + 1, T - 1]), (T, rep)
        keep = torch.ones_like(lse, dtype=torch.bool)
        keep[1, rep + 1, T - 1] = False
        keep_np = keep.cpu().numpy()
        check(out[keep], lse[keep], tuple(x[keep_np] for x in want), D, f"{T}", weight_floor(cache, vals, [n, n // 2], T))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128])
def test_all_keys_not_finite(cuda_lib, fmt, D):
    """No finite score anywhere, in one part and in many: NaN, not the zeros of a row that sees nothing."""
    for T, rep in FORMS:
        for n in (5, 600):
            q, cache, _ = make(1, rep, 1, D, T, [n], fmt, 304)
            for row in range(n + T):
                poison(cache, 0, 0, row, "k", block=row % 2)
            out, lse = attend(q, cache, [n])
            assert torch.isnan(out).all() and torch.isnan(lse).all(), (T, rep, n)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("exp", [0, -24])
def test_key_that_only_some_nodes_see(cuda_lib, fmt, D, exp):
    """A drafted node's key is not finite: it and its descendants come out NaN, the other branch of the tree
    exactly as well as ever (also where its keys and values are small against any fixed reference)."""
    parents = {3: [-1, -1, 1], 4: [-1, 0, -1, 2], 20: [*range(-1, 9), -1, *range(10, 19)]}
    for T, rep, n in ((3, 1, 29), (4, 4, 100), (20, 4, 300), (20, 4, 0)):
        par = parents[T]
        assert all(-1 <= x < i for i, x in enumerate(par))
        q, cache, _ = make(1, rep, 1, D, T, [n], fmt, 305)
        g = torch.Generator().manual_seed(306)
        new = torch.randn(2, 1, 1, n + T, D, generator=g)
        cache_write(cache, (new[0] * 2.0 ** exp).bfloat16().cuda(), (new[1] * 2.0 ** exp).bfloat16().cuda(), i32([0]))
        q = (q.float() * 2.0 ** -exp).bfloat16()
        poison(cache, 0, 0, n, "k")
        out, lse = attend(q, cache, [n], [par])
        vals = [t.double().cpu().numpy() for t in cache_read(cache, i32([0]), cache.capacity, dtype=torch.float32)]
        ref = oracle.tree_reference(q.double().cpu().numpy(), *vals, [n], [par], None, 0, 0, D ** -0.5)
        below = np.zeros(T, dtype=bool)
        for i in range(T):
            below[i] = i == 0 or (par[i] >= 0 and below[par[i]])
        assert below.any() and not below.all()
        bad = torch.from_numpy(below).cuda()
        assert torch.isnan(out[0][:, bad]).all() and torch.isnan(lse[0][:, bad]).all()
        keep = torch.zeros_like(lse, dtype=torch.bool)
        keep[:, :, ~bad] = True
        keep_np = keep.cpu().numpy()
        check(out[keep], lse[keep], tuple(x[keep_np] for x in ref), D, f"{T} {n}", weight_floor(cache, vals, [n], T))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("exp", [0, -24])
def test_value_block_that_is_not_finite(cuda_lib, fmt, D, exp):
    """A block of one committed row of V is not finite: out is NaN in the dimensions that it holds, and what
    it would be without it in the others; lse has nothing to do with V."""
    for T, rep, n in ((1, 4, 200), (3, 4, 700), (20, 4, 700)):
        q, cache, _ = make(1, rep, 1, D, T, [n], fmt, 307)
        g = torch.Generator().manual_seed(308)
        v = (torch.randn(1, 1, n + T, D, generator=g) * 2.0 ** exp).bfloat16().cuda()
        cache_write(cache, torch.randn(1, 1, n + T, D, generator=g).bfloat16().cuda(), v, i32([0]))
        poison(cache, 0, 0, 37, "v")
        out, lse = attend(q, cache, [n])
        vals = [t.double().cpu().numpy() for t in cache_read(cache, i32([0]), cache.capacity, dtype=torch.float32)]
        hit = np.isnan(vals[1][0, 0, 37])
        assert hit[32:64].any() and not hit[:32].any()
        assert torch.isnan(out[..., torch.from_numpy(hit).cuda()]).all()
        vals[1][0, 0, 37, hit] = 0.0
        ref = oracle.tree_reference(q.double().cpu().numpy(), *vals, [n], None, None, 0, 0, D ** -0.5)
        O, L, A, E = ref
        keep = ~hit
        check(out[..., torch.from_numpy(keep).cuda()], lse, (O[..., keep], L, A[..., keep], E), D, f"{T}",
              weight_floor(cache, vals, [n], T))
