"""GPU: causal attention with a sliding window and sinks, forward and gradients, against the fp64 oracle.

Forward tolerances as for attention over a cache (test_gpu_tree.check). Gradients: P and dS are
rounded to bf16 (2^-8 of each term), scores and lse enter P with es (see there), the result is
rounded once (2^-8), fp32 sums of up to S terms add 2^-16; all relative to the sums of the terms'
magnitudes that the oracle returns (mS bounds |dS| by P (|dO||V| + |dO||O|)).
"""
import numpy as np
import pytest
import torch

import oracle
from sequence_exact_attention_ring_b200 import (KVCache, RingAttnError, binding, cache_read, cache_write, ring_attention,
                                                status, tree_attention, window_attention, window_attention_backward)
from test_gpu_tree import check

pytestmark = pytest.mark.gpu


def inputs(B, Hq, Hkv, S, D, seed, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    q = spread * torch.randn(B, Hq, S, D, generator=g)
    k, v = torch.randn(B, Hkv, S, D, generator=g), torch.randn(B, Hkv, S, D, generator=g) + 0.25
    do = torch.randn(B, Hq, S, D, generator=g)
    k[..., 3::29] *= 3
    return [x.bfloat16().cuda() for x in (q, k, v, do)]


def f64(*xs):
    return [x.double().cpu().numpy() for x in xs]


def forward(q, k, v, W, sinks, what=""):
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    out, lse = window_attention(q, k, v, W, sinks, workspace=ws)
    assert status(ws) == 0, what
    ref = oracle.window_reference(*f64(q, k, v), W, sinks, q.shape[-1] ** -0.5)
    check(out, lse, ref, q.shape[-1], what)
    return out, lse, ref


def backward(q, k, v, do, out, lse, E, W, sinks, what=""):
    D = q.shape[-1]
    got = window_attention_backward(q, k, v, out, lse, do, W, sinks)
    ref = oracle.window_backward_reference(*f64(q, k, v, out, lse, do), W, sinks, D ** -0.5)
    es = D * 2.0 ** -23 * E.max() + 2.0 ** -16
    for name, g, r, m in zip(("dq", "dk", "dv"), got, ref[:3], ref[3:]):
        tol = (2 * 2.0 ** -8 + 3 * es) * m + 2.0 ** -100
        x = g.double().cpu().numpy()
        assert np.isfinite(x).all(), (what, name)
        worst = (np.abs(x - r) / tol).max()
        assert worst <= 1, f"{what} {name}: off by {worst:.2f} of its tolerance"
    return got


SHAPES = [
    # B, Hq, Hkv, S, window, sinks
    (1, 1, 1, 1, 1, 0),
    (1, 2, 1, 2, 1, 1),
    (2, 2, 2, 127, 16, 0),
    (1, 2, 2, 129, 64, 3),
    (1, 4, 2, 300, 1, 0),
    (1, 4, 1, 513, 100, 5),
    (1, 3, 3, 640, 128, 128),
    (1, 6, 2, 1025, 257, 130),
    (2, 2, 1, 777, 5000, 9),
    (1, 2, 2, 1300, 300, 700),
]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_forward_and_gradients(cuda_lib, D, shape):
    B, Hq, Hkv, S, W, sinks = shape
    q, k, v, do = inputs(B, Hq, Hkv, S, D, 7)
    out, lse, ref = forward(q, k, v, W, sinks, str(shape))
    backward(q, k, v, do, out, lse, ref[3], W, sinks, str(shape))


# more query tiles than SMs: the forward's units of two tiles, the backward without divided heads
MANY = [(40, 2, 2, 129, 64, 3), (26, 2, 2, 300, 1, 0), (8, 4, 1, 513, 100, 5), (10, 3, 3, 640, 128, 128),
        (3, 6, 2, 1025, 257, 130)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shape", MANY, ids=lambda s: "-".join(map(str, s)))
def test_many_tiles(cuda_lib, D, shape):
    B, Hq, Hkv, S, W, sinks = shape
    assert B * Hq * ((S + 127) // 128) > 148
    q, k, v, do = inputs(B, Hq, Hkv, S, D, 17)
    out, lse, ref = forward(q, k, v, W, sinks, str(shape))
    backward(q, k, v, do, out, lse, ref[3], W, sinks, str(shape))


@pytest.mark.parametrize("D", [64, 128])
def test_rows_of_a_long_sequence(cuda_lib, D):
    """Rows and keys picked from a long sequence (units in the middle, the cut sink tiles and their parts)."""
    B, Hq, Hkv, S, W, sinks = 1, 4, 2, 20011, 1500, 200
    q, k, v, do = inputs(B, Hq, Hkv, S, D, 8)
    out, lse = window_attention(q, k, v, W, sinks)
    dq, dk, dv = window_attention_backward(q, k, v, out, lse, do, W, sinks)
    Q, K, V, dO, O = (x.double() for x in (q, k, v, do, out))
    scale, r = D ** -0.5, np.random.default_rng(3)
    t = torch.arange(S, device="cuda")
    for h in range(Hq):
        g = h // 2
        for a in [0, 199, 200, 1500, 1700, S - 1] + r.integers(0, S, 20).tolist():
            sel = torch.nonzero((t <= a) & ((t > a - W) | (t < sinks)))[:, 0]
            o, l, A, E = oracle.masked_attention(Q[0, h, a:a + 1].cpu().numpy(), K[0, g, sel].cpu().numpy(),
                                                 V[0, g, sel].cpu().numpy(), np.ones((1, sel.numel()), bool), scale)
            check(out[0, h, a:a + 1], lse[0, h, a:a + 1], (o, l, A, E), D, f"row {a}")
            p = torch.exp(scale * (K[0, g, sel] @ Q[0, h, a]) - lse[0, h, a].double())
            dp = V[0, g, sel] @ dO[0, h, a]
            delta = (dO[0, h, a] * O[0, h, a]).sum()
            want = scale * ((p * (dp - delta)) @ K[0, g, sel])
            mag = scale * ((p * (V[0, g, sel].abs() @ dO[0, h, a].abs() + (dO[0, h, a] * O[0, h, a]).abs().sum())) @ K[0, g, sel].abs())
            assert ((dq[0, h, a].double() - want).abs() <= 2.0 ** -6 * mag).all(), f"dq {a}"
    for g in range(Hkv):
        for u in [0, 127, 128, 199, 200, 255, 256, S - 1] + r.integers(0, S, 12).tolist():
            wk = wv = mk = mv = 0
            for h in (2 * g, 2 * g + 1):
                sel = torch.nonzero((t >= u) & ((t < u + W) | (u < sinks)))[:, 0]
                p = torch.exp(scale * (Q[0, h, sel] @ K[0, g, u]) - lse[0, h, sel].double())
                dp = dO[0, h, sel] @ V[0, g, u]
                delta = (dO[0, h, sel] * O[0, h, sel]).sum(1)
                wv, mv = wv + p @ dO[0, h, sel], mv + p @ dO[0, h, sel].abs()
                wk = wk + scale * ((p * (dp - delta)) @ Q[0, h, sel])
                ms = p * (dO[0, h, sel].abs() @ V[0, g, u].abs() + (dO[0, h, sel] * O[0, h, sel]).abs().sum(1))
                mk = mk + scale * (ms @ Q[0, h, sel].abs())
            assert ((dk[0, g, u].double() - wk).abs() <= 2.0 ** -6 * mk).all(), f"dk {u}"
            assert ((dv[0, g, u].double() - wv).abs() <= 2.0 ** -6 * mv).all(), f"dv {u}"


def test_window_of_everything_is_ring_attention(cuda_lib):
    q, k, v, _ = inputs(1, 4, 2, 1024, 128, 9)
    out, lse = window_attention(q, k, v, 1024)
    o2, l2 = ring_attention(q, k, v, 4, True, "striped")
    assert (out.float() - o2.float()).abs().max().item() <= 2e-2
    assert ((lse - l2).abs() / l2.abs().clamp_min(1)).max().item() <= 1e-3


@pytest.mark.parametrize("D", [64, 128])
def test_large_scores(cuda_lib, D):
    """Scores far apart: the maximum rises from tile to tile and one key wins."""
    q, k, v, do = inputs(1, 2, 1, 700, D, 10, spread=40.0)
    k = (k.float() * torch.linspace(0.1, 3, 700, device="cuda")[:, None]).bfloat16()
    out, lse, ref = forward(q, k, v, 300, 4, "large")
    got = window_attention_backward(q, k, v, out, lse, do, 300, 4)
    assert all(torch.isfinite(x).all() for x in got)


def test_gradients_against_differences(cuda_lib):
    """The loss's change along the gradient, by the forward itself: sum(out * do) at q +- h d."""
    q, k, v, do = inputs(1, 2, 1, 400, 64, 12, spread=0.5)
    W, sinks = 90, 3
    out, lse = window_attention(q, k, v, W, sinks)
    grads = window_attention_backward(q, k, v, out, lse, do, W, sinks)
    g = torch.Generator().manual_seed(1)
    for i in range(3):
        xs = [x.double().cpu().numpy() for x in (q, k, v)]
        d = torch.randn(xs[i].shape, generator=g).double().numpy()
        vals = []
        for sign in (1, -1):
            ys = list(xs)
            ys[i] = xs[i] + sign * 1e-4 * d
            vals.append((oracle.window_reference(*ys, W, sinks, 1 / 8)[0] * do.double().cpu().numpy()).sum())
        want = (vals[0] - vals[1]) / 2e-4
        x = grads[i].double().cpu().numpy()
        # terms of random sign: the rounding errors (2^-7 of each) add in quadrature, 6 sigma
        assert abs((x * d).sum() - want) <= 6 * 2.0 ** -7 * np.sqrt(((x * d) ** 2).sum())


def test_same_bits_twice_and_graphs_with_one_workspace(cuda_lib):
    """Two captured calls that share a workspace, replayed in order, equal the eager calls bit by bit."""
    q, k, v, do = inputs(1, 4, 1, 2000, 64, 13)
    W, sinks = 200, 300
    out, lse = window_attention(q, k, v, W, sinks)
    eager = window_attention_backward(q, k, v, out, lse, do, W, sinks)
    n = binding.ring_attn_window_bwd_workspace_bytes(1, 4, 1, 2000, 64, W, sinks)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    graphs, got = [], []
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                o, l = window_attention(q, k, v, W, sinks, workspace=ws)
                got.append((o, l, *window_attention_backward(q, k, v, o, l, do, W, sinks, workspace=ws)))
            graphs.append(g)
        for _ in range(2):
            for g in graphs:
                g.replay()
    torch.cuda.synchronize()
    for x in got:
        for a, b in zip(x, (out, lse, *eager)):
            assert torch.equal(a, b)
    assert status(ws) == 0


def test_refusals(cuda_lib):
    q, k, v, do = inputs(1, 4, 2, 64, 64, 14)
    for bad in (dict(window=0), dict(sinks=-1)):
        with pytest.raises(ValueError):
            window_attention(q, k, v, **({"window": 8} | bad))
    with pytest.raises(ValueError):
        window_attention(q.float(), k.float(), v.float(), 8)
    with pytest.raises(ValueError):
        window_attention(q.transpose(1, 2), k, v, 8)
    with pytest.raises(ValueError):
        window_attention(q, k, v, 8, out=torch.empty(1, 4, 64, 64, device="cuda"))
    with pytest.raises(RingAttnError) as e:
        window_attention(q, k, v, 8, scale=0.0)
    assert e.value.code == binding.EINVAL
    with pytest.raises(RingAttnError) as e:
        window_attention(q, k, v, 8, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.code == binding.EWORKSPACE
    out, lse = window_attention(q, k, v, 8)
    with pytest.raises(ValueError):
        window_attention_backward(q, k, v, out, lse[..., :-1], do, 8)
    with pytest.raises(RingAttnError) as e:
        window_attention_backward(q, k, v, out, lse, do, 8, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.code == binding.EWORKSPACE


@pytest.mark.parametrize("what", ["window", "gradients", "tree", "read"])
def test_memory_of_a_call_on_another_stream_is_not_reused_early(cuda_lib, what):
    """A call on a given stream still runs when it returns: the scratch and outputs that it allocated must
    not be handed to the current stream's next tensors meanwhile."""
    q, k, v, do = inputs(1, 4, 2, 3000, 128, 19)
    out, lse = window_attention(q, k, v, 200, 4)
    cache = KVCache.allocate(1, 2, 3000, 128, "bf16")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache_write(cache, k, v, zero)
    length = zero + 2991
    calls = dict(window=lambda s: window_attention(q, k, v, 200, 4, stream=s),
                 gradients=lambda s: window_attention_backward(q, k, v, out, lse, do, 200, 4, stream=s),
                 tree=lambda s: tree_attention(q[:, :, :9], cache, length, stream=s),
                 read=lambda s: cache_read(cache, zero, 3000, stream=s))
    want = [t.clone() for t in calls[what](None)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(50_000_000)
    got = calls[what](s)
    kept = []
    sizes = [256, 1 << 12, 1 << 16, 1 << 20] + [t.nbytes for t in got] + [1 << 24, 1 << 25]
    for n in sizes * 3:
        kept.append(torch.full((n,), 0x5a, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert all((t == 0x5a).all() for t in kept)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # and dropped at once, outputs and all
    with torch.cuda.stream(s):
        torch.cuda._sleep(50_000_000)
    del got
    calls[what](s)
    kept = [torch.full((n,), 0x5a, dtype=torch.uint8, device="cuda") for n in sizes * 3]
    torch.cuda.synchronize()
    assert all((t == 0x5a).all() for t in kept)
    # what the current stream has freed is still read there
    old = [torch.full((n,), 0x5a, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)
    copies = [t.clone() for t in old]
    del old
    calls[what](s)
    torch.cuda.synchronize()
    assert all((t == 0x5a).all() for t in copies)
