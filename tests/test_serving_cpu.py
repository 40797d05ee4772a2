"""CPU: the oracle of the cache, tree and window operators, the window schedules, and refusals.

No compute call is made here: every library call below returns before touching CUDA.
"""
import numpy as np
import pytest
import torch

import oracle
from sequence_exact_attention_ring_b200 import KVCache, binding as B, tree_attention, window_attention
from sequence_exact_attention_ring_b200 import cache_read, cache_write, window_attention_backward


@pytest.fixture(scope="module")
def lib():
    from sequence_exact_attention_ring_b200 import build
    build.build()
    return B.load()


# ------------------------------------------------------------------------- formats
def test_e4m3_table_is_torchs():
    codes = torch.arange(127, dtype=torch.uint8)
    np.testing.assert_array_equal(oracle.element_values("mxfp8"), codes.view(torch.float8_e4m3fn).double().numpy())
    assert oracle.element_values("mxfp4").tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]


@pytest.mark.parametrize("fmt,top,half", [("mxfp8", 448.0, 2.0 ** -4), ("mxfp4", 6.0, 2.0 ** -2)])
def test_quantise_is_nearest_and_never_saturates(fmt, top, half):
    r = np.random.default_rng(1)
    x = r.standard_normal((200, 32)) * np.exp2(r.integers(-30, 30, (200, 1)))
    codes, scale, y = oracle.quantise(x, fmt)
    big = np.abs(x).max(1)
    unit = np.exp2(scale[:, 0].astype(float) - 127)
    assert (big <= top * unit).all() and (big > top * unit / 2).all()
    # half a step, relative to the value or to the smallest normal element
    least = 2.0 ** -6 if fmt == "mxfp8" else 1.0
    assert (np.abs(y - x) <= half * np.maximum(np.abs(x), least * unit[:, None])).all()
    again = oracle.quantise(y, fmt)
    np.testing.assert_array_equal(again[2], y)  # what is stored stays what it is


def test_quantise_borders():
    for fmt, top in (("mxfp8", 448.0), ("mxfp4", 6.0)):
        x = np.zeros((4, 32))
        x[0, 0], x[1, 0], x[2, 0] = top, top * (1 + 2.0 ** -20), -top * 2.0 ** -140
        _, s, y = oracle.quantise(x, fmt)
        assert s[:, 0].tolist() == [127, 128, 0, 0]
        assert y[0, 0] == top and not y[3].any()
    # ties go to the even code: 0.25 -> 0, 0.75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4
    x = np.zeros((1, 32))
    x[0, :8] = [6, 0.25, 0.75, 1.25, -1.75, 2.5, 3.5, 5]
    assert oracle.quantise(x, "mxfp4")[2][0, :8].tolist() == [6, 0, 1, 1, -2, 2, 4, 4]


# --------------------------------------------------------------------------- masks
def test_tree_chain_is_the_causal_window():
    """A chain of drafts behind n tokens is rows n.. of causal attention with the same window and sinks."""
    for n, T, W, sinks in ((0, 5, 0, 0), (7, 4, 3, 0), (7, 4, 3, 2), (20, 6, 100, 1), (3, 9, 2, 5)):
        S = n + T
        want = oracle.window_visible(S, W if W else S, sinks)[n:]
        np.testing.assert_array_equal(oracle.tree_visible(n, None, T, W, sinks), want)
        np.testing.assert_array_equal(oracle.tree_visible(n, list(range(-1, T - 1)), T, W, sinks), want)


def test_tree_siblings_do_not_see_each_other():
    ok = oracle.tree_visible(2, [-1, 0, 0, 1], 4, 0, 0)
    assert ok[:, 2:].astype(int).tolist() == [[1, 0, 0, 0], [1, 1, 0, 0], [1, 0, 1, 0], [1, 1, 0, 1]]
    assert ok[:, :2].all()


def test_window_of_everything_is_causal_attention():
    r = np.random.default_rng(2)
    q, k, v = (r.standard_normal((1, 2, 17, 8)) for _ in range(3))
    O, L, _, _ = oracle.window_reference(q, k, v, 17, 0, 0.3)
    O2, L2 = oracle.attention_reference(torch.tensor(q), torch.tensor(k), torch.tensor(v), True, 0.3)
    np.testing.assert_allclose(O, O2, atol=1e-13)
    np.testing.assert_allclose(L, L2, atol=1e-13)


@pytest.mark.parametrize("S,W,sinks", [(9, 3, 0), (9, 3, 2), (12, 1, 1), (6, 6, 0)])
def test_window_gradients_against_differences(S, W, sinks):
    r = np.random.default_rng(S * W)
    q, k, v = r.standard_normal((1, 4, S, 4)), r.standard_normal((1, 2, S, 4)), r.standard_normal((1, 2, S, 4))
    do = r.standard_normal(q.shape)
    O, L, _, _ = oracle.window_reference(q, k, v, W, sinks, 0.4)
    grads = oracle.window_backward_reference(q, k, v, O, L, do, W, sinks, 0.4)[:3]
    h = 1e-5
    for x, gx in zip((q, k, v), grads):
        for i in r.integers(0, x.size, 12):
            old = x.flat[i]
            vals = []
            for d in (h, -h):
                x.flat[i] = old + d
                vals.append((oracle.window_reference(q, k, v, W, sinks, 0.4)[0] * do).sum())
            x.flat[i] = old
            assert abs((vals[0] - vals[1]) / (2 * h) - gx.flat[i]) <= 1e-7


WINDOWS = [(1, 1, 0), (5, 1, 0), (130, 64, 0), (300, 1, 3), (700, 100, 0), (700, 100, 5), (1030, 257, 130),
           (1030, 2000, 7), (900, 899, 900), (1500, 640, 1200), (2049, 128, 1), (1281, 130, 300)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("S,W,sinks", WINDOWS)
def test_every_visible_pair_is_visited_once(lib, D, S, W, sinks):
    for Hq, Hkv in ((1, 1), (6, 2), (150, 150)):  # (one CTA per query tile, and in units)
        for pass_, times in ((0, 1), (1, Hq // Hkv), (2, 1)):
            counts = np.zeros((S, S), dtype=np.int32)
            n = B.ring_attn_debug_window_visit_counts(Hq, Hkv, S, D, W, sinks, pass_, counts.ctypes.data)
            assert n > 0
            np.testing.assert_array_equal(counts, times * oracle.window_visible(S, W, sinks))


def test_window_visits_are_few(lib):
    """The walks stay near the visible pairs: no more than the tiles that the diagonal and the window cut."""
    S, W = 4096, 1024
    counts = np.zeros((S, S), dtype=np.int32)
    assert B.ring_attn_debug_window_visit_counts(8, 8, S, 128, W, 4, 0, counts.ctypes.data) <= (S // 256) * (W // 128 + 3)
    assert B.ring_attn_debug_window_visit_counts(1, 1, S, 128, W, 4, 0, counts.ctypes.data) <= (S // 128) * (W // 128 + 2)
    assert B.ring_attn_debug_window_visit_counts(1, 1, S, 128, W, 0, 2, counts.ctypes.data) <= (S // 128) * (W // 64 + 2)


# ------------------------------------------------------------------------ refusals
FAKE = 0x10000


def write(**kw):
    a = dict(k=FAKE, v=FAKE, strides=(128,) * 6, dtype=1, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, fmt=1, B=1, Hkv=1, cap=16,
             D=128, T=1, T_src=1, start=FAKE, count=0, index=0, ws=0, wsb=0) | kw
    return B.ring_attn_cache_write(a["k"], a["v"], a["strides"], a["dtype"], a["kc"], a["vc"], a["ks"], a["vs"], a["fmt"],
                                   a["B"], a["Hkv"], a["cap"], a["D"], a["T"], a["T_src"], a["start"], a["count"],
                                   a["index"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("bad,code", [
    (dict(fmt=3), B.EINVAL), (dict(B=0), B.EINVAL), (dict(cap=17), B.EINVAL), (dict(cap=1 << 31), B.EINVAL),
    (dict(D=96), B.EUNSUPPORTED), (dict(kc=0), B.EINVAL), (dict(ks=0), B.EINVAL), (dict(kc=FAKE + 8), B.EALIGN),
    (dict(k=FAKE + 8), B.EALIGN), (dict(strides=(128, 128, 4, 128, 128, 128)), B.EALIGN), (dict(T=0), B.EINVAL),
    (dict(T=2, T_src=1), B.EINVAL), (dict(start=0), B.EINVAL), (dict(start=FAKE + 2), B.EALIGN), (dict(dtype=2), B.EINVAL),
    (dict(T=1 << 30, T_src=1 << 30), B.EINVAL), (dict(ws=FAKE, wsb=8), B.EWORKSPACE),
])
def test_cache_write_refuses(lib, bad, code):
    assert write(**bad) == code


@pytest.mark.parametrize("bad,code", [
    (dict(fmt=-1), B.EINVAL), (dict(T=0), B.EINVAL), (dict(out=0), B.EINVAL), (dict(out=FAKE + 4), B.EALIGN),
    (dict(dtype=9), B.EINVAL), (dict(start=0), B.EINVAL), (dict(vs=0), B.EINVAL),
])
def test_cache_read_refuses(lib, bad, code):
    a = dict(kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, fmt=1, T=1, start=FAKE, out=FAKE, dtype=1) | bad
    assert B.ring_attn_cache_read(a["kc"], a["vc"], a["ks"], a["vs"], a["fmt"], 1, 1, 16, 64, a["T"], a["start"], 0,
                                  a["out"], FAKE, a["dtype"], None) == code


@pytest.mark.parametrize("bad,code", [
    (dict(T=0), B.EINVAL), (dict(T=65), B.EINVAL), (dict(Hq=3), B.EINVAL), (dict(q=0), B.EINVAL), (dict(out=0), B.EINVAL),
    (dict(lengths=0), B.EINVAL), (dict(window=-1), B.EINVAL), (dict(sinks=-1), B.EINVAL), (dict(q=FAKE + 2), B.EALIGN),
    (dict(qs=(64, 64, 7)), B.EALIGN), (dict(parents=FAKE + 1), B.EALIGN), (dict(scale=0.0), B.EINVAL),
    (dict(scale=float("inf")), B.EINVAL), (dict(ws=0), B.EWORKSPACE), (dict(wsb=256), B.EWORKSPACE), (dict(fmt=7), B.EINVAL),
])
def test_tree_refuses(lib, bad, code):
    a = dict(q=FAKE, qs=(64, 64, 64), fmt=2, out=FAKE, Hq=4, T=2, lengths=FAKE, parents=0, window=0, sinks=0, scale=0.1,
             ws=FAKE, wsb=1 << 30) | bad
    assert B.ring_attn_tree(a["q"], a["qs"], FAKE, FAKE, FAKE, FAKE, a["fmt"], a["out"], FAKE, 1, a["Hq"], 2, 16, 64, a["T"],
                            a["lengths"], a["parents"], 0, a["window"], a["sinks"], a["scale"], a["ws"], a["wsb"],
                            None) == code
    assert B.ring_attn_tree_workspace_bytes(2, 1, 4, 2, 16, 64, 2) > 256
    assert B.ring_attn_tree_workspace_bytes(2, 1, 4, 2, 16, 64, 65) == 0


@pytest.mark.parametrize("bad,code", [
    (dict(S=0), B.EINVAL), (dict(window=0), B.EINVAL), (dict(sinks=-1), B.EINVAL), (dict(D=32), B.EUNSUPPORTED),
    (dict(Hq=3), B.EINVAL), (dict(q=0), B.EINVAL), (dict(q=FAKE + 8), B.EALIGN), (dict(ws=0), B.EWORKSPACE),
    (dict(wsb=16), B.EWORKSPACE), (dict(scale=-1.0), B.EINVAL), (dict(S=(1 << 30) + 1), B.EINVAL),
])
def test_window_refuses(lib, bad, code):
    a = dict(q=FAKE, Hq=4, S=100, D=64, window=10, sinks=1, scale=0.1, ws=FAKE, wsb=1 << 40) | bad
    assert B.ring_attn_window_fwd(a["q"], FAKE, FAKE, FAKE, FAKE, 1, a["Hq"], 2, a["S"], a["D"], a["window"], a["sinks"],
                                  a["scale"], a["ws"], a["wsb"], None) == code
    assert B.ring_attn_window_bwd(a["q"], FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1, a["Hq"], 2, a["S"], a["D"],
                                  a["window"], a["sinks"], a["scale"], a["ws"], a["wsb"], None) == code


def test_window_workspace_is_bounded(lib):
    """Partial sums of tiles with sinks stay bounded however many sinks there are."""
    for S, sinks in ((1 << 20, 4), (1 << 20, 1 << 19), (1 << 16, 1 << 15)):
        n = B.ring_attn_window_bwd_workspace_bytes(1, 8, 8, S, 128, 512, sinks)
        stats = 256 + 2 * 4 * 8 * S
        assert stats <= n <= stats + 2000 * 2 * 128 * 128 * 4


def test_python_refusals_without_a_gpu():
    u8, bf = torch.uint8, torch.bfloat16
    rows, scales = torch.zeros(1, 2, 16, 64, dtype=u8), torch.zeros(1, 2, 16, 2, dtype=u8)
    cache = KVCache("mxfp8", rows, rows.clone(), scales, scales.clone())
    assert (cache.B, cache.Hkv, cache.capacity, cache.D) == (1, 2, 16, 64)
    with pytest.raises(ValueError):
        KVCache("fp8", rows, rows)
    with pytest.raises(ValueError):
        KVCache("mxfp8", rows, rows, scales)
    with pytest.raises(ValueError):
        KVCache("mxfp4", rows, rows, scales, scales)   # D is 128 there: four scales a row
    with pytest.raises(ValueError):
        KVCache("bf16", rows, rows)
    with pytest.raises(ValueError):
        KVCache("bf16", rows.to(bf), rows.to(bf), scales, scales)
    assert KVCache.allocate(1, 2, 17, 128, "mxfp4", device="cpu").k.shape == (1, 2, 32, 64)
    start = torch.zeros(1, dtype=torch.int32)
    new = torch.zeros(1, 2, 1, 64, dtype=bf)
    for call in (lambda: cache_write(cache, new, new, start), lambda: cache_read(cache, start, 1),
                 lambda: tree_attention(new, cache, start)):
        with pytest.raises(ValueError):
            call()  # not on a CUDA device
    q = torch.zeros(1, 2, 8, 64, dtype=bf)
    with pytest.raises(ValueError):
        window_attention(q, q, q, 4)
    with pytest.raises(ValueError):
        window_attention_backward(q, q, q, q, torch.zeros(1, 2, 8), q, 4)
