"""GPU: calls of the cache and of attention over it that the other files do not make: writes of no rows,
batches of more than a warp of sequences, blocks of zeros.

Tolerances are test_gpu_tree.py's.
"""
import numpy as np
import pytest
import torch

from sequence_exact_attention_ring_b200 import (KVCache, RingAttnError, binding, cache_read, cache_write, status)
from test_gpu_tree import FORMATS, i32, make, random_tree, run

pytestmark = pytest.mark.gpu


def test_write_of_no_rows_clears_the_status(cuda_lib):
    """A step in which no token was accepted: nothing is written, and the status word says so whatever it held."""
    cache = KVCache.allocate(2, 1, 16, 64, "mxfp8")
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        t.fill_(0x5a)
    new = torch.ones(2, 1, 4, 64, device="cuda")
    none, start = new[:, :, :0], i32([0, 14])
    for kw, rows in ((dict(), none), (dict(index=i32([[], []])), new)):
        for dtype in (torch.uint8, torch.float32):
            ws = torch.full((256,), 7, dtype=dtype, device="cuda")
            cache_write(cache, rows, rows, start, workspace=ws, **kw)
            assert status(ws) == 0
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        assert (t == 0x5a).all()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    cache_write(cache, new, new, start, workspace=ws)
    assert status(ws) == binding.EINVAL
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    cache_write(cache, none, none, start, workspace=ws, stream=s)
    assert status(ws, stream=s) == 0
    # its arguments are looked at all the same
    for kw in (dict(start=None), dict(start=i32([0])), dict(count=i32([0]))):
        with pytest.raises(ValueError):
            cache_write(cache, none, none, **(dict(start=start) | kw))
    with pytest.raises(RingAttnError) as e:
        cache_write(cache, none, none, start, workspace=torch.zeros(8, dtype=torch.uint8, device="cuda"))
    assert e.value.code == binding.EWORKSPACE
    with pytest.raises(ValueError):
        cache_write(cache, none, none, start, index=i32([[0], [0]]))
    k, v = cache_read(cache, start, 0)
    assert k.shape == v.shape == (2, 1, 0, 64)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("B", [33, 70])
@pytest.mark.parametrize("T,rep", [(1, 2), (3, 8)])
def test_more_sequences_than_a_warp_has_lanes(cuda_lib, fmt, B, T, rep):
    """Lengths from 0 to some hundreds, empty and refused sequences among them: their shares are found 32
    sequences at a time."""
    r = np.random.default_rng(B)
    lengths = [int(x) for x in r.integers(0, 700, B)]
    lengths[0] = lengths[31] = 0
    lengths[32], lengths[-1] = 699, 1
    q, cache, vals = make(B, rep, 1, 64, T, lengths, fmt, 401)
    counts = [int(x) for x in r.integers(0, T + 1, B)]
    counts[32] = T
    run(q, cache, vals, lengths, random_tree(B, T, 402), counts, what="counts")
    run(q, cache, vals, lengths, what="chain")
    run(q, cache, vals, lengths, window=65, sinks=3, what="window")


def test_more_sequences_than_ctas(cuda_lib):
    """More units than CTAs: most of them are done by one CTA each."""
    B, T = 200, 2
    lengths = [(37 * b) % 90 for b in range(B)]
    for rep in (2, 12):
        q, cache, vals = make(B, 2 * rep, 2, 64, T, lengths, "mxfp8", 403)
        run(q, cache, vals, lengths, what=f"{rep}")


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_rows_of_zeros_among_others(cuda_lib, fmt):
    """Blocks of zeros (scale byte 0) in K and in V, as padded head dimensions leave them, for both forms."""
    n, D = 400, 128
    g = torch.Generator().manual_seed(404)
    for T, rep in ((1, 4), (20, 4)):
        cache = KVCache.allocate(1, 1, n + T, D, fmt)
        k, v = torch.randn(1, 1, n + T, D, generator=g), torch.randn(1, 1, n + T, D, generator=g)
        k[..., 96:], v[..., 96:] = 0.0, 0.0
        cache_write(cache, k.cuda(), v.cuda(), i32([0]))
        vals = [t.double().cpu().numpy() for t in cache_read(cache, i32([0]), cache.capacity, dtype=torch.float32)]
        q = torch.randn(1, rep, T, D, generator=g).bfloat16().cuda()
        out, _ = run(q, cache, vals, [n], what="padded")
        assert not out[..., 96:].any()
