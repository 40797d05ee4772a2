"""GPU: writing rows into a cache in its format and reading them back, against the fp64 oracle.

Codes, scales and values are exact: scaling by a power of two loses nothing, the element
rounding is to nearest even on both sides, and bf16 holds every stored value.
"""
import numpy as np
import pytest
import torch

import oracle
from sequence_exact_attention_ring_b200 import KVCache, binding, cache_read, cache_write, status

pytestmark = pytest.mark.gpu


def rows(shape, seed, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * torch.exp2(torch.randint(-12, 13, (*shape[:-1], 1), generator=g).float())
    x[..., ::7] *= 30.0
    return x.to(dtype)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def filled(B, Hkv, cap, D, fmt, byte=0x5a):
    c = KVCache.allocate(B, Hkv, cap, D, fmt)
    for t in (c.k, c.v, c.k_scale, c.v_scale):
        if t is not None:
            t.view(torch.uint8).fill_(byte)
    return c


def unpack(codes, fmt):
    c = codes.cpu().numpy().astype(np.int64)
    if fmt == "mxfp4":
        c = np.stack((c & 15, c >> 4), -1).reshape(*c.shape[:-1], 2 * c.shape[-1])
    return c


def same_code(a, b, fmt):
    """Equal codes; the two zeros count as equal."""
    top = 8 if fmt == "mxfp4" else 128
    return (a == b) | ((a % top == 0) & (b % top == 0))


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,Hkv,T", [(1, 1, 1), (3, 2, 37), (2, 3, 200)])
def test_write_and_read_back(cuda_lib, fmt, D, dtype, B, Hkv, T):
    k, v = rows((B, Hkv, T, D), 1, dtype), rows((B, Hkv, T, D), 2, dtype)
    k[0, 0, 0, 32:64] = 0.0
    cache = filled(B, Hkv, T + 50, D, fmt)
    before = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    start = [5 * b for b in range(B)]
    cache_write(cache, k.cuda(), v.cuda(), i32(start))
    ko, vo = cache_read(cache, i32(start), T, dtype=dtype)
    for new, codes, scale, old, old_s, got in ((k, cache.k, cache.k_scale, before[0], before[2], ko),
                                               (v, cache.v, cache.v_scale, before[1], before[3], vo)):
        want_c, want_s, want = oracle.quantise(new.double().numpy(), fmt)
        np.testing.assert_array_equal(got.double().cpu().numpy(), want)
        c, s = unpack(codes, fmt), scale.cpu().numpy()
        for b in range(B):
            assert same_code(c[b, :, start[b]:start[b] + T], want_c[b], fmt).all()
            np.testing.assert_array_equal(s[b, :, start[b]:start[b] + T], want_s[b])
            # no other row is touched
            keep = np.ones(cache.capacity, dtype=bool)
            keep[start[b]:start[b] + T] = False
            np.testing.assert_array_equal(codes[b].cpu().numpy()[:, keep], old[b].cpu().numpy()[:, keep])
            np.testing.assert_array_equal(s[b][:, keep], old_s[b].cpu().numpy()[:, keep])


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "mxfp4"])
def test_counts_strides_index_and_many_rows(cuda_lib, fmt):
    """Rows from a fused projection, a padded batch, accepted nodes picked by index (one of them twice),
    and enough rows for the four-rows-per-thread form."""
    B, Hkv, T, D = 3, 2, 900, 128
    both = torch.randn(B, T, 2, Hkv, D, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    k, v = both[:, :, 0].transpose(1, 2), both[:, :, 1].transpose(1, 2)
    cache = filled(B, Hkv, 20000, D, fmt, 0)
    count, start = [900, 0, 17], [100, 200, 19000]
    cache_write(cache, k, v, i32(start), count=i32(count))
    ko, vo = cache_read(cache, i32(start), T, count=i32(count))
    for got, new in ((ko, k), (vo, v)):
        want = new.double().cpu().numpy()
        want = want if fmt == "bf16" else oracle.quantise(want, fmt)[2]
        for b in range(B):
            np.testing.assert_array_equal(got[b, :, :count[b]].double().cpu().numpy(), want[b][:, :count[b]])
            assert not got[b, :, count[b]:].any()
    idx = [[5, 0, 5, 899], [1, 2, 3, 4], [10, 9, 8, 7]]
    cache_write(cache, k, v, i32([0, 8, 16]), index=i32(idx))
    ko, _ = cache_read(cache, i32([0, 8, 16]), 4, dtype=torch.float32)
    for b in range(B):
        want = k[b][:, idx[b]].double().cpu().numpy()
        want = want if fmt == "bf16" else oracle.quantise(want, fmt)[2]
        np.testing.assert_array_equal(ko[b].double().cpu().numpy(), want)
    big = torch.randn(1, 2, 60000, 64, generator=torch.Generator().manual_seed(4)).cuda()
    wide = filled(1, 2, 60001, 64, fmt, 0)
    cache_write(wide, big, -big, i32([1]))
    ko, vo = cache_read(wide, i32([1]), 60000, dtype=torch.float32)
    assert torch.equal(ko, -vo)
    pick = torch.arange(0, 60000, 997)
    want = big[:, :, pick].cpu()
    want = want.bfloat16().double().numpy() if fmt == "bf16" else oracle.quantise(want.double().numpy(), fmt)[2]
    np.testing.assert_array_equal(ko[:, :, pick].double().cpu().numpy(), want)


def test_special_values(cuda_lib):
    """Zeros, subnormals, the largest finite values, and blocks with a NaN or an infinity."""
    x = torch.zeros(1, 1, 6, 64)
    x[0, 0, 0, 0] = float("nan")
    x[0, 0, 1, 40] = float("inf")
    x[0, 0, 2, :] = 3e38
    x[0, 0, 3, 1] = 1e-45
    x[0, 0, 4, :32] = torch.linspace(-448, 448, 32)
    x[0, 0, 4, 32:] = torch.linspace(-6.01, 6.01, 32)
    for fmt in ("mxfp8", "mxfp4"):
        cache = filled(1, 1, 16, 64, fmt)
        cache_write(cache, x.cuda(), x.cuda(), i32([2]))
        got, _ = cache_read(cache, i32([2]), 6, dtype=torch.float32)
        _, want_s, want = oracle.quantise(x.double().numpy(), fmt)
        np.testing.assert_array_equal(cache.k_scale[0, :, 2:8].cpu().numpy(), want_s[0])
        np.testing.assert_array_equal(got.double().cpu().numpy(), want.astype(np.float32).astype(np.float64))


def test_rows_outside_the_cache_are_skipped_and_reported(cuda_lib):
    cache = filled(2, 1, 16, 64, "mxfp8", 0)
    k = torch.ones(2, 1, 4, 64, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    cache_write(cache, k, k, i32([0, 12]), workspace=ws)
    assert status(ws) == 0
    cache_write(cache, 2 * k, 2 * k, i32([-2, 14]), workspace=ws)
    assert status(ws) == binding.EINVAL
    ko, _ = cache_read(cache, i32([-1, 11]), 6)
    assert ko[0, 0, :, 0].tolist() == [0, 2, 2, 1, 1, 0]
    assert ko[1, 0, :, 0].tolist() == [0, 1, 1, 2, 2, 0]
    cache_write(cache, k, k, i32([0, 0]), index=i32([[0, 4], [-1, 3]]), workspace=ws)
    assert status(ws) == binding.EINVAL


def test_graph_replay_and_side_stream(cuda_lib):
    """The same call captured once and replayed on new data, on a stream that is not the current one."""
    cache = filled(1, 2, 64, 128, "mxfp4", 0)
    new = torch.zeros(1, 2, 3, 128, device="cuda")
    start = i32([7])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        cache_write(cache, new, new, start, stream=s)
        with torch.cuda.graph(graph, stream=s):
            cache_write(cache, new, new, start)
            ko, _ = cache_read(cache, start, 3, dtype=torch.float32)
    for seed in (1, 2):
        x = rows((1, 2, 3, 128), seed)
        new.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(ko.double().cpu().numpy(), oracle.quantise(x.double().numpy(), "mxfp4")[2])
