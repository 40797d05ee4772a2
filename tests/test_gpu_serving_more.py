"""GPU: calls of the cache and of attention over it that the other files do not make: writes of no rows."""
import pytest
import torch

from sequence_exact_attention_ring_b200 import (KVCache, RingAttnError, binding, cache_read, cache_write, status)
from test_gpu_tree import i32

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
