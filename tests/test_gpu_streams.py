"""GPU: calls on a stream that is not the current one, with tensors that are dropped while they are still in use.

The caller orders the streams; whose memory may be handed out again, and when, is the library's
part: an output that is read late on the current stream must not become the next call's output on the
other stream, and an input that the call has not read yet must not become a new tensor of the current stream.
"""
import pytest
import torch

from sequence_exact_attention_ring_b200 import (KVCache, cache_read, cache_write, tree_attention, window_attention,
                                                window_attention_backward)

pytestmark = pytest.mark.gpu

SLEEP = 100_000_000  # clocks: some 50 ms


def randn(*shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


def full_cache(fmt, seed, n=320, D=128):
    cache = KVCache.allocate(2, 2, n, D, fmt)
    cache_write(cache, randn(2, 2, n, D, seed=seed), randn(2, 2, n, D, seed=seed + 1),
                torch.zeros(2, dtype=torch.int32, device="cuda"))
    return cache


def calls():
    """name, inputs of a seed (a list of tensors), call(inputs, stream) -> outputs"""
    S, D = 300, 128

    def tree(T):
        def inputs(seed):
            return [randn(2, 8, T, D, seed=seed), torch.tensor([S, 77], dtype=torch.int32, device="cuda"),
                    torch.tensor([[j - 1 for j in range(T)]] * 2, dtype=torch.int32, device="cuda"),
                    torch.tensor([T, max(1, T - 1)], dtype=torch.int32, device="cuda")]

        cache = full_cache("mxfp8", 5)
        return inputs, lambda x, stream: tree_attention(x[0], cache, x[1], x[2], x[3], stream=stream)

    def read():
        cache = full_cache("mxfp4", 6)
        return (lambda seed: [torch.tensor([seed, 2 * seed], dtype=torch.int32, device="cuda"),
                              torch.tensor([200, 100], dtype=torch.int32, device="cuda")],
                lambda x, stream: cache_read(cache, x[0], 256, x[1], stream=stream))

    def write():  # the cache is the output, and new each time
        def call(x, stream):
            cache = KVCache("bf16", *x[4:])
            cache_write(cache, x[0], x[1], x[2], x[3], stream=stream)
            return x[4], x[5]
        return (lambda seed: [randn(2, 2, S, D, seed=seed), randn(2, 2, S, D, seed=seed + 9),
                              torch.tensor([seed, 0], dtype=torch.int32, device="cuda"),
                              torch.tensor([S - 9, 3], dtype=torch.int32, device="cuda"),
                              randn(2, 2, 320, D, seed=1), randn(2, 2, 320, D, seed=2)], call)

    def fwd():
        return (lambda seed: [randn(1, 4, S, D, seed=seed), randn(1, 2, S, D, seed=seed + 1), randn(1, 2, S, D, seed=seed + 2)],
                lambda x, stream: window_attention(*x, 64, 4, stream=stream))

    def bwd():
        def inputs(seed):
            x = fwd()[0](seed)
            return [*x, *window_attention(*x, 64, 4), randn(1, 4, S, D, seed=seed + 3)]
        return inputs, lambda x, stream: window_attention_backward(*x, 64, 4, stream=stream)

    return {"token": tree(1), "tree": tree(30), "read": read(), "write": write(), "window": fwd(), "gradients": bwd()}


@pytest.mark.parametrize("name", ["token", "tree", "read", "window", "gradients"])
def test_outputs_read_late_and_dropped(cuda_lib, name):
    inputs, call = calls()[name]
    a, b = inputs(11), inputs(23)
    want = [t.clone() for t in call(a, None)]
    torch.cuda.synchronize()
    s, cur = torch.cuda.Stream(), torch.cuda.current_stream()
    s.wait_stream(cur)
    outs = call(a, s)
    cur.wait_stream(s)
    torch.cuda._sleep(SLEEP)
    got = [t.clone() for t in outs]  # behind the sleep
    del outs
    for _ in range(3):
        call(b, s)  # s does not wait for the current stream
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g, w)


@pytest.mark.parametrize("name", ["token", "tree", "read", "write", "window", "gradients"])
def test_inputs_dropped_before_they_are_read(cuda_lib, name):
    inputs, call = calls()[name]
    want = [t.clone() for t in call(inputs(11), None)]
    x = inputs(11)
    torch.cuda.synchronize()
    s, cur = torch.cuda.Stream(), torch.cuda.current_stream()
    s.wait_stream(cur)
    with torch.cuda.stream(s):
        torch.cuda._sleep(SLEEP)
    outs = call(x, s)
    like = [t for t in x if not any(t is o for o in outs)]
    shapes = [(t.shape, t.dtype) for t in like]
    del x, like
    # new tensors of the current stream, of the same sizes
    new = [torch.ones(shape, dtype=dtype, device="cuda") for shape, dtype in shapes for _ in range(2)]
    torch.cuda.synchronize()
    for g, w in zip(outs, want):
        assert torch.equal(g, w)
    del new


@pytest.mark.parametrize("name", ["token", "tree", "read", "window", "gradients"])
def test_captured_call_on_a_forked_stream(cuda_lib, name):
    """A call on another stream inside a capture, its streams ordered by the caller; replayed after what it
    returned eagerly was dropped."""
    inputs, call = calls()[name]
    x = inputs(11)
    want = [t.clone() for t in call(x, None)]
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        cur = torch.cuda.current_stream()
        s.wait_stream(cur)
        outs = call(x, s)
        cur.wait_stream(s)
        outs = [t + 0 for t in outs]
    for _ in range(2):
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for g, w in zip(outs, want):
            assert torch.equal(g, w)
