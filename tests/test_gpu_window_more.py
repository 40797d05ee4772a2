"""GPU: gradients of window attention where the scores are large, and against its own forward.

Tolerances as in test_gpu_window.py.
"""
import numpy as np
import pytest
import torch

import oracle
from sequence_exact_attention_ring_b200 import window_attention, window_attention_backward
from test_gpu_window import backward, f64, forward, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
def test_gradients_of_large_scores(cuda_lib, D):
    """Scores far apart, one key of most rows wins: the gradients' values, not their finiteness alone."""
    q, k, v, do = inputs(1, 2, 1, 700, D, 10, spread=40.0)
    k = (k.float() * torch.linspace(0.1, 3, 700, device="cuda")[:, None]).bfloat16()
    out, lse, ref = forward(q, k, v, 300, 4, "large")
    backward(q, k, v, do, out, lse, ref[3], 300, 4, "large")


@pytest.mark.parametrize("D", [64, 128])
def test_gradients_against_the_kernels_own_differences(cuda_lib, D):
    """sum(out * do) at two points on either side of q, k or v, both by window_attention itself, against the
    gradient along the line between them.

    The forward is off by at most 2 2^-8 A per element (A = sum p |v|; the weights' and the result's rounding),
    the former alike in all of a row's dimensions: 2 2^-8 sum_d A |do| a row, independent from row to row and
    in the two points, six sigma. What the line's curvature adds is known exactly: the 64-bit oracle's
    difference at the same points less its gradient along the line. The gradient itself is off by 2^-7 of each
    of its terms, in quadrature, six sigma.
    """
    W, sinks, scale = 90, 3, D ** -0.5
    q, k, v, do = inputs(1, 2, 1, 400, D, 12, spread=0.5)
    out, lse = window_attention(q, k, v, W, sinks)
    grads = window_attention_backward(q, k, v, out, lse, do, W, sinks)
    O, L, A, _ = oracle.window_reference(*f64(q, k, v), W, sinks, scale)
    exact = oracle.window_backward_reference(*f64(q, k, v), O, L, *f64(do), W, sinks, scale)[:3]
    dn = f64(do)[0]
    rows = 2 * 2.0 ** -8 * (A * np.abs(dn)).sum(-1)
    noise = 6 * np.sqrt(2 * (rows ** 2).sum())
    for i, name in enumerate("qkv"):
        g = grads[i].float()
        step = g * (0.3 / g.square().mean().sqrt())
        at = []
        for sign in (1, -1):
            x = [q, k, v]
            x[i] = (x[i].float() + sign * step).bfloat16()
            o, _ = window_attention(*x, W, sinks)
            at.append((x, (f64(o)[0] * dn).sum(), (oracle.window_reference(*f64(*x), W, sinks, scale)[0] * dn).sum()))
        line = f64(at[0][0][i])[0] - f64(at[1][0][i])[0]
        own, true = at[0][1] - at[1][1], at[0][2] - at[1][2]
        curve = true - (exact[i] * line).sum()
        along = f64(grads[i])[0] * line
        tol = noise + 6 * 2.0 ** -7 * np.sqrt((along ** 2).sum())
        assert abs(along.sum()) > 4 * tol, f"d{name}: nothing to see"
        assert abs(along.sum() + curve - own) <= tol, f"d{name}: {along.sum() + curve} against {own}, tolerance {tol}"
