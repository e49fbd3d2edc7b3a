"""The split product where its clusters just do not fit the GPU at once."""

import pytest
import torch

import weight_gated_mlp_b200 as ittt

from test_gpu_linear import check, make

pytestmark = pytest.mark.gpu

# 128-column tiles: 15, 33 and 48 clusters of 8 fit at one, two and three CTAs an SM; 33, 71
# and 104 of 4
TILES = [15, 16, 18, 33, 34, 37, 48, 49, 55, 71, 72, 74, 104, 105, 111]


@pytest.mark.parametrize("tiles", TILES)
@pytest.mark.parametrize("M,K", [(1, 2048), (40, 2048), (100, 1032)])
def test_tiles_around_the_number_of_places(M, K, tiles):
    N = 128 * tiles - 3
    X, W, b, R = make(M, K, N, "bf16", seed=31)
    Y = ittt.linear(X, W, b, R, act="silu")
    check(Y, X, W, b, R, "silu", "bf16")
    assert torch.equal(Y, ittt.linear(X, W, b, R, act="silu"))


@pytest.mark.parametrize("M", [1, 64])
@pytest.mark.parametrize("few,more", [(18, 20), (36, 40)])
def test_fewer_outputs_take_no_longer(M, few, more):
    """Clusters without a place wait for a whole run of the others: 1.4 to 1.7 times the
    time of a call with more outputs, whose clusters all fit.  The best of many short
    loops taken in turn, so that a busy moment does not count."""
    calls = []
    for tiles in (few, more):
        X, W, b, _ = make(M, 9728, 128 * tiles, "bf16", seed=32)
        out = ittt.linear(X, W, b)
        calls.append(lambda X=X, W=W, b=b, out=out: ittt.linear(X, W, b, out=out))
    best = [float("inf")] * 2
    for _ in range(15):
        for i, call in enumerate(calls):
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            start.record()
            for _ in range(40):
                call()
            end.record()
            end.synchronize()
            best[i] = min(best[i], start.elapsed_time(end))
    assert best[0] <= 1.2 * best[1], best
