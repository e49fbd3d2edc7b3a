"""GPU parity of the product with bias, activation and residual.

Every value is held to the oracle's running fp32 bound plus half a step of the
output type."""

import numpy as np
import pytest
import torch

import weight_gated_mlp_b200 as ittt
from oracle import mixer_oracle as mx

from _helpers import host, rel_err

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def half_step(ref, dtype):
    """Half a step of the type relative to the value (bf16 2^-8, fp32 2^-24)."""
    return torch.finfo(DT[dtype]).eps / 2 * np.abs(ref)


def make(M, K, N, dtype, wide=0, seed=0):
    g = torch.Generator().manual_seed(seed)
    X = torch.randn((M, K + wide), generator=g).to(DT[dtype])
    W = (torch.randn((N, K), generator=g) * K ** -0.5).to(DT[dtype])
    b = torch.randn(N, generator=g).to(DT[dtype])
    R = torch.randn((M, N), generator=g).to(DT[dtype])
    return X.cuda()[:, :K], W.cuda(), b.cuda(), R.cuda()


def check(Y, X, W, b, R, act, dtype):
    ref, bound = mx.linear(host(X), host(W), None if b is None else host(b),
                           None if R is None else host(R), act)
    got = host(Y)
    assert ittt.get_last_error() == ittt.OK
    off = np.abs(got - ref) - bound - half_step(ref, dtype) * (1 + 1e-6)
    assert (off <= 0).all(), (np.unravel_index(off.argmax(), off.shape), off.max())


SHAPES = [(1, 8, 1), (1, 2560, 640), (2, 64, 33), (7, 520, 130), (8, 1024, 24), (9, 128, 256),
          (16, 72, 65), (17, 2568, 192), (33, 256, 1000), (64, 520, 264), (65, 192, 40),
          (127, 64, 129), (128, 128, 128), (129, 136, 257), (255, 2048, 192), (257, 640, 512),
          (600, 320, 776), (1100, 256, 1032),
          (1700, 72, 1400), (2500, 136, 1033), (129, 8, 9500),    # CTA pairs
          (200, 2560, 10304)]                                    # pairs, W beyond L2's share


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_product(M, K, N, dtype):
    X, W, b, R = make(M, K, N, dtype)
    check(ittt.linear(X, W), X, W, None, None, "none", dtype)
    check(ittt.linear(X, W, b, R, act="silu"), X, W, b, R, "silu", dtype)


@pytest.mark.parametrize("M,K,N", [(700, 600, 1300), (700, 601, 1297), (1300, 300, 3301), (1100, 255, 2000)])
def test_product_f32_many_tiles(M, K, N):
    """K split over four CTAs, two and one where the tiles alone fill the GPU."""
    X, W, b, R = make(M, K, N, "f32", seed=6)
    check(ittt.linear(X, W, b, R, act="silu"), X, W, b, R, "silu", "f32")


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("M,K,N,dtype", [(1, 256, 72, "bf16"), (5, 256, 71, "bf16"),
                                         (40, 256, 100, "bf16"), (300, 256, 520, "bf16"),
                                         (1700, 64, 1400, "bf16"), (50, 37, 61, "f32"),
                                         (1, 37, 61, "f32"), (1700, 20, 1400, "f32")])
def test_activations(act, M, K, N, dtype):
    X, W, b, R = make(M, K, N, dtype, seed=1)
    check(ittt.linear(X, W, b, act=act), X, W, b, None, act, dtype)
    check(ittt.linear(X, W, None, R, act=act), X, W, None, R, act, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N", [(m, n) for m in (1, 3, 20, 150, 700) for n in (64, 130, 251)] +
                         [(2300, 1290), (5000, 517)])
def test_strides(dtype, M, N):
    """X, residual and Y as column slices of wider matrices; what stands beside
    Y's columns stays; in place on the residual."""
    K = 96
    X, W, b, R = make(M, K, N, dtype, wide=32, seed=2)
    big = torch.full((M, N + 13), 3.0, dtype=DT[dtype], device="cuda")
    wideR = torch.cat([R, R], dim=1)
    Y = ittt.linear(X, W, b, wideR[:, N:], act="gelu", out=big[:, 5:5 + N])
    check(Y, X, W, b, R, "gelu", dtype)
    assert (big[:, :5] == 3.0).all() and (big[:, 5 + N:] == 3.0).all()
    big[:, 5:5 + N] = R
    ittt.linear(X, W, b, big[:, 5:5 + N], out=big[:, 5:5 + N])
    check(big[:, 5:5 + N], X, W, b, R, "none", dtype)
    Y3 = ittt.linear(X.reshape(1, M, K) if X.is_contiguous() else X[None], W)
    assert Y3.shape == (1, M, N)


@pytest.mark.parametrize("M,N", [(1, 200), (4, 200), (24, 200), (200, 200), (2000, 1300)])
def test_nan_and_inf_stay_in_their_rows(M, N):
    X, W, b, R = make(M, 128, N, "bf16", seed=3)
    X[M // 2, 7] = float("nan")
    Y = ittt.linear(X, W, b, R, act="silu")
    bad = torch.isnan(Y).all(dim=1)
    assert bad[M // 2] and bad.sum() == 1 and not torch.isnan(Y[~bad]).any()
    b[3], b[4] = float("-inf"), float("inf")
    X[M // 2, 7] = 1.0
    for act in ("relu", "silu", "gelu", "gelu_tanh"):
        Y = ittt.linear(X, W, b, act=act)
        assert (Y[:, 3] == 0).all() and (Y[:, 4] == float("inf")).all()


def test_the_same_bits_every_time_and_on_another_stream():
    for M, K, N in ((1, 9728, 2560), (64, 9728, 320), (777, 5120, 192)):
        X, W, b, R = make(M, K, N, "bf16", seed=4)
        Y = ittt.linear(X, W, b, R, act="silu")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        Z = ittt.linear(X, W, b, R, act="silu", stream=side)
        with torch.cuda.stream(side):
            V = ittt.linear(X, W, b, R, act="silu")
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(Y, Z) and torch.equal(Y, V)
        assert torch.equal(Y, ittt.linear(X, W, b, R, act="silu"))


def test_two_captured_calls_replayed():
    """Two products in one graph, replayed on new inputs."""
    X, W, b, R = make(24, 4096, 320, "bf16", seed=5)
    X2, W2, _, _ = make(24, 320, 64, "bf16", seed=6)
    ittt.linear(X, W)  # the library's one-time setup is not captured
    ittt.linear(X2, W2)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        h = ittt.linear(X, W, b, R, act="relu")
        y = ittt.linear(h, W2)
    for seed in (7, 8):
        X.copy_(make(24, 4096, 320, "bf16", seed=seed)[0])
        g.replay()
        torch.cuda.synchronize()
        check(h, X, W, b, R, "relu", "bf16")
        check(y, h, W2, None, None, "none", "bf16")


def test_long_rows_pass_32_bit_offsets():
    """Rows further apart than 2^31 elements in all: X and Y are slices of one
    matrix of 2.2e9 elements."""
    M, wide = 2200, 1 << 20
    big = torch.empty((M, wide), dtype=torch.bfloat16, device="cuda")
    X, W, b, _ = make(M, 64, 40, "bf16", seed=9)
    big[:, wide - 128:wide - 64] = X
    Y = ittt.linear(big[:, wide - 128:wide - 64], W, b, out=big[:, 5:45])
    check(Y, X, W, b, None, "none", "bf16")


def test_workloads_down_projection():
    """The plain MLP's down projection at qwen3-4b widths, added to the stream."""
    X, W, b, R = make(512, 9728, 2560, "bf16", seed=10)
    Y = ittt.linear(X, W, None, R)
    ref = X.double() @ W.double().t() + R.double()
    assert rel_err(host(Y), host(ref.float())) <= 2.0 ** -8


def test_buffer_checks():
    X, W, b, R = make(24, 4096, 320, "bf16", seed=11)
    want = ittt.linear(X, W, b, R)
    ittt.set_checks(1)
    try:
        assert torch.equal(ittt.linear(X, W, b, R), want)
    finally:
        ittt.set_checks(0)


def test_refusals():
    X, W, b, R = make(4, 64, 32, "bf16", seed=12)
    with pytest.raises(ValueError, match="dtype"):
        ittt.linear(X, W.float())
    with pytest.raises(ValueError, match="shape"):
        ittt.linear(X, W, b[:-1].contiguous())
    with pytest.raises(ValueError, match="is on"):
        ittt.linear(X, W.cpu())
    with pytest.raises(ValueError, match="column slice"):
        ittt.linear(X[:, ::2], W[:, :32].contiguous())
    with pytest.raises(ittt.IttTError):
        ittt.linear(X[:, 1:], W[:, 1:].contiguous())          # K % 8
    with pytest.raises(ittt.IttTError):
        ittt.linear(torch.zeros(4, 72, dtype=torch.bfloat16, device="cuda")[:, 4:68], W)  # alignment
