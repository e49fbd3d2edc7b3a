"""The oracle of the operators around the layer against other ways to write them."""

import numpy as np
import pytest

from oracle import ittt_oracle as orc
from oracle import mixer_oracle as mx


def test_causal_conv_is_the_lookahead_conv_backwards_in_time():
    rng = np.random.default_rng(0)
    X, w = rng.standard_normal((1, 23, 5)), rng.standard_normal((5, 4))
    Y, _, last = mx.causal_conv(X, w)
    ref = orc.conv_rows(X[0, ::-1], w[:, ::-1], 23, "sequence")[::-1]
    assert np.allclose(Y[0], ref, atol=1e-13)
    assert np.array_equal(last[0], X[0, -3:])


@pytest.mark.parametrize("cut", [1, 2, 7, 22])
def test_segments_carry_their_state(cut):
    rng = np.random.default_rng(1)
    X, w = rng.standard_normal((2, 23, 5)), rng.standard_normal((5, 4))
    Y, _, last = mx.causal_conv(X, w, act="silu")
    Y1, _, s = mx.causal_conv(X[:, :cut], w, act="silu")
    Y2, _, s = mx.causal_conv(X[:, cut:], w, act="silu", state=s)
    assert np.allclose(np.concatenate([Y1, Y2], 1), Y) and np.array_equal(s, last)


def test_scan_is_the_sum_over_earlier_tokens():
    """h_t = sum_s exp(A sum_(s<r<=t) step_r) step_s u_s B_s."""
    rng = np.random.default_rng(2)
    B, T, d, N = 1, 9, 4, 3
    U, delta = rng.standard_normal((B, T, d)), rng.uniform(0.01, 0.5, (B, T, d))
    A = -rng.uniform(0.5, 4.0, (d, N))
    Bm, Cm = rng.standard_normal((B, T, N)), rng.standard_normal((B, T, N))
    Y, _, h, _ = mx.selective_scan(U, delta, A, Bm, Cm)
    cum = np.cumsum(delta[0], axis=0)
    for t in range(T):
        ref = sum(np.exp(A * (cum[t] - cum[s])[:, None]) * (delta[0, s] * U[0, s])[:, None] * Bm[0, s]
                  for s in range(t + 1))
        assert np.allclose((ref * Cm[0, t]).sum(1), Y[0, t])
    assert np.allclose(ref, h[0])


def test_groups_lengths_and_state():
    rng = np.random.default_rng(3)
    B, T, d, N, G = 3, 8, 6, 2, 3
    U, delta = rng.standard_normal((B, T, d)), rng.standard_normal((B, T, d))
    A = -rng.uniform(0.5, 4.0, (d, N))
    Bm, Cm = rng.standard_normal((B, T, G, N)), rng.standard_normal((B, T, G, N))
    s0, lengths = rng.standard_normal((B, d, N)), [8, 3, 0]
    base = np.full((B, T, d), 7.0)
    Y, _, h, _ = mx.selective_scan(U, delta, A, Bm, Cm, dt_softplus=True, state=s0, lengths=lengths,
                                   base=base)
    assert np.array_equal(h[2], s0[2]) and (Y[2] == 7.0).all() and (Y[1, 3:] == 7.0).all()
    for g in range(G):
        c = slice(2 * g, 2 * g + 2)
        y, _, hg, _ = mx.selective_scan(U[1:2, :3, c], delta[1:2, :3, c], A[c], Bm[1:2, :3, g],
                                        Cm[1:2, :3, g], dt_softplus=True, state=s0[1:2, c])
        assert np.allclose(y[0], Y[1, :3, c]) and np.allclose(hg[0], h[1, c])
