"""Argument checks of the operators around the layer, without a GPU."""

import ctypes

import pytest
import torch

import weight_gated_mlp_b200 as ittt
from weight_gated_mlp_b200 import _build

FAKE = ctypes.c_void_p(1 << 20)  # never dereferenced: the checks fail first
INV, UNS = ittt.ERR_INVALID_ARG, ittt.ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return ittt.load_library()


def _linear(**kw):
    v = dict(M=4, N=24, K=16, ldx=0, ldr=0, ldy=0, dtype=ittt.BF16, act=0)
    v.update(kw)
    return ittt.LinearProblem(*v.values())


@pytest.mark.parametrize("kw,status", [
    (dict(M=0), INV), (dict(N=-1), INV), (dict(K=0), INV), (dict(dtype=2), INV), (dict(act=5), INV),
    (dict(act=-1), INV), (dict(ldx=8), INV), (dict(ldr=23), INV), (dict(ldy=1), INV),
    (dict(ldx=-16), INV), (dict(K=12), UNS), (dict(ldx=20), UNS), (dict(M=1 << 31), UNS),
    (dict(M=(1 << 31) - 512), UNS), (dict(N=(1 << 31) - 8), UNS),
])
def test_linear_problems(lib, kw, status):
    p = _linear(**kw)
    assert lib.ittt_linear(ctypes.byref(p), FAKE, FAKE, None, None, FAKE, None) == status


def test_linear_pointers(lib):
    p = _linear()
    r = ctypes.byref(p)
    odd = ctypes.c_void_p((1 << 20) + 2)
    assert lib.ittt_linear(r, None, FAKE, None, None, FAKE, None) == INV
    assert lib.ittt_linear(r, FAKE, None, None, None, FAKE, None) == INV
    assert lib.ittt_linear(r, FAKE, FAKE, None, None, None, None) == INV
    y = ctypes.c_void_p(1 << 23)
    assert lib.ittt_linear(r, odd, FAKE, None, None, y, None) == UNS
    assert lib.ittt_linear(r, FAKE, odd, None, None, y, None) == UNS
    # Y may be the residual, not an operand of the product
    assert lib.ittt_linear(r, FAKE, ctypes.c_void_p(1 << 22), None, None, FAKE, None) == INV
    assert lib.ittt_linear(r, ctypes.c_void_p(1 << 22), FAKE, None, None, FAKE, None) == INV
    # in place only with one row stride
    q = _linear(ldr=32)
    assert lib.ittt_linear(ctypes.byref(q), FAKE, FAKE, None, FAKE, FAKE, None) == INV
    assert lib.ittt_linear(None, FAKE, FAKE, None, None, FAKE, None) == INV


def _conv(**kw):
    v = dict(B=2, T=5, d=16, ldx=0, ldy=0, k=4, dtype=ittt.BF16, act=2, reserved=0)
    v.update(kw)
    return ittt.ConvProblem(*v.values())


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), INV), (dict(T=0), INV), (dict(d=-1), INV), (dict(k=0), INV), (dict(k=17), UNS),
    (dict(dtype=9), INV), (dict(act=9), INV), (dict(reserved=1), INV), (dict(ldx=15), INV),
    (dict(ldy=2), INV), (dict(T=1 << 31), UNS), (dict(d=1 << 31), UNS), (dict(B=1 << 16), UNS),
    (dict(B=4, T=1 << 29), UNS),
])
def test_conv_problems(lib, kw, status):
    p = _conv(**kw)
    other = ctypes.c_void_p(1 << 21)
    assert lib.ittt_causal_conv(ctypes.byref(p), FAKE, FAKE, None, None, None, other, None,
                                None) == status


def test_conv_pointers(lib):
    r, other = ctypes.byref(_conv()), ctypes.c_void_p(1 << 21)
    assert lib.ittt_causal_conv(r, None, FAKE, None, None, None, other, None, None) == INV
    assert lib.ittt_causal_conv(r, FAKE, None, None, None, None, other, None, None) == INV
    assert lib.ittt_causal_conv(r, FAKE, FAKE, None, None, None, None, None, None) == INV
    assert lib.ittt_causal_conv(r, FAKE, FAKE, None, None, None, FAKE, None, None) == INV  # Y = X
    assert lib.ittt_causal_conv(r, FAKE, FAKE, None, other, None, other, None, None) == INV
    assert lib.ittt_causal_conv(r, FAKE, FAKE, None, None, None, other, other, None) == INV
    x, w, bias, y = (ctypes.c_void_p(n << 22) for n in range(1, 5))
    for out in (w, bias):
        assert lib.ittt_causal_conv(r, x, w, bias, None, None, out, None, None) == INV
    for state_out in (x, w, bias):
        assert lib.ittt_causal_conv(r, x, w, bias, None, None, y, state_out, None) == INV


def _scan(**kw):
    v = dict(B=2, T=5, d=16, ldu=0, ldt=0, ldb=0, ldc=0, ldz=0, ldy=0, N=8, G=2, dtype=ittt.BF16,
             flags=0)
    v.update(kw)
    return ittt.ScanProblem(*v.values())


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), INV), (dict(T=-3), INV), (dict(d=0), INV), (dict(N=0), INV), (dict(G=0), INV),
    (dict(G=3), INV), (dict(N=257), UNS), (dict(dtype=-1), INV), (dict(flags=2), INV),
    (dict(ldu=15), INV), (dict(ldt=1), INV), (dict(ldb=15), INV), (dict(ldc=8), INV),
    (dict(ldz=-16), INV), (dict(ldy=4), INV), (dict(B=1 << 16, T=1 << 15), UNS),
    (dict(B=(1 << 30) + 1, T=1, d=1, N=1, G=1), UNS),
])
def test_scan_problems(lib, kw, status):
    p, n, other = _scan(**kw), ctypes.c_size_t(0), ctypes.c_void_p(1 << 21)
    assert lib.ittt_selective_scan_workspace_size(ctypes.byref(p), ctypes.byref(n)) == status
    assert lib.ittt_selective_scan(ctypes.byref(p), FAKE, FAKE, FAKE, FAKE, FAKE, None, None, None,
                                   None, None, other, None, None, 0, None) == status


def test_scan_pointers(lib):
    r, y = ctypes.byref(_scan()), ctypes.c_void_p(1 << 21)
    for missing in range(5):
        args = [FAKE] * 5
        args[missing] = None
        assert lib.ittt_selective_scan(r, *args, None, None, None, None, None, y, None, None, 0,
                                       None) == INV
    assert lib.ittt_selective_scan(r, *[FAKE] * 5, None, None, None, None, None, None, None, None, 0,
                                   None) == INV
    assert lib.ittt_selective_scan(r, *[FAKE] * 5, None, None, None, None, None, FAKE, None, None, 0,
                                   None) == INV  # Y = U
    assert lib.ittt_selective_scan_workspace_size(r, None) == INV
    # no output may be another tensor (but state_out state_in)
    u, delta, a, bm, cm, d, bias, z, state, y = (ctypes.c_void_p(n << 22) for n in range(1, 11))
    for out in (u, delta, a, bm, cm, d, bias, z, state):
        assert lib.ittt_selective_scan(r, u, delta, a, bm, cm, d, bias, z, state, None, out, None, None,
                                       0, None) == INV
    for out in (u, delta, a, bm, cm, d, bias, z, y):
        assert lib.ittt_selective_scan(r, u, delta, a, bm, cm, d, bias, z, state, None, y, out, None, 0,
                                       None) == INV


def test_rows_of_a_view():
    """The row stride of dense tensors, column slices, single tokens; others are refused."""
    rows = lambda t: ittt._marshal().row_stride(t, 1)  # noqa: E731
    base = torch.zeros(3, 5, 24)
    assert rows(base) == 0
    assert rows(base[:, :, 8:16]) == 24
    assert rows(base[:1, :, 8:16]) == 24
    assert rows(base[:, :1, :8]) == 5 * 24        # one token: the sequences' distance
    assert rows(base[:1, :1, :8]) in (0, 8)
    for bad in (base[:, ::2], base[:, :4], base[:, :, ::2], base.transpose(0, 1),
                base[:, :1].expand(3, 5, 24), base[:1].expand(3, 5, 24), base[:1, :1].expand(3, 5, 24)):
        with pytest.raises(ValueError, match="column slice"):
            rows(bad)
    assert rows(base[:1, ::2]) == 48              # one sequence, every other row
    four = torch.zeros(3, 5, 4, 6)                # the groups of a token side by side
    row4 = lambda t: ittt._marshal().row_stride(t, 2)  # noqa: E731
    assert row4(four) == 0 and row4(four[:, :, 1:3]) == 24 and row4(four[:, :, 2:3]) == 24
    for bad in (four[:, :, ::2], four[..., :3], four.transpose(2, 3)):
        with pytest.raises(ValueError, match="side by side"):
            row4(bad)


def test_binding_refusals():
    x, w = torch.zeros(4, 16), torch.zeros(24, 16)
    with pytest.raises(ValueError, match="CUDA tensors"):
        ittt.linear(x, w)
    with pytest.raises(ValueError, match="columns"):
        ittt.linear(x, torch.zeros(24, 8))
    with pytest.raises(ValueError, match="CUDA tensors"):
        ittt.causal_conv(torch.zeros(1, 4, 8), torch.zeros(8, 4))
    with pytest.raises(ValueError, match="shape"):
        ittt.causal_conv(torch.zeros(4, 8), torch.zeros(8, 4))
    with pytest.raises(TypeError, match="dtype"):
        ittt.linear(x.half(), w.half())
    with pytest.raises(ValueError, match="CUDA tensors"):
        ittt.selective_scan(torch.zeros(1, 4, 8), torch.zeros(1, 4, 8), torch.zeros(8, 2),
                            torch.zeros(1, 4, 2), torch.zeros(1, 4, 2))
    with pytest.raises(ValueError, match="activation"):
        ittt.linear(x, w, act="swish")
    with pytest.raises(TypeError, match="tensor"):
        ittt.linear([1.0], w)
