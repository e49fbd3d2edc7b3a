"""GPU parity of the causal convolution and the selective scan, for prompts and
for single tokens, and of a whole mixer made of them."""

import numpy as np
import pytest
import torch

import weight_gated_mlp_b200 as ittt
from oracle import ittt_oracle as orc
from oracle import mixer_oracle as mx

from _helpers import TOL, host, rel_err
from test_gpu_linear import DT, half_step

pytestmark = pytest.mark.gpu


def within(got, ref, bound, dtype):
    got = host(got) if isinstance(got, torch.Tensor) else got
    off = np.abs(got - ref) - bound - half_step(ref, dtype) * (1 + 1e-6)
    assert (off <= 0).all(), (np.unravel_index(off.argmax(), off.shape), off.max())


def opt(t):
    return None if t is None else host(t)


# ------------------------------------------------------------------- conv

def conv_inputs(B, T, d, k, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g).to(DT[dtype]).cuda()  # noqa: E731
    return r(B, T, d), r(d, k), r(d), r(B, k - 1, d)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,d,k", [
    (1, 1, 8, 4), (3, 1, 40, 4), (1, 2, 33, 4), (2, 3, 64, 4), (2, 5, 100, 4), (1, 33, 256, 4),
    (2, 130, 72, 4), (1, 64, 16, 1), (2, 17, 24, 2), (2, 29, 24, 3), (1, 40, 520, 8), (1, 50, 31, 16),
    (70, 1, 264, 4), (5, 7, 8, 5)])
@pytest.mark.parametrize("act,extra", [("silu", True), ("none", False)])
def test_conv(B, T, d, k, dtype, act, extra):
    X, w, b, s = conv_inputs(B, T, d, k, dtype)
    if not extra:
        b = s = None
    Y, last = ittt.causal_conv(X, w, b, act=act, state=s)
    assert ittt.get_last_error() == ittt.OK
    ref, bound, last_ref = mx.causal_conv(host(X), host(w), opt(b), act, opt(s))
    within(Y, ref, bound, dtype)
    assert np.array_equal(host(last), last_ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,lengths", [(9, 32, [9, 0, 1, 2, 3, 8]), (70, 33, [70, 69, 1, 0, 16, 17]),
                                         (1, 32, [1, 0, 1, 1, 0, 5]), (40, 16, [-3, 100, 40, 0, 4, 31])])
def test_conv_padded_batch(dtype, T, d, lengths):
    """Rows behind a sequence's end hold NaN and are neither read nor written."""
    k, B = 4, len(lengths)
    X, w, b, s = conv_inputs(B, T, d, k, dtype, seed=1)
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    clean = X.clone()
    for i, m in enumerate(lengths):
        X[i, max(m, 0):] = float("nan")
    out = torch.full_like(X, 5.0)
    state = s.clone()
    Y, last = ittt.causal_conv(X, w, b, act="silu", state=state, lengths=n, out=out, state_out=state)
    assert Y is out and last is state
    ref, bound, last_ref = mx.causal_conv(host(clean), host(w), host(b), "silu", host(s), lengths,
                                          np.full(X.shape, 5.0))
    within(Y, ref, bound, dtype)
    assert np.array_equal(host(last), last_ref)
    Y2, _ = ittt.causal_conv(X, w, b, lengths=n)      # rows behind the end: zeros where it allocates
    for i, m in enumerate(lengths):
        assert (Y2[i, max(m, 0):] == 0).all()


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 50), ("f32", 64)])
def test_conv_slices(dtype, d):
    X, w, b, s = conv_inputs(2, 37, 2 * d + 8, 4, dtype, seed=2)
    w, b, s = w[:d].contiguous(), b[:d].contiguous(), s[:, :, :d].contiguous()
    big = torch.full((2, 37, 3 * d), 9.0, dtype=DT[dtype], device="cuda")
    for at in (0, 8, d):
        x = X[:, :, at:at + d]
        Y, last = ittt.causal_conv(x, w, b, act="silu", state=s, out=big[:, :, d:2 * d])
        ref, bound, last_ref = mx.causal_conv(host(x), host(w), host(b), "silu", host(s))
        within(Y, ref, bound, dtype)
        assert np.array_equal(host(last), last_ref)
    assert (big[:, :, :d] == 9.0).all() and (big[:, :, 2 * d:] == 9.0).all()


@pytest.mark.parametrize("B,T,d,part,dtype,lengths", [
    (2, 5003, 4104, 72, "bf16", None), (3, 4001, 2560, 64, "bf16", [4001, 0, 2999]),
    (8, 3001, 1001, 11, "f32", None), (2, 4099, 2052, 108, "f32", [4098, 17])])
def test_conv_more_than_the_gpu_holds(B, T, d, part, dtype, lengths):
    """Many tokens and channels: the bits of calls on a part of the channels, which are cut
    otherwise, and the oracle's values at the first ones."""
    X, w, b, s = conv_inputs(B, T, d, 4, dtype, seed=9)
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    Y, last = ittt.causal_conv(X, w, b, act="silu", state=s, lengths=n)
    for c in (0, (d // part // 2) * part, d - part):
        at = slice(c, c + part)
        few, few_last = ittt.causal_conv(X[:, :, at].contiguous(), w[at].contiguous(), b[at].contiguous(),
                                         act="silu", state=s[:, :, at].contiguous(), lengths=n)
        assert torch.equal(Y[:, :, at], few) and torch.equal(last[:, :, at], few_last)
    ref, bound, last_ref = mx.causal_conv(host(X[:, :, :8]), host(w[:8]), host(b[:8]), "silu", host(s[:, :, :8]),
                                          lengths, np.zeros((B, T, 8)))
    within(Y[:, :, :8], ref, bound, dtype)
    assert np.array_equal(host(last[:, :, :8]), last_ref)


# ------------------------------------------------------------------- scan

def scan_inputs(B, T, d, N, G, dtype, seed=0, softplus=True, lo=1e-3, hi=1e-1):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    t = lambda x: x.to(DT[dtype]).cuda()  # noqa: E731
    step = torch.exp(torch.empty(d).uniform_(np.log(lo), np.log(hi), generator=g))
    v = dict(U=t(r(B, T, d)), Bm=t(r(B, T, G, N)), Cm=t(r(B, T, G, N)), Z=t(r(B, T, d)),
             A=-(torch.arange(1, N + 1) * torch.empty(d, N).uniform_(0.5, 1.5, generator=g)).cuda(),
             D=r(d).cuda(), state=r(B, d, N).cuda(), dt_softplus=softplus)
    if softplus:
        v["delta"], v["dt_bias"] = t(0.5 * r(B, T, d)), (step + torch.log(-torch.expm1(-step))).cuda()
    else:
        v["delta"], v["dt_bias"] = t(step * torch.empty(B, T, d).uniform_(0.5, 2.0, generator=g)), None
    return v


def scan_ref(v, lengths=None, base=None):
    arr = {k: (x if isinstance(x, bool) else opt(x)) for k, x in v.items()}
    return mx.selective_scan(arr["U"], arr["delta"], arr["A"], arr["Bm"], arr["Cm"], arr["D"],
                             arr["Z"], arr["dt_bias"], arr["dt_softplus"], arr["state"], lengths, base)


def check_scan(v, dtype, lengths=None, out=None, **kw):
    base = None if out is None else host(out)
    ref, bound, h, hb = scan_ref(v, None if lengths is None else lengths.tolist(), base)
    Y, s = ittt.selective_scan(**v, lengths=lengths, out=out, **kw)
    assert ittt.get_last_error() == ittt.OK
    within(Y, ref, bound, dtype)
    within(s, h, hb, "f32")
    return Y, s


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,d,N,G", [
    (1, 1, 8, 16, 1), (3, 1, 40, 16, 2), (2, 1, 33, 5, 1), (65, 1, 64, 16, 1), (1, 2, 16, 16, 1),
    (2, 15, 31, 16, 1), (1, 64, 48, 8, 1), (2, 100, 20, 1, 1), (1, 129, 64, 16, 4), (1, 130, 18, 33, 3),
    (2, 257, 16, 64, 1), (1, 20, 24, 256, 1), (1, 300, 7, 4, 7), (3, 40, 100, 3, 2), (1, 515, 40, 16, 1)])
def test_scan(B, T, d, N, G, dtype):
    check_scan(scan_inputs(B, T, d, N, G, dtype), dtype)


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("missing", ["Z", "D", "state", "dt_bias", "all"])
@pytest.mark.parametrize("T", [1, 50])
def test_scan_optional_tensors(softplus, missing, T):
    v = scan_inputs(2, T, 24, 16, 1, "f32", seed=1, softplus=softplus)
    for name in ("Z", "D", "state", "dt_bias"):
        if missing in (name, "all"):
            v[name] = None
    check_scan(v, "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,lengths", [(40, [40, 0, 1, 39, 16, 17]), (300, [0, 300, 128, 129, 256, 2]),
                                       (1, [1, 0, 0, 1, 1, 1]), (20, [-1, 50, 20, 0, 3, 8])])
def test_scan_padded_batch(dtype, T, lengths):
    v = scan_inputs(len(lengths), T, 20, 16, 1, dtype, seed=2)
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    ref, bound, h, hb = scan_ref(v, lengths, np.full((len(lengths), T, 20), 5.0))
    for i, m in enumerate(lengths):
        for name in ("U", "delta", "Bm", "Cm", "Z"):
            v[name][i, max(m, 0):] = float("nan")
    out = torch.full_like(v["U"], 5.0)
    s0 = v["state"].clone()
    Y, s = ittt.selective_scan(**{**v, "state": s0}, lengths=n, out=out, state_out=s0)
    assert Y is out and s is s0
    within(Y, ref, bound, dtype)
    within(s, h, hb, "f32")
    for i, m in enumerate(lengths):
        if m <= 0:
            assert torch.equal(s[i], v["state"][i])
    Y2, _ = ittt.selective_scan(**v, lengths=n)
    for i, m in enumerate(lengths):
        assert (Y2[i, max(m, 0):] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scan_slices(dtype):
    """U and Z halves of one projection, delta, B and C of another."""
    B, T, d, N = 2, 70, 48, 16
    v = scan_inputs(B, T, d, N, 1, dtype, seed=3)
    uz = torch.cat([v["U"], v["Z"]], dim=2)
    rest = torch.cat([v["delta"], v["Bm"][:, :, 0], v["Cm"][:, :, 0]], dim=2)
    big = torch.full((B, T, d + 3), 9.0, dtype=DT[dtype], device="cuda")
    v.update(U=uz[:, :, :d], Z=uz[:, :, d:], delta=rest[:, :, :d], Bm=rest[:, :, d:d + N],
             Cm=rest[:, :, d + N:])
    check_scan(v, dtype, out=big[:, :, 1:1 + d])
    assert (big[:, :, :1] == 9.0).all() and (big[:, :, 1 + d:] == 9.0).all()


@pytest.mark.parametrize("kind", ["slow", "fast", "large", "growing"])
@pytest.mark.parametrize("T", [1, 200])
def test_scan_decay_range(kind, T):
    """Steps that hardly decay, that forget everything, softplus far out on both
    sides, and a positive A."""
    v = scan_inputs(1, T, 16, 16, 1, "f32", seed=4)
    if kind == "slow":
        v["dt_bias"] = torch.full_like(v["dt_bias"], -18.0)
    elif kind == "fast":
        v["A"] = v["A"] * 1e4
    elif kind == "large":
        v["delta"] = v["delta"] * 100.0
    else:
        v["A"], v["dt_bias"] = v["A"].abs() * 0.05, v["dt_bias"]
    check_scan(v, "f32")


def test_scan_nan_stays_in_its_channel_and_later_tokens():
    v = scan_inputs(2, 40, 24, 16, 1, "f32", seed=5)
    v["U"][1, 20, 3] = float("nan")
    Y, s = ittt.selective_scan(**v)
    bad = torch.isnan(Y)
    assert bad[1, 20:, 3].all() and bad.sum() == 20
    assert torch.isnan(s[1, 3]).all() and torch.isnan(s).sum() == 16


@pytest.mark.parametrize("B,T,d,N,dtype", [(1, 3000, 16, 16, "f32"), (2, 1500, 24, 8, "bf16"),
                                           (1, 900, 40, 256, "bf16"), (1, 700, 16, 130, "f32"),
                                           (1, 2100, 20, 33, "f32")])
def test_scan_long_and_narrow(B, T, d, N, dtype):
    """Few channels and many tokens: the scan is split over time."""
    v = scan_inputs(B, T, d, N, 1, dtype, seed=6)
    check_scan(v, dtype)
    n = torch.tensor([T - 700, 0][:B], dtype=torch.int32, device="cuda")
    check_scan(v, dtype, lengths=n, out=torch.zeros_like(v["U"]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths", [None, [2100, 1024, 1025, 0]])
def test_scan_long_and_wide(dtype, lengths):
    """Channel blocks for every CTA and a long prompt: runs handed from CTA to CTA."""
    v = scan_inputs(4, 2100, 900, 4, 1, dtype, seed=10)
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    out = None if lengths is None else torch.full_like(v["U"], 5.0)
    Y, s = check_scan(v, dtype, lengths=n, out=out)
    Y2, s2 = ittt.selective_scan(**v, lengths=n, out=None if out is None else out.clone())
    assert torch.equal(Y, Y2) and torch.equal(s, s2)


@pytest.mark.parametrize("B,T,d,N,G,lengths", [
    (8, 300, 900, 4, 1, None),
    (8, 280, 904, 16, 2, None),                                        # grouped projections
    (8, 300, 909, 5, 1, None),                                         # rows without 16-byte pieces
    (8, 1300, 900, 3, 1, [1300, 1025, 1024, 0, 1, 256, 257, 700]),     # runs handed on
    (1, 28500, 250, 4, 1, None),                                       # independent runs
])
def test_scan_many_channels(B, T, d, N, G, lengths):
    """Enough work for the wider channel blocks (two passes of channels a CTA)."""
    v = scan_inputs(B, T, d, N, G, "bf16", seed=11)
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    out = None if lengths is None else torch.full_like(v["U"], 5.0)
    Y, s = check_scan(v, "bf16", lengths=n, out=out)
    v["Z"] = v["D"] = v["state"] = None
    check_scan(v, "bf16", lengths=n, out=None if out is None else torch.full_like(out, 5.0))


@pytest.mark.parametrize("cuts", [[1], [7, 8], [64, 200], [128]])
def test_segments_match_the_whole(cuts):
    """A prompt in pieces, its states carried in place."""
    B, T, d, N, k = 2, 300, 40, 16, 4
    v = scan_inputs(B, T, d, N, 1, "f32", seed=7)
    X, w, b, _ = conv_inputs(B, T, d, k, "f32", seed=7)
    whole, last = ittt.selective_scan(**v)
    cwhole, clast = ittt.causal_conv(X, w, b, act="silu")
    s, cs = v["state"].clone(), torch.zeros_like(clast)
    ys, cys = [], []
    for lo, hi in zip([0] + cuts, cuts + [T]):
        part = {n: (x[:, lo:hi].contiguous() if n in ("U", "delta", "Bm", "Cm", "Z") else x)
                for n, x in v.items()}
        part["state"] = s
        ys.append(ittt.selective_scan(**part, state_out=s)[0])
        cys.append(ittt.causal_conv(X[:, lo:hi].contiguous(), w, b, act="silu", state=cs, state_out=cs)[0])
    ref, bound, h, hb = scan_ref(v)
    within(torch.cat(ys, 1), ref, bound, "f32")
    within(s, h, hb, "f32")
    assert torch.equal(torch.cat(cys, 1), cwhole) and torch.equal(cs, clast)


def test_streams_graphs_and_repeats():
    v = scan_inputs(1, 2500, 24, 16, 1, "bf16", seed=8)     # split over time: a workspace
    w = scan_inputs(1, 2500, 24, 16, 1, "bf16", seed=9)
    X, cw, cb, cs = conv_inputs(2, 100, 64, 4, "bf16", seed=8)
    Y, s = ittt.selective_scan(**v)
    cY, cl = ittt.causal_conv(X, cw, cb, act="silu", state=cs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    Y1, s1 = ittt.selective_scan(**v, stream=side)
    Y2, s2 = ittt.selective_scan(**w)                        # at the same time
    cY1, cl1 = ittt.causal_conv(X, cw, cb, act="silu", state=cs, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(Y, Y1) and torch.equal(s, s1) and torch.equal(cY, cY1) and torch.equal(cl, cl1)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gY, gs = ittt.selective_scan(**v)
        gY2, gs2 = ittt.selective_scan(**w)
        gc, _ = ittt.causal_conv(X, cw, cb, act="silu", state=cs)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(gY, Y) and torch.equal(gs, s) and torch.equal(gc, cY)
    assert torch.equal(gY2, Y2) and torch.equal(gs2, s2)
    ittt.set_checks(1)
    try:
        assert torch.equal(ittt.selective_scan(**v)[0], Y)
        assert torch.equal(ittt.causal_conv(X, cw, cb, act="silu", state=cs)[0], cY)
    finally:
        ittt.set_checks(0)


def test_refusals():
    v = scan_inputs(1, 4, 16, 16, 1, "bf16")
    X, w, b, s = conv_inputs(1, 4, 16, 4, "bf16")
    with pytest.raises(ValueError, match="state"):
        ittt.causal_conv(X, w, b, state=s.float())
    with pytest.raises(ValueError, match="lengths"):
        ittt.causal_conv(X, w, b, lengths=torch.tensor([3], device="cuda"))
    with pytest.raises(ittt.IttTError):
        ittt.causal_conv(X, w, b, out=X)
    with pytest.raises(ValueError, match="Bm|Cm"):
        ittt.selective_scan(**{**v, "Cm": v["Cm"][..., :8]})
    with pytest.raises(ValueError, match="A has dtype"):
        ittt.selective_scan(**{**v, "A": v["A"].bfloat16()})
    with pytest.raises(ValueError, match="side by side"):
        two = torch.zeros(1, 4, 4, 16, dtype=torch.bfloat16, device="cuda")
        ittt.selective_scan(**{**v, "Bm": two[:, :, ::2], "Cm": two[:, :, 1::2]})
    with pytest.raises(ittt.IttTError):
        ittt.selective_scan(**v, out=v["U"])


# ------------------------------------------------------------- the mixer

class Mixer:
    """A mixer block from the public calls: projection, short convolution,
    selection, scan, projection back onto the residual stream."""

    def __init__(self, d, inner, rank, N, k, dtype, seed=0):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: (torch.randn(s, generator=g) * s[-1] ** -0.5).to(DT[dtype]).cuda()  # noqa: E731
        self.inner, self.rank, self.N, self.k = inner, rank, N, k
        self.w_in, self.w_conv, self.b_conv = r(2 * inner, d), r(inner, k), r(inner)
        self.w_sel, self.w_dt, self.w_out = r(rank + 2 * N, inner), r(inner, rank), r(d, inner)
        self.A = -torch.arange(1, N + 1, dtype=torch.float32).repeat(inner, 1).cuda()
        self.D = torch.ones(inner, device="cuda")
        self.dt_bias = torch.full((inner,), -4.0, device="cuda")

    def states(self, B, dtype):
        return (torch.zeros((B, self.k - 1, self.inner), dtype=DT[dtype], device="cuda"),
                torch.zeros((B, self.inner, self.N), device="cuda"))

    def __call__(self, H, conv_state, state, lengths=None):
        xz = ittt.linear(H, self.w_in)
        x, _ = ittt.causal_conv(xz[:, :, :self.inner], self.w_conv, self.b_conv, act="silu",
                                state=conv_state, state_out=conv_state, lengths=lengths)
        sel = ittt.linear(x, self.w_sel)
        R, N = self.rank, self.N
        delta = ittt.linear(sel[:, :, :R], self.w_dt)
        y, _ = ittt.selective_scan(x, delta, self.A, sel[:, :, R:R + N], sel[:, :, R + N:], D=self.D,
                                   Z=xz[:, :, self.inner:], dt_bias=self.dt_bias, dt_softplus=True,
                                   state=state, state_out=state, lengths=lengths)
        return ittt.linear(y, self.w_out, residual=H)

    def oracle(self, H):
        f = lambda t: host(t)  # noqa: E731
        B, T, d = H.shape
        out = []
        for b in range(B):
            xz = H[b] @ f(self.w_in).T
            x = mx.causal_conv(xz[None, :, :self.inner], f(self.w_conv), f(self.b_conv), "silu")[0]
            sel = x[0] @ f(self.w_sel).T
            R, N = self.rank, self.N
            delta = sel[:, :R] @ f(self.w_dt).T
            y = mx.selective_scan(x, delta[None], f(self.A), sel[None, :, R:R + N], sel[None, :, R + N:],
                                  f(self.D), xz[None, :, self.inner:], f(self.dt_bias), True)[0]
            out.append(y[0] @ f(self.w_out).T + H[b])
        return np.stack(out)


@pytest.mark.parametrize("dtype,tol", [("f32", 1e-5), ("bf16", 1e-2)])
def test_mixer_prompt_then_tokens(dtype, tol):
    """A prompt and then single tokens, against the whole sequence at once.  bf16:
    six roundings of half a step, 2^-8 each at most and 2^-9 rms, on values of
    the output's size in a row: 6 * 2^-9 = 1.2e-2 in the worst alignment; they
    are independent: sqrt(6) * 2^-9 / sqrt(3) = 2.8e-3 is expected."""
    B, T, d = 2, 150, 64
    m = Mixer(d, 128, 8, 16, 4, dtype)
    H = torch.randn((B, T, d), generator=torch.Generator().manual_seed(1)).to(DT[dtype]).cuda()
    conv_state, state = m.states(B, dtype)
    parts = [m(H[:, :137].contiguous(), conv_state, state)]
    for t in range(137, T):
        parts.append(m(H[:, t:t + 1].contiguous(), conv_state, state))
    got = torch.cat(parts, dim=1)
    assert ittt.get_last_error() == ittt.OK
    assert rel_err(host(got), m.oracle(host(H))) <= tol


def test_mixer_token_step_in_a_graph():
    """The token step captured once and replayed: the same bits as the calls."""
    m = Mixer(64, 128, 8, 16, 4, "bf16")
    H = torch.randn((3, 12, 64), generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    a, b = m.states(3, "bf16"), m.states(3, "bf16")
    want = [m(H[:, t:t + 1].contiguous(), *a).clone() for t in range(12)]
    tok = H[:, :1].clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = m(tok, *b)
    for t in range(12):
        tok.copy_(H[:, t:t + 1])
        g.replay()
        assert torch.equal(y, want[t]), t
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_mixer_then_fast_weight_mlp():
    """The block's output through the fast-weight layer, as a model runs them."""
    d, f, T, C, k = 128, 256, 256, 128, 4
    m = Mixer(d, 256, 8, 16, 4, "bf16", seed=3)
    g = torch.Generator().manual_seed(4)
    r = lambda *s, sd=1.0: (torch.randn(s, generator=g) * sd).bfloat16().cuda()  # noqa: E731
    X = r(1, T, d)
    H = m(X, *m.states(1, "bf16"))
    Wg, Wu, Wd = r(f, d, sd=d ** -0.5), r(f, d, sd=d ** -0.5), r(d, f, sd=f ** -0.5)
    K, Wt = r(d, k, sd=0.3), r(d, d, sd=0.1 * d ** -0.5)
    O, W = ittt.fast_mlp_forward(H, X, Wg, Wu, Wd, K, Wt, eta=0.01, C=C)
    assert ittt.get_last_error() == ittt.OK
    inp = {"H": host(H), "X0": host(X), "W_gate": host(Wg), "W_up": host(Wu), "W_down0": host(Wd),
           "conv_kernel": host(K), "W_target": host(Wt)}
    Oref, Wref = orc.forward_sequential(inp, 0.01, C)
    assert rel_err(host(O), Oref) <= TOL["bf16"] and rel_err(host(W), Wref) <= TOL["bf16"]
    # a plain layer of the same widths from the same calls: eta = 0
    Z = ittt.gated_activations(H, Wg, Wu)
    Y = ittt.linear(Z, Wd, residual=H.reshape(T, d))
    O0, _ = ittt.fast_mlp_forward(H, X, Wg, Wu, Wd, K, Wt, eta=0.0, C=C)
    # both round the product once: O0 alone, Y after the sum with H
    diff = np.abs(host(Y) - (host(O0)[0] + host(H)[0]))
    assert (diff <= 2.0 ** -8 * (np.abs(host(O0)[0]) + np.abs(host(Y))) + 1e-5).all()
