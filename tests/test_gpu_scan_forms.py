"""The forms that a long selective scan is cut into: that the calls below take the
form they are meant for, and that each form keeps the promises of the call."""

import ctypes

import pytest
import torch

import weight_gated_mlp_b200 as ittt

from test_gpu_mixer import check_scan, scan_inputs, scan_ref, within

pytestmark = pytest.mark.gpu


def form(B, T, d, N, G, dtype):
    """("whole", 1, 0): no workspace, the sequences are not cut.  ("runs", n, 0):
    n independent runs, whose states before each and step sums are [n, B, d, N] and
    [n - 1, B, d].  ("chained", 0, c): runs handed from CTA to CTA in blocks of c
    channels, one state a block and a counter word for each and one more."""
    p = ittt.ScanProblem(B=B, T=T, d=d, N=N, G=G, dtype=ittt.BF16 if dtype == "bf16" else ittt.F32)
    n = ctypes.c_size_t(0)
    assert ittt.load_library().ittt_selective_scan_workspace_size(ctypes.byref(p), ctypes.byref(n)) == ittt.OK
    if n.value == 0:
        return "whole", 1, 0
    up = lambda words: -(-4 * words // 256) * 256  # noqa: E731
    runs = [r for r in range(2, -(-T // 256) + 1) if up(r * B * d * N) + up((r - 1) * B * d) == n.value]
    if runs:
        return "runs", runs[0], 0
    for c in (8, 16):
        blocks = B * G * -(-(d // G) // c)
        if up(1 + blocks) + up(blocks * c * (-(-N // 4) * 4)) == n.value:
            return "chained", 0, c
    raise AssertionError(f"a workspace of {n.value} bytes fits no form")


def check_in_place(v, lengths=None):
    """state_out = state_in against a state of its own, bit for bit, many times."""
    out = torch.zeros_like(v["U"])
    Y, s = ittt.selective_scan(**v, lengths=lengths, out=out)
    for _ in range(20):
        state = v["state"].clone()
        Y2, s2 = ittt.selective_scan(**{**v, "state": state}, lengths=lengths, out=torch.zeros_like(out),
                                     state_out=state)
        assert s2 is state and torch.equal(Y2, Y) and torch.equal(state, s)
    assert ittt.get_last_error() == ittt.OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,d,N,G,lengths", [
    (1, 513, 31, 3, 1, None), (1, 2049, 33, 5, 1, None), (1, 4097, 63, 5, 1, None), (1, 4097, 64, 16, 1, None),
    (2, 2561, 24, 3, 1, [2561, 2305]), (5, 1025, 31, 4, 1, [1025, 257, 256, 0, 1]),
    (5, 1025, 40, 16, 1, [513, 1025, 769, 512, 1024]), (1, 1025, 40, 130, 1, None), (4, 4353, 48, 4, 2, None)])
def test_independent_runs_with_the_state_in_place(B, T, d, N, G, lengths, dtype):
    """The last run, one token long here, ends long before the first one."""
    assert form(B, T, d, N, G, dtype)[0] == "runs"
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    check_in_place(scan_inputs(B, T, d, N, G, dtype, seed=21), n)


def test_independent_runs_of_two_passes_with_the_state_in_place():
    assert form(1, 28417, 250, 4, 1, "bf16")[0] == "runs"
    check_in_place(scan_inputs(1, 28417, 250, 4, 1, "bf16", seed=22))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_chained_runs_with_the_state_in_place(dtype):
    assert form(4, 2049, 900, 4, 1, dtype)[0] == "chained"
    check_in_place(scan_inputs(4, 2049, 900, 4, 1, dtype, seed=23),
                   torch.tensor([2049, 1025, 1024, 0], dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_segments_of_independent_runs(dtype):
    """A long prompt in two segments, each cut into runs, its state carried in place,
    against the oracle's whole sequence."""
    B, T, d, N, cut = 1, 2300, 33, 5, 1281
    v = scan_inputs(B, T, d, N, 1, dtype, seed=24)
    for part in (cut, T - cut):
        assert form(B, part, d, N, 1, dtype)[0] == "runs"
    ref, bound, h, hb = scan_ref(v)
    s, ys = v["state"].clone(), []
    for at in (slice(0, cut), slice(cut, T)):
        part = {k: (x[:, at].contiguous() if k in ("U", "delta", "Bm", "Cm", "Z") else x) for k, x in v.items()}
        ys.append(ittt.selective_scan(**{**part, "state": s}, state_out=s)[0])
    within(torch.cat(ys, dim=1), ref, bound, dtype)
    within(s, h, hb, "f32")


@pytest.mark.parametrize("start", ["zeros", "small"])
@pytest.mark.parametrize("B,T,d,N,G,dtype,growth", [
    (1, 28417, 250, 4, 1, "bf16", 19.0), (4, 4353, 48, 4, 2, "f32", 50.0), (1, 12289, 66, 4, 2, "bf16", 50.0)])
def test_growth_past_the_range_over_a_run(B, T, d, N, G, dtype, growth, start):
    """A > 0: every 256 tokens grow by at most e^growth, which fp32 holds, every run by
    more than it holds.  Zeros first (a prompt padded in front), or a small state that
    meets one such run and then ends."""
    kind, runs, _ = form(B, T, d, N, G, dtype)
    run = -(-(-(-T // 256)) // runs)                             # chunks of 256 tokens a run
    assert kind == "runs" and growth < 88 < growth * run * 0.95
    v = scan_inputs(B, T, d, N, G, dtype, seed=26, softplus=False)
    v["delta"].fill_(0.0625)                                     # 16 in 256 tokens
    v["A"] = torch.linspace(0.9, 1.0, d * N, device="cuda").reshape(d, N) * (growth / 16)
    if start == "zeros":
        v["U"][:, :T - 300] = 0
        v["state"] = None
        n = out = None
    else:
        v["U"].zero_()
        v["state"] *= 1e-30
        n = torch.full((B,), 256 * run + 3, dtype=torch.int32, device="cuda")
        out = torch.zeros_like(v["U"])
    Y, s = check_scan(v, dtype, lengths=n, out=out)
    assert torch.isfinite(Y).all() and torch.isfinite(s).all()


@pytest.mark.parametrize("B,T,d,N,G,dtype,want", [
    # the calls of test_gpu_mixer.py that are meant for a form
    (1, 3000, 16, 16, 1, "f32", "runs"), (2, 1500, 24, 8, 1, "bf16", "runs"), (1, 900, 40, 256, 1, "bf16", "runs"),
    (1, 700, 16, 130, 1, "f32", "runs"), (1, 2100, 20, 33, 1, "f32", "runs"), (1, 2500, 24, 16, 1, "bf16", "runs"),
    (1, 28500, 250, 4, 1, "bf16", "runs"), (4, 2100, 900, 4, 1, "bf16", "chained"),
    (4, 2100, 900, 4, 1, "f32", "chained"), (8, 1300, 900, 3, 1, "bf16", "chained")])
def test_the_forms_that_are_tested(B, T, d, N, G, dtype, want):
    assert form(B, T, d, N, G, dtype)[0] == want


@pytest.mark.parametrize("lengths", [None, [1300, 1025, 1024, 0, 1, 256, 257, 700]])
def test_grouped_blocks_of_sixteen_channels(lengths):
    """Grouped projections in the wider channel blocks, which the workspace shows."""
    assert form(8, 1300, 904, 16, 2, "bf16") == ("chained", 0, 16)
    v = scan_inputs(8, 1300, 904, 16, 2, "bf16", seed=25)
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    check_scan(v, "bf16", lengths=n, out=None if lengths is None else torch.full_like(v["U"], 5.0))
