"""The operators around the fast-weight MLP layer, as they are measured.

``linear`` (a product with bias, activation and residual), ``causal_conv``
(the short depthwise convolution over the tokens before) and
``selective_scan`` (a diagonal state space recurrence whose step size and
projections depend on the token), for prompts and for single tokens.  Where
``own`` is false, ``run`` computes them from elementary torch operations in 32
bits; where it is true, by the calls of ``weight_gated_mlp_b200``.

Widths are those of the layer's workloads (2560 x 9728) with mixers of twice
the model width (5120), a state of 16 and a step-size rank of 2560 / 16.
"""

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_ES = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------- cases

def _linear(name, M, K, N, dtype="bf16", act="none", bias=False, residual=False, wide=0):
    """``wide``: columns that each row of X has beyond the K of the product (a
    slice of a wider projection)."""
    return {"name": name, "op": "linear", "M": M, "K": K, "N": N, "dtype": dtype, "act": act,
            "bias": bias, "residual": residual, "wide": wide}


def _conv(name, B, T, d, dtype="bf16", k=4, act="silu", bias=True, state=True, ragged=False):
    return {"name": name, "op": "conv", "B": B, "T": T, "d": d, "k": k, "dtype": dtype, "act": act,
            "bias": bias, "state": state, "ragged": ragged}


def _scan(name, B, T, d, N=16, G=1, dtype="bf16", softplus=True, gate=True, skip=True, state=True,
          ragged=False):
    return {"name": name, "op": "scan", "B": B, "T": T, "d": d, "N": N, "G": G, "dtype": dtype,
            "softplus": softplus, "gate": gate, "skip": skip, "state": state, "ragged": ragged}


def listed():
    return [
        # one token of one sequence through a plain MLP's down projection: weight bytes
        _linear("linear one token", 1, 9728, 2560, bias=True, residual=True),
        # 64 sequences' tokens through a mixer's input projection
        _linear("linear 64 tokens", 64, 2560, 10240),
        # a prompt of 777 tokens through the narrow projection to step size, B and C
        _linear("linear narrow, ragged", 777, 5120, 192),
        # the down projection of an 8k prompt, added to the residual stream
        _linear("linear 8k prompt", 8192, 9728, 2560, residual=True),
        # 32-bit weights at odd sizes, X a slice of a wider matrix
        _linear("linear f32 odd", 333, 1000, 1001, dtype="f32", act="gelu", bias=True, wide=24),
        # the short convolution of an 8k prompt
        _conv("conv 8k prompt", 1, 8192, 5120, state=False),
        # a padded batch of odd lengths, one of them empty, in 32 bits, continued from a state
        _conv("conv padded f32", 4, 1001, 1001, dtype="f32", k=3, act="none", ragged=True),
        # one token of 64 sequences
        _conv("conv 64 tokens", 64, 1, 5120),
        # the scan of an 8k prompt, gated
        _scan("scan 8k prompt", 1, 8192, 5120, state=False),
        # few channels, a long document continued from a state: the split over time
        _scan("scan long, narrow", 1, 32768, 512),
        # a padded batch, one sequence empty, 32 bits, grouped projections, a larger state
        _scan("scan padded f32", 3, 1111, 1000, N=32, G=2, dtype="f32", ragged=True, gate=False),
        # one token of 64 sequences: state bytes
        _scan("scan 64 tokens", 64, 1, 5120),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "conv", "scan", "scan"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "linear":
        M, K, N = _log(rng, 1, 8192), 8 * _log(rng, 8, 1216), _log(rng, 16, 10240)
        most = 2.0e11 if dtype == "bf16" else 1.0e10
        while M * K * N > most:
            M, N = max(1, M * 3 // 4), max(16, N * 3 // 4)
        if dtype == "f32":
            K -= rng.randrange(8)
        c = _linear("", M, K, N, dtype, rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]),
                    rng.random() < 0.5, rng.random() < 0.5, rng.choice([0, 0, 8, 64]))
    else:
        B, d = _log(rng, 1, 64), _log(rng, 64, 8192)
        if rng.random() < 0.7:
            d = max(64, d // 8 * 8)
        T = 1 if rng.random() < 0.25 else _log(rng, 2, 16384)
        N = rng.choice([4, 8, 16, 16, 16, 24, 32, 64]) if op == "scan" else 16
        while B * T * d * N > 4.0e8:
            B, T = max(1, B * 3 // 4), max(1, T * 3 // 4)
        ragged = T > 1 and rng.random() < 0.4
        if op == "conv":
            c = _conv("", B, T, d, dtype, rng.randrange(2, 9), rng.choice(["none", "silu"]),
                      rng.random() < 0.5, T == 1 or rng.random() < 0.5, ragged)
        else:
            G = rng.choice([g for g in (1, 1, 2, 4) if d % g == 0])
            c = _scan("", B, T, d, N, G, dtype, rng.random() < 0.7, rng.random() < 0.6,
                      rng.random() < 0.7, T == 1 or rng.random() < 0.5, ragged)
    del c["name"]
    return c


def _lengths(case):
    """Tokens of each sequence of a padded batch: from all of them down to none."""
    B, T = case["B"], case["T"]
    if not case["ragged"]:
        return [T] * B
    return [T - b * T // max(B - 1, 1) for b in range(B)]


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = _DT[case["dtype"]]

    def normal(*shape, std=1.0, dtype=dt):
        return torch.empty(shape, device="cuda").normal_(0.0, std, generator=g).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.empty(shape, device="cuda").uniform_(lo, hi, generator=g)

    st = {"case": dict(case)}
    if case["op"] == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        st["X"] = normal(M, K + case["wide"])[:, :K]
        st["W"] = normal(N, K, std=K ** -0.5)
        st["bias"] = normal(N, std=0.5) if case["bias"] else None
        st["residual"] = normal(M, N) if case["residual"] else None
        return st
    B, T, d = case["B"], case["T"], case["d"]
    n = _lengths(case)
    st["lengths"] = torch.tensor(n, dtype=torch.int32, device="cuda") if case["ragged"] else None
    st["out"] = normal(B, T, d) if case["ragged"] else None
    if case["op"] == "conv":
        k = case["k"]
        st["X"] = normal(B, T, d)
        st["w"] = normal(d, k, std=k ** -0.5)
        st["bias"] = normal(d, std=0.1) if case["bias"] else None
        st["state"] = normal(B, k - 1, d) if case["state"] else None
        return st
    N, G = case["N"], case["G"]
    # the short convolution's outputs after silu; the gate is half of a projection of twice the width
    x = normal(B, T, d, dtype=torch.float32)
    st["U"] = (x / (1.0 + torch.exp(-x))).to(dt)
    st["Z"] = normal(B, T, 2 * d)[:, :, d:] if case["gate"] else None
    # step sizes between 1e-3 and 1e-1, as such layers are initialised
    step = torch.exp(uniform(d, lo=math.log(1e-3), hi=math.log(1e-1)))
    if case["softplus"]:
        st["delta"] = normal(B, T, d, std=0.5)
        st["dt_bias"] = step + torch.log(-torch.expm1(-step))
    else:
        st["delta"] = (step * uniform(B, T, d, lo=0.5, hi=2.0)).to(dt)
        st["dt_bias"] = None
    st["A"] = -(torch.arange(1, N + 1, device="cuda", dtype=torch.float32) * uniform(d, N, lo=0.8, hi=1.2))
    # B and C stand side by side in one projection of the token
    bc = normal(B, T, 2, G, N)
    st["B"], st["C"] = bc[:, :, 0], bc[:, :, 1]
    st["D"] = normal(d, dtype=torch.float32) if case["skip"] else None
    st["state"] = normal(B, d, N, dtype=torch.float32) if case["state"] else None
    return st


# --------------------------------------------------------- the plain forms

def _act(x, name):
    if name == "relu":
        return torch.clamp(x, min=0.0)
    if name == "silu":
        return x / (1.0 + torch.exp(-x))
    if name == "gelu":
        return 0.5 * x * (1.0 + torch.erf(x * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))
    return x


def _plain_linear(st):
    c = st["case"]
    y = st["X"].float() @ st["W"].float().t()
    if st["bias"] is not None:
        y = y + st["bias"].float()
    y = _act(y, c["act"])
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return y.to(_DT[c["dtype"]])


def _within(st):
    """[B, T, 1]: tokens inside their sequences; None where all of them are."""
    if st["lengths"] is None:
        return None
    t = torch.arange(st["case"]["T"], device="cuda")
    return (t[None, :] < st["lengths"][:, None])[:, :, None]


def _plain_conv(st):
    c = st["case"]
    k, T, dt = c["k"], c["T"], _DT[c["dtype"]]
    X = st["X"]
    before = st["state"] if st["state"] is not None else torch.zeros_like(X[:, :1]).expand(-1, k - 1, -1)
    rows = torch.cat([before, X], dim=1)                       # [B, k - 1 + T, d]
    taps = rows.float().unfold(1, k, 1)                        # [B, T, d, k]
    y = (taps * st["w"].float()).sum(-1)
    if st["bias"] is not None:
        y = y + st["bias"].float()
    y = _act(y, c["act"]).to(dt)
    inside = _within(st)
    if inside is None:
        return y, rows[:, T:].contiguous()
    at = st["lengths"].long()[:, None] + torch.arange(k - 1, device="cuda")[None, :]
    last = torch.gather(rows, 1, at[:, :, None].expand(-1, -1, c["d"]))
    return torch.where(inside, y, st["out"]), last


def _plain_scan(st):
    c = st["case"]
    B, T, d, N, G, dt = c["B"], c["T"], c["d"], c["N"], c["G"], _DT[c["dtype"]]
    u = st["U"].float()
    step = st["delta"].float()
    if st["dt_bias"] is not None:
        step = step + st["dt_bias"]
    if c["softplus"]:
        step = torch.clamp(step, min=0.0) + torch.log1p(torch.exp(-step.abs()))
    inside = _within(st)
    if inside is not None:  # a token behind its sequence's end leaves the state as it is
        step = torch.where(inside, step, torch.zeros_like(step))
    Bm = st["B"].float().repeat_interleave(d // G, dim=2)      # [B, T, d, N], or broadcast for one group
    Cm = st["C"].float().repeat_interleave(d // G, dim=2)
    a = torch.exp(step[..., None] * st["A"])
    b = (step * u)[..., None] * Bm
    if st["state"] is not None:
        b[:, 0] += a[:, 0] * st["state"]
    # h_t = a_t h_(t-1) + b_t for all t: spans of 1, 2, 4, ... tokens joined to the span before
    span = 1
    while span < T:
        b = torch.cat([b[:, :span], b[:, span:] + a[:, span:] * b[:, :-span]], dim=1)
        a = torch.cat([a[:, :span], a[:, span:] * a[:, :-span]], dim=1)
        span *= 2
    y = (b * Cm).sum(-1)
    if st["D"] is not None:
        y = y + st["D"] * u
    if st["Z"] is not None:
        y = y * _act(st["Z"].float(), "silu")
    y = y.to(dt)
    return (y if inside is None else torch.where(inside, y, st["out"])), b[:, T - 1].clone()


# -------------------------------------------------------------------- runs

def run(st):
    op = st["case"]["op"]
    if not own:
        return {"linear": _plain_linear, "conv": _plain_conv, "scan": _plain_scan}[op](st)
    import weight_gated_mlp_b200 as ittt

    c = st["case"]
    if op == "linear":
        return ittt.linear(st["X"], st["W"], st["bias"], st["residual"], act=c["act"])
    if op == "conv":
        return ittt.causal_conv(st["X"], st["w"], st["bias"], act=c["act"], state=st["state"],
                                lengths=st["lengths"], out=st["out"])
    return ittt.selective_scan(st["U"], st["delta"], st["A"], st["B"], st["C"], D=st["D"], Z=st["Z"],
                               dt_bias=st["dt_bias"], dt_softplus=c["softplus"], state=st["state"],
                               lengths=st["lengths"], out=st["out"])


def work(case):
    es = _ES[case["dtype"]]
    if case["op"] == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": es * (M * K + N * K + M * N * (1 + case["residual"]) + N * case["bias"]),
                "flops": 2 * M * N * K}
    d, tokens = case["d"], sum(_lengths(case))
    if case["op"] == "conv":
        k = case["k"]
        return {"bytes": es * (2 * tokens * d + k * d + case["B"] * (k - 1) * d * (1 + case["state"])),
                "flops": 2 * k * tokens * d}
    N, G = case["N"], case["G"]
    # each state element and token: step A, exp, step u B, one multiply-add into h, one into y
    return {"bytes": es * tokens * (d * (3 + case["gate"]) + 2 * G * N)
            + 4 * (case["B"] * d * N * (1 + case["state"]) + d * N),
            "flops": 7 * tokens * d * N}


# ------------------------------------------------------- the 64-bit values

def exact(case, seed):
    st = prepare(case, seed)
    f8 = torch.float64
    if case["op"] == "linear":
        s = torch.einsum("mk,nk->mn", st["X"].to(f8), st["W"].to(f8))
        if case["bias"]:
            s += st["bias"].to(f8)
        if case["act"] == "relu":
            s = s * (s > 0)
        elif case["act"] == "silu":
            s = s * torch.sigmoid(s)
        elif case["act"] == "gelu":
            s = s * torch.special.ndtr(s)
        elif case["act"] == "gelu_tanh":
            s = s * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (s + 0.044715 * s ** 3))
        return s + st["residual"].to(f8) if case["residual"] else s
    B, T, d = case["B"], case["T"], case["d"]
    n = _lengths(case)
    base = st["out"].to(f8) if case["ragged"] else torch.empty((B, T, d), device="cuda", dtype=f8)
    if case["op"] == "conv":
        k = case["k"]
        w = st["w"].to(f8)
        last = torch.empty((B, k - 1, d), device="cuda", dtype=f8)
        for b in range(B):
            rows = torch.zeros((k - 1 + n[b], d), device="cuda", dtype=f8)
            if case["state"]:
                rows[:k - 1] = st["state"][b]
            rows[k - 1:] = st["X"][b, :n[b]]
            s = sum(w[:, j] * rows[j:j + n[b]] for j in range(k))
            if case["bias"]:
                s = s + st["bias"].to(f8)
            base[b, :n[b]] = s * torch.sigmoid(s) if case["act"] == "silu" else s
            last[b] = rows[n[b]:]
        return base, last
    N, G = case["N"], case["G"]
    A = st["A"].to(f8)
    h = st["state"].to(f8) if case["state"] else torch.zeros((B, d, N), device="cuda", dtype=f8)
    bias = st["dt_bias"].to(f8) if st["dt_bias"] is not None else 0.0
    live = [sum(1 for x in n if x > t) for t in range(T)]      # sequences by falling length
    for t in range(T):
        m = live[t]
        if m == 0:
            break
        s = st["delta"][:m, t].to(f8) + bias
        if case["softplus"]:
            s = torch.logaddexp(s, torch.zeros_like(s))
        u = st["U"][:m, t].to(f8)
        Bt = st["B"][:m, t].to(f8)[:, :, None, :].expand(m, G, d // G, N).reshape(m, d, N)
        Ct = st["C"][:m, t].to(f8)[:, :, None, :].expand(m, G, d // G, N).reshape(m, d, N)
        h[:m] = torch.exp(s[:, :, None] * A) * h[:m] + (s * u)[:, :, None] * Bt
        y = torch.einsum("bdn,bdn->bd", h[:m], Ct)
        if case["skip"]:
            y = y + st["D"].to(f8) * u
        if case["gate"]:
            z = st["Z"][:m, t].to(f8)
            y = y * z * torch.sigmoid(z)
        base[:m, t] = y
    return base, h
