"""Work cases of the recurrent block's trainable operators, for timing and comparison.

Four operators, each reached through the package's public calls when ``own`` is true and
computed from elementary torch operations in 32 bits otherwise:

  recurrence   the gated linear recurrence over long (also packed) sequences, per channel
               h_t = exp(g_t) h_{t-1} + sigmoid(b_t) x_t,  g_t = -exp(A_log) softplus(a_t + dt_bias):
               its forward pass, and forward + backward as a training step makes them
  layer_norm   y = (x - mean) rstd weight + bias, forward, and forward + backward
  conv         the backward pass of the four-tap causal convolution + SiLU
  gated_norm   the backward pass of the gated RMS normalisation

Inputs follow the package's synthetic recipe: normal activations and gates,
A_log ~ U(0, ln 16), dt_bias the inverse softplus of a step size in [1e-3, 1e-1].
"""

import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_EPS_LN = 1e-5
_EPS_RMS = 1e-6

# A drawn case is never larger than these (elements of the activation tensor): the largest
# listed cases of each operator.
_MOST = {"recurrence": 8192 * 6144, "layer_norm": 8192 * 6144, "conv": 8192 * 18432,
         "gated_norm": 8192 * 48 * 128}


# ------------------------------------------------------------------------------- the cases


def listed():
    rec = dict(op="recurrence", B=1, lens="", dtype="bf16", init=True, fused=False, train=True)
    return [
        # one token for each of 64 running requests, 48 heads x 128 channels: a serving step
        dict(rec, name="recurrence_decode_b64", B=64, T=1, C=6144, train=False),
        # a long prompt through a narrow layer (8 heads x 128): few channels, long time axis
        dict(rec, name="recurrence_long_prompt", T=65536, C=1024, init=False, train=False),
        # a training step's layer on one long sequence; x, a, b are slices of one projection
        dict(rec, name="recurrence_train_8k", T=8192, C=6144, fused=True),
        # the same layer on documents of mixed lengths packed into one row, one of them empty
        dict(rec, name="recurrence_train_packed", T=0, C=6144,
             lens="1733,256,3001,0,911,64,1300,517"),
        # fp32 training at odd sizes: a ragged last tile in time and in channels
        dict(rec, name="recurrence_train_f32_odd", B=2, T=777, C=1160, dtype="f32"),
        # the block's input norm in a serving step
        dict(op="layer_norm", name="layer_norm_decode_b64", rows=64, d=6144, dtype="bf16",
             bias=True, train=False),
        # the block's input norm in a training step
        dict(op="layer_norm", name="layer_norm_train_8k", rows=8192, d=6144, dtype="bf16",
             bias=True, train=True),
        # fp32, odd numbers of rows and of columns, no bias
        dict(op="layer_norm", name="layer_norm_train_f32_odd", rows=1001, d=1160, dtype="f32",
             bias=False, train=True),
        # the q | k | v channels of 48 heads over one long training sequence
        dict(op="conv", name="conv_bwd_8k", B=1, T=8192, C=18432, bias=False, state=False),
        # a resumed batch: a carried state, a bias, a ragged last channel tile
        dict(op="conv", name="conv_bwd_odd", B=3, T=777, C=1160, bias=True, state=True),
        # every (token, head) of a long training sequence
        dict(op="gated_norm", name="gated_norm_bwd_8k", rows=8192 * 48, d=128, zdtype="bf16"),
        # a small layer, narrow heads, fp32 gate
        dict(op="gated_norm", name="gated_norm_bwd_f32_odd", rows=3001, d=64, zdtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["recurrence", "recurrence", "layer_norm", "conv", "gated_norm"])
    most = _MOST[op]
    if op == "layer_norm":
        d = 8 * _log_int(rng, 8, 1024)
        return dict(op=op, rows=_log_int(rng, 1, min(65536, most // d)), d=d,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), bias=rng.random() < 0.7,
                    train=rng.random() < 0.7)
    if op == "gated_norm":
        d = rng.choice([32, 64, 128])
        return dict(op=op, rows=_log_int(rng, 1, min(400000, most // d)), d=d,
                    zdtype=rng.choice(["bf16", "bf16", "f32"]))
    C = 8 * _log_int(rng, 8, 2304 if op == "conv" else 768)
    if op == "conv":
        B = rng.choice([1, 1, 2, 3, 8])
        return dict(op=op, B=B, T=_log_int(rng, 1, min(16384, most // (B * C))), C=C,
                    bias=rng.random() < 0.5, state=rng.random() < 0.5)
    case = dict(op=op, C=C, dtype=rng.choice(["bf16", "bf16", "f32"]),
                init=rng.random() < 0.5, fused=rng.random() < 0.5)
    kind = rng.choice(["decode", "dense", "dense", "packed"])
    if kind == "decode":
        B = _log_int(rng, 1, 256)
        return dict(case, B=B, T=rng.choice([1, 1, 1, 2, 4]), lens="", train=False)
    if kind == "packed":
        n = rng.randint(1, 12)
        top = max(16, min(4096, most // (2 * C * n)))
        lens = [0 if rng.random() < 0.08 else _log_int(rng, 1, top) for _ in range(n)]
        lens[rng.randrange(n)] = top
        return dict(case, B=1, T=0, lens=",".join(map(str, lens)), train=rng.random() < 0.7)
    B = rng.choice([1, 1, 2, 4])
    # fp32 inputs weigh twice as much
    return dict(case, B=B, T=_log_int(rng, 8, min(65536, most // (2 * B * C))), lens="",
                train=rng.random() < 0.7)


# ------------------------------------------------------------------------------ the inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(shape, device="cuda", generator=g) * std).to(dtype)

    def uniform(lo, hi, *shape):
        return torch.rand(shape, device="cuda", generator=g) * (hi - lo) + lo

    s = dict(case=case)
    op = case["op"]
    if op == "recurrence":
        dt, C = _DT[case["dtype"]], case["C"]
        lens = [int(n) for n in case["lens"].split(",")] if case["lens"] else None
        B, T = (1, sum(lens)) if lens else (case["B"], case["T"])
        nseq = len(lens) if lens else B
        if case["fused"]:  # slices of one projection, as a fused input layer leaves them
            s["x"], s["a"], s["b"] = normal(B, T, 3 * C, dtype=dt).split(C, dim=2)
        else:
            s["x"], s["a"], s["b"] = (normal(B, T, C, dtype=dt) for _ in range(3))
        s["A_log"] = uniform(0.0, math.log(16.0), C)
        step = torch.exp(uniform(math.log(1e-3), math.log(1e-1), C).double())
        s["dt_bias"] = torch.log(torch.expm1(step)).float()
        s["init"] = normal(nseq, C) if case["init"] else None
        s["cu"] = None
        if lens:
            s["cu"] = torch.tensor([0] + list(np.cumsum(lens)), device="cuda", dtype=torch.int32)
        if case["train"]:
            s["dout"], s["dfinal"] = normal(B, T, C), normal(nseq, C)
        else:  # a serving loop keeps its output buffers
            s["out"] = torch.empty(B, T, C, device="cuda")
            s["final"] = torch.empty(nseq, C, device="cuda")
    elif op == "layer_norm":
        dt, rows, d = _DT[case["dtype"]], case["rows"], case["d"]
        # a residual stream: channels of different scale around a common offset
        s["x"] = (normal(rows, d) * uniform(0.5, 2.0, d) + normal(d, std=0.3)).to(dt)
        s["w"] = uniform(0.5, 1.5, d)
        s["bias"] = normal(d, std=0.1) if case["bias"] else None
        s["dy"] = normal(rows, d, dtype=dt) if case["train"] else None
    elif op == "conv":
        B, T, C = case["B"], case["T"], case["C"]
        s["x"] = normal(B, T, C, dtype=torch.bfloat16)
        s["w"] = normal(C, 4, std=0.5)
        s["bias"] = normal(C, std=0.1) if case["bias"] else None
        s["state"] = normal(B, C, 3) if case["state"] else None
        s["dy"] = normal(B, T, C, dtype=torch.bfloat16)
        s["dstate"] = normal(B, C, 3) if case["state"] else None
    else:
        rows, d = case["rows"], case["d"]
        s["o"] = normal(rows, d)
        s["z"] = normal(rows, d, dtype=_DT[case["zdtype"]])
        s["w"] = uniform(0.5, 1.5, d)
        s["dy"] = normal(rows, d)
    return s


# -------------------------------------------------------------------- one pass of each kind


def run(s):
    if own:
        return _run_own(s)
    return {"recurrence": _recurrence, "layer_norm": _layer_norm, "conv": _conv,
            "gated_norm": _gated_norm}[s["case"]["op"]](s)


def _run_own(s):
    import gated_delta_rule_145_b200 as gdr

    case = s["case"]
    if case["op"] == "recurrence":
        x, a, b = s["x"], s["a"], s["b"]
        if not case["train"]:
            B, T, C = x.shape
            call = (gdr.gdr_linear_recurrence if case["dtype"] == "bf16" else
                    gdr.gdr_linear_recurrence_f32)
            nseq = B if s["cu"] is None else s["cu"].numel() - 1
            call(x, a, b, s["A_log"], s["dt_bias"], s["init"], s["out"], s["final"], s["cu"], nseq,
                 T, C, x.stride(1))
            return s["out"], s["final"]
        out, final = gdr.linear_recurrence(x, a, b, s["A_log"], s["dt_bias"], s["init"], s["cu"])
        grads = gdr.linear_recurrence_backward(x, a, b, s["A_log"], s["dt_bias"], out, s["dout"],
                                               s["dfinal"], s["init"], s["cu"])
        return (out, final) + grads
    if case["op"] == "layer_norm":
        y, mean, rstd = gdr.layer_norm(s["x"], s["w"], s["bias"], _EPS_LN)
        if not case["train"]:
            return y, mean, rstd
        dx, dw, db = gdr.layer_norm_backward(s["x"], s["w"], mean, rstd, s["dy"])
        return y, mean, rstd, dx, dw, db
    if case["op"] == "conv":
        return gdr.short_conv_silu_backward(s["x"], s["w"], s["dy"], s["bias"], s["state"],
                                            s["dstate"])
    return gdr.gated_rmsnorm_backward(s["o"], s["z"], s["w"], s["dy"], _EPS_RMS)


# ------------------------------------------------------------------------- the plain forms


def _scan(decay, u):
    """h_t = decay_t h_{t-1} + u_t along dim 1 from zero: pairs at distances 1, 2, 4, ... are
    composed, which takes log2(T) rounds (a running product of decays would underflow)."""
    step = 1
    while step < u.shape[1]:
        head_u, head_d = u[:, :step], decay[:, :step]
        u = torch.cat([head_u, u[:, step:] + decay[:, step:] * u[:, :-step]], 1)
        decay = torch.cat([head_d, decay[:, step:] * decay[:, :-step]], 1)
        step *= 2
    return u


def _bounds(s, B, T, device):
    """(batch row, first token, last token) of every sequence and which sequences have tokens."""
    if s["cu"] is None:
        row = torch.arange(B, device=device)
        first = torch.zeros(B, dtype=torch.long, device=device)
        last = first + T - 1
    else:
        cu = s["cu"].long()
        first, last = cu[:-1], cu[1:] - 1
        row = torch.zeros_like(first)
    return row, first, last, last >= first


def _recurrence(s):
    x, a, b = s["x"].float(), s["a"].float(), s["b"].float()
    B, T, C = x.shape
    A = torch.exp(s["A_log"])
    z = a + s["dt_bias"]
    p = torch.clamp(z, min=0) + torch.log1p(torch.exp(-torch.abs(z)))  # softplus
    decay = torch.exp(-A * p)
    gate = 1 / (1 + torch.exp(-b))
    row, first, last, some = _bounds(s, B, T, x.device)
    init = s["init"] if s["init"] is not None else x.new_zeros(len(row), C)
    # a sequence's first token takes its initial state through its own input
    at = row[some], first[some]
    u = gate * x
    u[at] += decay[at] * init[some]
    broken = decay.clone()
    broken[at] = 0
    h = _scan(broken, u)
    final = init.clone()
    final[some] = h[row[some], last[some]]
    if not s["case"]["train"]:
        return h, final
    prev = torch.cat([h.new_zeros(B, 1, C), h[:, :-1]], 1)
    prev[at] = init[some]
    # the adjoint runs the other way: D_t = dout_t + decay_{t+1} D_{t+1}
    d = s["dout"].clone()
    d[row[some], last[some]] += s["dfinal"][some]
    after = torch.cat([broken[:, 1:], h.new_zeros(B, 1, C)], 1)
    D = _scan(after.flip(1), d.flip(1)).flip(1)
    dg = D * prev * decay
    da = dg * -A / (1 + torch.exp(-z))
    dinit = s["dfinal"].clone()
    dinit[some] = (D * decay)[at]
    dt = _DT[s["case"]["dtype"]]
    return (h, final, (D * gate).to(dt), da.to(dt), (D * x * gate * (1 - gate)).to(dt),
            (dg * -A * p).sum((0, 1)), da.sum((0, 1)), dinit)


def _layer_norm(s):
    x, dt = s["x"].float(), _DT[s["case"]["dtype"]]
    mean = x.sum(1, keepdim=True) / x.shape[1]
    xc = x - mean
    rstd = 1 / torch.sqrt((xc * xc).sum(1, keepdim=True) / x.shape[1] + _EPS_LN)
    xh = xc * rstd
    y = xh * s["w"]
    if s["bias"] is not None:
        y = y + s["bias"]
    if not s["case"]["train"]:
        return y.to(dt), mean[:, 0], rstd[:, 0]
    dy = s["dy"].float()
    dyw = dy * s["w"]
    m1 = dyw.sum(1, keepdim=True) / x.shape[1]
    m2 = (dyw * xh).sum(1, keepdim=True) / x.shape[1]
    dx = rstd * (dyw - m1 - xh * m2)
    return y.to(dt), mean[:, 0], rstd[:, 0], dx.to(dt), (dy * xh).sum(0), dy.sum(0)


def _conv(s):
    x, dy, w = s["x"].float(), s["dy"].float(), s["w"]
    B, T, C = x.shape
    before = s["state"].transpose(1, 2) if s["state"] is not None else x.new_zeros(B, 3, C)
    hist = torch.cat([before, x], 1)
    pre = (w[:, 0] * hist[:, :T] + w[:, 1] * hist[:, 1:T + 1] + w[:, 2] * hist[:, 2:T + 2] +
           w[:, 3] * x)
    if s["bias"] is not None:
        pre = pre + s["bias"]
    sig = 1 / (1 + torch.exp(-pre))
    ds = dy * sig * (1 + pre * (1 - sig))
    dw = torch.stack([(ds * hist[:, :T]).sum((0, 1)), (ds * hist[:, 1:T + 1]).sum((0, 1)),
                      (ds * hist[:, 2:T + 2]).sum((0, 1)), (ds * x).sum((0, 1))], 1)
    dhist = torch.zeros_like(hist)
    dhist[:, :T] += w[:, 0] * ds
    dhist[:, 1:T + 1] += w[:, 1] * ds
    dhist[:, 2:T + 2] += w[:, 2] * ds
    dhist[:, 3:] += w[:, 3] * ds
    if s["dstate"] is not None:
        dhist[:, T:] += s["dstate"].transpose(1, 2)
    return (dhist[:, 3:].bfloat16(), dw, ds.sum((0, 1)),
            dhist[:, :3].transpose(1, 2).contiguous())


def _gated_norm(s):
    o, z, w, dy = s["o"], s["z"].float(), s["w"], s["dy"]
    r = 1 / torch.sqrt((o * o).sum(1, keepdim=True) / o.shape[1] + _EPS_RMS)
    sig = 1 / (1 + torch.exp(-z))
    gate = z * sig
    q = dy * w * gate
    do = r * q - o * (r * r * r) * ((q * o).sum(1, keepdim=True) / o.shape[1])
    dz = dy * o * r * w * sig * (1 + z * (1 - sig))
    return do, dz.to(s["z"].dtype), (dy * o * r * gate).sum(0)


# ---------------------------------------------------------- the definition, step by step


def exact(case, seed):
    s = prepare(case, seed)
    return {"recurrence": _exact_recurrence, "layer_norm": _exact_layer_norm,
            "conv": _exact_conv, "gated_norm": _exact_gated_norm}[case["op"]](s)


def _exact_recurrence(s):
    """One token after the other, and the chain rule one token after the other backwards."""
    x, a, b = s["x"].double(), s["a"].double(), s["b"].double()
    B, T, C = x.shape
    z = a + s["dt_bias"].double()
    p = torch.logaddexp(z, torch.zeros_like(z))
    g = -torch.exp(s["A_log"].double()) * p
    lam, gate = torch.exp(g), torch.sigmoid(b)
    cu = None if s["cu"] is None else s["cu"].tolist()
    # spans of tokens that share their bounds: all rows of a dense batch, or one sequence
    if cu is None:
        spans = [(slice(0, B), 0, T)]
    else:
        spans = [(slice(i, i + 1), lo, hi) for i, (lo, hi) in enumerate(zip(cu, cu[1:]))]
    nseq = B if cu is None else len(cu) - 1
    init = s["init"].double() if s["init"] is not None else x.new_zeros(nseq, C)
    h, u = torch.empty_like(x), gate * x
    final = init.clone()
    for sq, lo, hi in spans:
        state = init[sq].clone()
        for t in range(lo, hi):
            state = torch.addcmul(u[:, t], lam[:, t], state)
            h[:, t] = state
        final[sq] = state
    if not s["case"]["train"]:
        return h, final
    dx, da, db = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    dA_log, dinit = x.new_zeros(C), s["dfinal"].double()
    dout = s["dout"]
    for sq, lo, hi in spans:
        grad = dinit[sq].clone()
        D, prev = x.new_empty(B, hi - lo, C), x.new_empty(B, hi - lo, C)
        for t in range(hi - 1, lo - 1, -1):
            grad = grad + dout[:, t]
            D[:, t - lo] = grad
            grad = grad * lam[:, t]
        dinit[sq] = grad
        if hi == lo:
            continue
        prev[:, 0] = init[sq]
        prev[:, 1:] = h[:, lo:hi - 1]
        sl = slice(lo, hi)
        dx[:, sl] = D * gate[:, sl]
        db[:, sl] = D * x[:, sl] * torch.sigmoid(b[:, sl]) * torch.sigmoid(-b[:, sl])
        dgl = D * prev * lam[:, sl]
        da[:, sl] = dgl * -torch.exp(s["A_log"].double()) * torch.sigmoid(z[:, sl])
        dA_log += (dgl * g[:, sl]).sum((0, 1))
    return h, final, dx, da, db, dA_log, da.sum((0, 1)), dinit


def _leaf(t):
    return t.double().requires_grad_()


def _exact_layer_norm(s):
    x, w = _leaf(s["x"]), _leaf(s["w"])
    bias = _leaf(s["bias"] if s["bias"] is not None else torch.zeros_like(s["w"]))
    mean = x.mean(1)
    rstd = (x.var(1, unbiased=False) + _EPS_LN).rsqrt()
    y = (x - mean[:, None]) * rstd[:, None] * w + bias
    out = [y.detach(), mean.detach(), rstd.detach()]
    if s["case"]["train"]:
        out += torch.autograd.grad(y, (x, w, bias), s["dy"].double())
    return out


def _exact_conv(s):
    B, T, C = s["x"].shape
    x, w = _leaf(s["x"]), _leaf(s["w"])
    bias = _leaf(s["bias"] if s["bias"] is not None else s["w"].new_zeros(C))
    state = _leaf(s["state"] if s["state"] is not None else s["w"].new_zeros(B, C, 3))
    hist = torch.cat([state.transpose(1, 2), x], 1)
    pre = sum(hist[:, i:i + T] * w[:, i] for i in range(4)) + bias
    total = (pre * torch.sigmoid(pre) * s["dy"].double()).sum()
    if s["dstate"] is not None:
        total = total + (hist[:, T:].transpose(1, 2) * s["dstate"].double()).sum()
    return list(torch.autograd.grad(total, (x, w, bias, state)))


def _exact_gated_norm(s):
    o, z, w = _leaf(s["o"]), _leaf(s["z"]), _leaf(s["w"])
    y = o * (o.square().mean(1, keepdim=True) + _EPS_RMS).rsqrt() * w * z * torch.sigmoid(z)
    return list(torch.autograd.grad(y, (o, z, w), s["dy"].double()))


# --------------------------------------------------------- what a pass cannot do without


def work(case):
    op = case["op"]
    if op == "recurrence":
        e, C = (2 if case["dtype"] == "bf16" else 4), case["C"]
        lens = [int(n) for n in case["lens"].split(",")] if case["lens"] else None
        n = (sum(lens) if lens else case["B"] * case["T"]) * C
        states = (len(lens) if lens else case["B"]) * C
        # forward: x, a, b in, h out; states in and out
        nbytes = n * (3 * e + 4) + states * 4 * (1 + case["init"]) + 8 * C
        flops = 12 * n
        if case["train"]:
            # backward: x, a, b, h, dout in, dx, da, db out; three vectors per sequence
            nbytes += n * (6 * e + 8) + states * 4 * (2 + case["init"]) + 16 * C
            flops += 30 * n
        return {"bytes": nbytes, "flops": flops}
    if op == "layer_norm":
        e, d, rows = (2 if case["dtype"] == "bf16" else 4), case["d"], case["rows"]
        nbytes, flops = rows * d * 2 * e + rows * 8 + 4 * d * (1 + case["bias"]), 7 * rows * d
        if case["train"]:
            nbytes += rows * d * 3 * e + rows * 8 + 12 * d
            flops += 14 * rows * d
        return {"bytes": nbytes, "flops": flops}
    if op == "conv":
        n, C = case["B"] * case["T"] * case["C"], case["C"]
        # x, dy in, dx out; taps in, their gradients out; states
        return {"bytes": n * 6 + C * 36 + C * 4 * case["bias"] +
                case["B"] * C * 12 * (1 + 2 * case["state"]), "flops": 36 * n}
    e, n = (2 if case["zdtype"] == "bf16" else 4), case["rows"] * case["d"]
    # o, z, dy in, do, dz out
    return {"bytes": n * (12 + 2 * e) + 8 * case["d"], "flops": 25 * n}
