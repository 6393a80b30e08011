"""The gated linear recurrence (gdr_linear_recurrence[_f32] and its backward calls) against the
fp64 oracle, and its refusals.

Tolerances, from the arithmetic before any run.  With u = 2^-22 (the special-function unit's
exponential and reciprocal; fp32 roundings are 2^-24): the relative error of a log-decay is a
few u, and x e^-x <= 0.37 bounds what it does to a decay; a state passes at most 16 rounded
per-token decays inside a tile, 8 joins of tile parts, and one join of two roundings per 64
tokens.  So |err h| <= (32 + T / 64) u * H with H the same recurrence over absolute values,
likewise for the adjoint D; products of both get the sum of the two, and sums over tokens
(64 + T / 16) u of the sum of magnitudes.  A bf16 output adds half a step, 2^-8 of its value."""

import numpy as np
import pytest

import gated_delta_rule_145_b200 as gdr
from gated_delta_rule_145_b200 import synth
from oracle import block

torch = pytest.importorskip("torch")
U = 2.0 ** -22
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
NAMES = ("h", "final", "dx", "da", "db", "dA_log", "ddt_bias", "dinit")


def make(B, T, C, dtype="bf16", seed=0, lens=None, init=True, gate_scale=1.0):
    rng = np.random.default_rng(seed)
    cu = None
    if lens is not None:
        cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        B, T = 1, max(T, int(cu[-1]))
    n = B if cu is None else len(lens)
    r = synth.round_to_bf16 if dtype == "bf16" else (lambda v: v)
    f = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
    dt = np.exp(rng.uniform(np.log(1e-3), np.log(1e-1), C))
    return dict(x=r(f(B, T, C)), a=r(gate_scale * f(B, T, C)), b=r(gate_scale * f(B, T, C)),
                A_log=rng.uniform(0, synth.LN16, C).astype(np.float32),
                dt_bias=np.log(np.expm1(dt)).astype(np.float32),
                init=f(n, C) if init else None, cu=cu, go=f(B, T, C),
                gf=f(n, C) if init else None, dtype=dtype, n=n)


def dev(v, dtype=None):
    if v is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(v)).cuda()
    return t if dtype is None else t.to(dtype)


def on_gpu(m, fused=False):
    """(arguments of the forward call, out, final, the six gradients)"""
    dt = torch.bfloat16 if m["dtype"] == "bf16" else torch.float32
    x, a, b = (dev(m[k], dt) for k in ("x", "a", "b"))
    if fused:
        C = x.shape[2]
        x, a, b = torch.cat([x, a, b], 2).split(C, 2)
    args = (x, a, b, dev(m["A_log"]), dev(m["dt_bias"]))
    init, cu = dev(m["init"]), dev(m["cu"])
    out, final = gdr.linear_recurrence(*args, init, cu)
    grads = gdr.linear_recurrence_backward(*args, out, dev(m["go"]), dev(m["gf"]), init, cu)
    torch.cuda.synchronize()
    assert gdr.gdr_device_status() == gdr.GDR_OK
    return args, (out, final) + tuple(grads)


def expected(m):
    args = (m["x"], m["a"], m["b"], m["A_log"], m["dt_bias"])
    ref = block.linear_recurrence(*args, m["init"], m["cu"])
    ref += block.linear_recurrence_backward(*args, m["go"], m["gf"], m["init"], m["cu"])
    return ref, block.recurrence_magnitude(*args, m["go"], m["gf"], m["init"], m["cu"])


def check(m, got, ref, mag, longest):
    state, both, sums = 32 + longest / 64, 80 + longest / 32, 96 + m["x"].shape[1] / 16
    factor = dict(h=state, final=state, dx=4 + state, da=both, db=8 + state, dA_log=sums,
                  ddt_bias=sums, dinit=4 + state)
    for name, g, r, k in zip(NAMES, got, ref, mag):
        g = g.float().cpu().numpy().astype(np.float64)
        inside = np.isfinite(r)  # rows outside the sequences are not written
        tol = factor[name] * U * k + 1e-30
        if name in ("dx", "da", "db"):
            tol = tol + HALF[m["dtype"]] * np.abs(r)
        bad = ~(np.abs(g - r) <= tol) & inside
        worst = np.max((np.abs(g - r) / tol)[inside]) if inside.any() else 0.0
        assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} outside, worst {worst:.2f} x"


gpu = pytest.mark.gpu

# lengths around the token counts of a warp (8, 16), of a tile (64, 128) and of a cluster's
# step; channel counts around a strip (64), below one and far above
DENSE = [(1, 1, 8), (3, 1, 64), (64, 1, 72), (2, 2, 136), (1, 15, 64), (2, 16, 64), (1, 17, 8),
         (1, 63, 64), (2, 64, 56), (1, 65, 128), (2, 127, 64), (1, 128, 200), (1, 129, 64),
         (1, 255, 64), (3, 257, 72), (1, 1023, 64), (1, 1024, 64), (1, 1025, 8), (2, 777, 1160),
         (1, 2500, 136), (40, 33, 64)]


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,C", DENSE)
def test_dense(B, T, C, dtype):
    m = make(B, T, C, dtype, seed=T * 7 + C, init=(T + C) % 3 != 0)
    ref, mag = expected(m)
    check(m, on_gpu(m)[1], ref, mag, T)


# around the tiles of the forms with one CTA per SM (48 to 256 tokens), their clusters' steps, and
# those of the forms with two, which take many sequences
EDGES = [(1, t, 64) for t in (39, 41, 48, 56, 79, 81, 95, 97, 111, 113, 159, 161, 225, 256, 449, 511,
                              513, 1281, 3000)] + [(160, t, 136) for t in (129, 191, 193, 256)]


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,C", EDGES)
def test_tile_edges(B, T, C, dtype):
    m = make(B, T, C, dtype, seed=T + C, init=T % 2 == 0)
    got = on_gpu(m)[1]
    m, got = some_channels(m, got, 1 + B // 40)
    ref, mag = expected(m)
    check(m, got, ref, mag, T)


PACKED = [[1], [0, 5, 0], [1, 1, 1, 1], [17, 0, 64, 1, 130], [300, 3, 128, 129, 0, 1, 255],
          [0, 1500, 2], [64, 64, 64], [2000]]


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", PACKED)
def test_packed(lens, dtype):
    m = make(1, 0, 136, dtype, seed=sum(lens) + len(lens), lens=lens)
    ref, mag = expected(m)
    check(m, on_gpu(m)[1], ref, mag, max(lens))


def median_ms(call, n=9):
    times = []
    for _ in range(n + 2):
        start, end = torch.cuda.Event(True), torch.cuda.Event(True)
        start.record()
        call()
        end.record()
        end.synchronize()
        times.append(start.elapsed_time(end))
    return sorted(times[2:])[n // 2]


@gpu
@pytest.mark.parametrize("longest,others,each", [(2048, 255, 1), (8192, 255, 1), (30000, 999, 6)])
def test_a_long_prompt_among_short_sequences(longest, others, each):
    """the mean length says short sequences, for which a token at a time is best: the long one must
    not be walked that way, which took 6 to 22 times as long as the same tokens in equal sequences"""
    C, T = 6144, longest + others * each
    x, a, b = (torch.randn(1, T, C, device="cuda").bfloat16() for _ in range(3))
    p, go = torch.zeros(C, device="cuda"), torch.randn(1, T, C, device="cuda")
    equal = [T // (others + 1)] * (others + 1)
    equal[0] += T - sum(equal)
    times = []
    for lens in ([longest] + [each] * others, equal):
        cu = dev(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))
        out, final = gdr.linear_recurrence(x, a, b, p, p, None, cu)
        times.append((median_ms(lambda: gdr.linear_recurrence(x, a, b, p, p, None, cu, out, final)),
                      median_ms(lambda: gdr.linear_recurrence_backward(x, a, b, p, p, out, go, None, None, cu))))
    assert times[0][0] <= 4 * times[1][0] and times[0][1] <= 4 * times[1][1], times


# long sequences among many short ones: none long, one, several, lengths around the limit that
# parts them (some 80 tokens here), the first, the last and empty ones, all tokens in one
def _mixed(long, n=300):
    lens = [(7 * i) % 6 for i in range(n)]
    for at, length in long.items():
        lens[at] = length
    return lens


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,C", [
    (_mixed({}), 1024), (_mixed({0: 3000}), 1000), (_mixed({299: 901, 298: 0, 0: 333}), 1024),
    (_mixed({i: 70 + i // 7 for i in range(3, 290, 14)}), 1096), ([0] * 299 + [2000], 1024),
    ([2000] + [0] * 299, 520), (_mixed({40: 5000}, 900), 6144)])
def test_packed_with_long_and_short_sequences(lens, C, dtype):
    m = make(1, 0, C, dtype, seed=len(lens) + C, lens=lens)
    got = on_gpu(m)[1]
    again = on_gpu(m)[1]
    for name, p, q in zip(NAMES, got, again):
        assert torch.equal(p, q), name
    m, got = some_channels(m, got, max(1, C // 64) | 1)
    ref, mag = expected(m)
    check(m, got, ref, mag, max(lens))


@gpu
def test_packed_with_long_sequences_in_place_and_replayed_on_other_lengths():
    """the lengths are read on the device: a graph of one batch serves the next, whose long sequences
    are others; states updated in place have the bits of those apart"""
    C, n = 1024, 300
    batches = [_mixed({5: 1500, 200: 700}), _mixed({0: 90, 299: 2000}), _mixed({7: 64, 8: 0})]
    T = max(map(sum, batches)) + 50
    g = torch.Generator(device="cuda").manual_seed(8)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    x, a, b = (r(1, T, C).bfloat16() for _ in range(3))
    A, d, init, gf, go = r(C), r(C), r(n, C), r(n, C), r(1, T, C)
    cus = [dev(np.concatenate([[0], np.cumsum(v)]).astype(np.int32)) for v in batches]
    cu, state = cus[0].clone(), init.clone()

    def step(state):
        out, final = gdr.linear_recurrence(x, a, b, A, d, state, cu, final_state=state)
        return (out, final) + gdr.linear_recurrence_backward(x, a, b, A, d, out, go, gf, init, cu)

    step(state)
    graph, cap = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    cap.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=cap):
        got = step(state)
    torch.cuda.current_stream().wait_stream(cap)
    for other in cus:
        out, final = gdr.linear_recurrence(x, a, b, A, d, init, other)
        want = (out, final) + gdr.linear_recurrence_backward(x, a, b, A, d, out, go, gf, init, other)
        cu.copy_(other)
        state.copy_(init)
        graph.replay()
        torch.cuda.synchronize()
        for name, p, q in zip(NAMES, want, got):
            assert torch.equal(p, q), name
    del graph


def some_channels(m, got, every):
    """the case and its results at every `every`-th channel: channels do not mix"""
    cut = dict(m)
    for k in ("x", "a", "b", "go", "A_log", "dt_bias", "init", "gf"):
        if m[k] is not None:
            cut[k] = m[k][..., ::every]
    return cut, tuple(g[..., ::every] for g in got)


# calls large enough for clusters of CTAs and for sequences cut between them: few strips and long,
# some strips, a strip count that no cluster count divides, many strips; ragged lengths; the
# last one's sequences differ in nothing but their place
LARGE = [(1, 30000, 192, "bf16"), (1, 20011, 1024, "bf16"), (1, 5000, 6144, "bf16"),
         (2, 4099, 2048, "bf16"), (3, 1500, 4104, "bf16"), (1, 6000, 328, "f32"),
         (2, 3000, 2048, "f32"), (1, 9001, 5000, "f32"), (5, 700, 4096, "f32")]


@gpu
@pytest.mark.parametrize("B,T,C,dtype", LARGE)
def test_large(B, T, C, dtype):
    m = make(B, T, C, dtype, seed=C)
    got = on_gpu(m)[1]
    again = on_gpu(m)[1]
    for name, p, q in zip(NAMES, got, again):
        assert torch.equal(p, q), name
    m, got = some_channels(m, got, max(1, B * T * C // 3_000_000))
    ref, mag = expected(m)
    check(m, got, ref, mag, T)


# more strips than the SMs take at once
MANY = [(5, 1300, 4104, "bf16"), (8, 520, 6144, "bf16"), (3, 1999, 5000, "f32"), (6, 640, 4160, "f32")]


@gpu
@pytest.mark.parametrize("B,T,C,dtype", MANY)
def test_more_strips_than_sms(B, T, C, dtype):
    m = make(B, T, C, dtype, seed=T)
    got = on_gpu(m)[1]
    again = on_gpu(m)[1]
    for name, p, q in zip(NAMES, got, again):
        assert torch.equal(p, q), name
    m, got = some_channels(m, got, max(1, B * T * C // 3_000_000))
    ref, mag = expected(m)
    check(m, got, ref, mag, T)


# packed documents of ragged lengths, empty ones among them, by units (strips x documents): more
# than the SMs take at once, between one and two per SM, and so few that clusters take them
WIDE = [([433, 64, 751, 0, 228, 16, 325, 129], 6144), ([900, 0, 411, 77], 4096),
        ([1733, 256, 3001, 0, 911, 64, 1300, 517], 1024), ([2500, 0, 1999], 2056), ([0, 7001, 3], 520)]


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,C", WIDE)
def test_wide_packed(lens, C, dtype):
    m = make(1, 0, C, dtype, seed=C + len(lens), lens=lens)
    got = on_gpu(m)[1]
    again = on_gpu(m)[1]
    for name, p, q in zip(NAMES, got, again):
        assert torch.equal(p, q), name
    for i, n in enumerate(lens):
        if n == 0:
            assert torch.equal(got[1][i], dev(m["init"])[i]) and torch.equal(got[7][i], dev(m["gf"])[i])
    m, got = some_channels(m, got, max(1, sum(lens) * C // 2_000_000) | 1)
    ref, mag = expected(m)
    check(m, got, ref, mag, max(lens))


@gpu
def test_large_calls_on_two_streams_and_from_a_graph():
    """calls whose clusters hand states to one another, two at a time"""
    ms = [make(1, 5000, 6144, seed=3), make(1, 20011, 1024, seed=4)]
    want = [on_gpu(m)[1] for m in ms]
    ready = [([dev(m[k], torch.bfloat16) for k in ("x", "a", "b")] +
              [dev(m["A_log"]), dev(m["dt_bias"])], dev(m["init"]), dev(m["go"]), dev(m["gf"]))
             for m in ms]
    streams = [torch.cuda.Stream() for _ in ms]
    torch.cuda.synchronize()
    got = [None, None]

    def both():
        for i, s in enumerate(streams):
            args, init, go, gf = ready[i]
            with torch.cuda.stream(s):
                out, final = gdr.linear_recurrence(*args, init)
                got[i] = (out, final) + gdr.linear_recurrence_backward(*args, out, go, gf, init)

    for _ in range(4):
        both()
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for name, p, q in zip(NAMES, w, g):
            assert torch.equal(p, q), name
    graph, cap = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    cap.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=cap):
        for s in streams:
            s.wait_stream(cap)
        both()
        for s in streams:
            cap.wait_stream(s)
    torch.cuda.current_stream().wait_stream(cap)
    for _ in range(3):
        for g in got:
            for t in g:
                t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            for name, p, q in zip(NAMES, w, g):
                assert torch.equal(p, q), name
    assert gdr.gdr_device_status() == gdr.GDR_OK
    del graph


@gpu
@pytest.mark.parametrize("B,T,C", [(1, 1, 64), (2, 300, 72), (3, 20, 136)])
def test_slices_of_one_projection(B, T, C):
    """x, a, b as slices of [B, T, 3 C], the gradients written into slices of one buffer:
    bit-identical to dense inputs, and the buffer's other columns untouched"""
    m = make(B, T, C, seed=5)
    _, dense = on_gpu(m)
    args, fused = on_gpu(m, fused=True)
    for name, p, q in zip(NAMES, dense, fused):
        assert torch.equal(p, q), name
    pad = torch.full((B, T, 3 * C + 16), 7.0, device="cuda", dtype=torch.bfloat16)
    gx, ga, gb = pad[..., 8:8 + 3 * C].split(C, 2)
    gdr.linear_recurrence_backward(*args, fused[0], dev(m["go"]), dev(m["gf"]), dev(m["init"]),
                                   grad_x=gx, grad_a=ga, grad_b=gb)
    torch.cuda.synchronize()
    for p, q in zip((gx, ga, gb), dense[2:5]):
        assert torch.equal(p, q)
    assert (pad[..., :8] == 7).all() and (pad[..., 8 + 3 * C:] == 7).all()


@gpu
@pytest.mark.parametrize("lens,lead", [([100, 30, 200], 0), ([3, 2], 0), ([70, 5], 12)])
def test_rows_outside_the_sequences_stay_and_are_not_read(lens, lead):
    """tokens before cu_seqlens[0] and behind cu_seqlens[-1] hold NaN and stay as they were"""
    C, tail = 72, 37
    m = make(1, 0, C, seed=3, lens=lens)
    T = lead + sum(lens) + tail
    big = {}
    for k in ("x", "a", "b", "go"):
        big[k] = np.full((1, T, C), np.nan, np.float32)
        big[k][:, lead:lead + sum(lens)] = m[k]
    cu = dev((m["cu"] + lead).astype(np.int32))
    x, a, b = (dev(big[k], torch.bfloat16) for k in ("x", "a", "b"))
    args = (x, a, b, dev(m["A_log"]), dev(m["dt_bias"]))
    out = torch.full((1, T, C), 5.0, device="cuda")
    grads = [torch.full((1, T, C), 5.0, device="cuda", dtype=torch.bfloat16) for _ in range(3)]
    _, final = gdr.linear_recurrence(*args, dev(m["init"]), cu, out=out)
    kept = out.clone()
    kept[:, :lead] = float("nan")
    kept[:, lead + sum(lens):] = float("nan")
    got = gdr.linear_recurrence_backward(*args, kept, dev(big["go"]), dev(m["gf"]),
                                         dev(m["init"]), cu, *grads)
    torch.cuda.synchronize()
    inner = slice(lead, lead + sum(lens))
    for v in (out,) + tuple(got[:3]):
        assert (v[:, :lead] == 5).all() and (v[:, lead + sum(lens):] == 5).all()
    # (not bit by bit against a call without the outer rows: the number of tokens chooses
    # among forms that add in another order)
    ref, mag = expected(m)
    check(m, (out[:, inner], final) + tuple(g[:, inner] for g in got[:3]) + tuple(got[3:]), ref,
          mag, max(lens))


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,lead,tail", [([100, 30, 200], 0, 37), ([70, 5], 12, 0), ([0, 0], 3, 9),
                                            ([900, 700], 40, 2000)])
def test_rows_outside_the_sequences_are_zero_in_tensors_that_the_call_allocates(lens, lead, tail,
                                                                                dtype):
    """whatever the memory held before: a padded row is then nothing in the sums that follow"""
    C, T = 136, lead + sum(lens) + tail
    g = torch.Generator(device="cuda").manual_seed(T)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    x, a, b = (r(1, T, C).to(dtype) for _ in range(3))
    A, d, init, gf, go = r(C), r(C), r(len(lens), C), r(len(lens), C), r(1, T, C)
    cu = dev((lead + np.concatenate([[0], np.cumsum(lens)])).astype(np.int32))
    kept = torch.full((1, T, C), 7.0, device="cuda")
    want = [torch.full((1, T, C), 7.0, device="cuda", dtype=dtype) for _ in range(3)]
    gdr.linear_recurrence(x, a, b, A, d, init, cu, out=kept)
    gdr.linear_recurrence_backward(x, a, b, A, d, kept, go, gf, init, cu, *want)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    waste = [torch.full((1, T, C), float("nan"), device="cuda", dtype=t)
             for t in (torch.float32, dtype) for _ in range(6)]
    del waste
    out, _ = gdr.linear_recurrence(x, a, b, A, d, init, cu)
    grads = gdr.linear_recurrence_backward(x, a, b, A, d, out, go, gf, init, cu)[:3]
    torch.cuda.synchronize()
    inner = torch.zeros(T, device="cuda", dtype=torch.bool)
    inner[lead:lead + sum(lens)] = True
    for v, w in zip((out, *grads), (kept, *want)):
        assert (v[:, ~inner] == 0).all() and (w[:, ~inner] == 7).all()
        assert torch.equal(v[:, inner], w[:, inner])


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_extreme_gates(dtype):
    """decays that underflow in one token, decays of exactly 1, closed and open input gates"""
    m = make(2, 300, 64, dtype, seed=11)
    m["a"][:, ::3] = -200.0
    m["a"][:, 1::7] = 100.0
    m["b"][:, ::5] = 150.0
    m["b"][:, 2::5] = -150.0
    ref, mag = expected(m)
    check(m, on_gpu(m)[1], ref, mag, 300)


@gpu
@pytest.mark.parametrize("lo,hi", [(-80, -30), (-30, -4), (-4, 4), (4, 80)])
@pytest.mark.parametrize("B,T,C", [(3, 7, 136), (2, 700, 64), (5, 1300, 4104)])
def test_fp32_input_gates_to_fp32_rounding(B, T, C, lo, hi):
    """with the past forgotten at every token and x and grad_out of one, h is sigmoid(b), dx too,
    db sigmoid(b) sigmoid(-b).  Each is at most an exponential (2 ulps, 2^-22, and three roundings
    of its correction), a sum, two reciprocals (an ulp, 2^-23, each) and three products: below
    14 x 2^-24 < 2^-20 of its value"""
    g = torch.Generator(device="cuda").manual_seed(T)
    b = torch.rand(B, T, C, device="cuda", generator=g) * (hi - lo) + lo
    one, p = torch.ones_like(b), torch.zeros(C, device="cuda")
    a = torch.full_like(b, 1e30)
    h, _ = gdr.linear_recurrence(one, a, b, p, p)
    dx, _, db, *_ = gdr.linear_recurrence_backward(one, a, b, p, p, h, one)
    s = torch.sigmoid(b.double())
    for name, got, ref in (("h", h, s), ("dx", dx, s), ("db", db, s * torch.sigmoid(-b.double()))):
        off = float(((got.double() - ref).abs() / (2.0 ** -20 * ref + 1e-36)).max())
        assert off <= 1, f"{name}: {off:.2f} x"


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,C", [(2, 5, 64), (2, 300, 64), (1, 5000, 192), (5, 1300, 4104)])
def test_gates_masked_with_the_highest_and_lowest_values(B, T, C, dtype):
    """a and b at the type's ends, as masks write them: the state is forgotten or kept, the input gate
    shut or open, and every gradient is finite"""
    m = make(B, T, C, dtype, seed=23)
    high = torch.finfo(torch.bfloat16 if dtype == "bf16" else torch.float32).max
    m["a"][:, 2::9], m["a"][:, 3::11, ::2] = high, -high
    m["a"][:, 4::13, 1::2] = -np.inf
    m["b"][:, 1::7], m["b"][:, 2::5, ::2], m["b"][:, 3::17, 1::2] = -high, high, -np.inf
    got = on_gpu(m)[1]
    m, got = some_channels(m, got, max(1, B * T * C // 3_000_000) | 1)
    ref, mag = expected(m)
    assert all(np.isfinite(r).all() for r in ref)
    check(m, got, ref, mag, T)


@gpu
def test_infinite_and_nan_inputs_stay_in_their_channel_and_after_their_token():
    m = make(2, 200, 64, "f32", seed=12, init=False)
    clean = on_gpu(m)[1]
    m["x"][0, 90, 3] = np.inf
    m["x"][0, 100, 5] = np.nan
    out, final = on_gpu(m)[1][:2]
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[0, 90:, 3] = True
    hit[0, 100:, 5] = True
    assert torch.equal(out[~hit], clean[0][~hit])
    assert torch.isinf(out[0, 90, 3]) and torch.isnan(out[0, 100:, 5]).all()
    assert torch.equal(final[1], clean[1][1])


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,C", [(2, 40, 64), (1, 300, 64), (1, 5000, 192), (3, 3000, 2048),
                                   (160, 256, 136), (5, 1300, 4104)])
def test_an_infinite_state_stays_infinite(B, T, C, dtype):
    """whatever form takes the call: no tile border makes inf - inf of it, nor an underflowing decay,
    of one token or of many, 0 inf; the same for its gradient"""
    m = make(B, T, C, dtype, seed=21)
    m["A_log"][::2], m["A_log"][1::2] = synth.LN16, -2.0  # 2^-40 per token or so, some 2^-130; and slow
    m["dt_bias"][::2], m["dt_bias"][1::2] = 1.5, -4.0
    m["x"][0, 7, ::5], m["x"][0, 9, 1::5] = np.inf, -np.inf
    m["init"][-1, 2::5] = np.inf
    m["go"][0, T - 5, 3::5] = -np.inf
    got = on_gpu(m)[1]
    m, got = some_channels(m, got, max(1, B * T * C // 3_000_000) | 1)
    with np.errstate(invalid="ignore"):
        ref, mag = expected(m)
    for i in (0, 1, 2, 7):  # h, the final state, dx and dinit
        g, r = got[i].float().cpu().numpy(), ref[i]
        assert np.isinf(r).any() and not np.isnan(r).any()
        assert np.array_equal(np.isinf(g), np.isinf(r)), NAMES[i]
        assert (g[np.isinf(r)] == r[np.isinf(r)]).all(), NAMES[i]
    with np.errstate(invalid="ignore"):
        check(m, [got[i] for i in (0, 1, 2)], ref[:3], mag[:3], T)


@gpu
@pytest.mark.parametrize("B,T,C", [(2, 40, 64), (1, 300, 64), (1, 5000, 192), (5, 1300, 4104)])
def test_a_nan_gate_makes_the_state_nan(B, T, C):
    m = make(B, T, C, "f32", seed=22)
    m["a"][0, 20, 3], m["b"][0, 21, 5] = np.nan, np.nan
    got = on_gpu(m)[1]
    hit = torch.zeros_like(got[0], dtype=torch.bool)
    hit[0, 20:, 3] = True
    hit[0, 21:, 5] = True
    assert torch.equal(torch.isnan(got[0]), hit) and torch.equal(torch.isnan(got[1]), hit[:, -1])
    back = torch.zeros_like(hit)  # the gradients of what a NaN decay hands on
    back[0, :20, 3] = True
    assert torch.isnan(got[2][back]).all() and torch.isnan(got[7][0, 3])
    assert torch.isnan(got[5][3]) and torch.isnan(got[6][3]) and torch.isnan(got[4][0, 21, 5])


@gpu
@pytest.mark.parametrize("T0", [1, 40, 300])
def test_steps_continue_a_prompt_in_place(T0):
    """a prompt, then single-token calls that update the state in place, equal one call"""
    m = make(3, T0 + 6, 136, seed=T0)
    args, want = on_gpu(m)
    x, a, b, A, dt = args
    part = lambda t, lo, hi: t[:, lo:hi].contiguous()  # noqa: E731
    outs = []
    out, state = gdr.linear_recurrence(*(part(t, 0, T0) for t in (x, a, b)), A, dt,
                                       dev(m["init"]))
    outs.append(out)
    for t in range(T0, T0 + 6):
        o, s = gdr.linear_recurrence(*(part(v, t, t + 1) for v in (x, a, b)), A, dt, state,
                                     final_state=state)
        assert s is state
        outs.append(o)
    torch.cuda.synchronize()
    ref, mag = expected(m)
    got = torch.cat(outs, 1).cpu().numpy()
    assert (np.abs(got - ref[0]) <= (40 + T0 / 64) * U * mag[0] + 1e-30).all()
    assert (np.abs(state.cpu().numpy() - ref[1]) <= (40 + T0 / 64) * U * mag[1] + 1e-30).all()


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,T,C", [(70, 3, 136), (300, 150, 64), (2, 5000, 64), (3, 3000, 2048)])
def test_a_state_in_place_has_the_bits_of_one_apart(B, T, C, dtype):
    """final_state may be init_state and grad_init_state grad_final_state: one CTA, clusters,
    and units cut between clusters"""
    g = torch.Generator(device="cuda").manual_seed(B + T)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    x, a, b = (r(B, T, C).to(dtype) for _ in range(3))
    A, dt, init, gf, go = r(C), r(C), r(B, C), r(B, C), r(B, T, C)
    out, final = gdr.linear_recurrence(x, a, b, A, dt, init)
    apart = gdr.linear_recurrence_backward(x, a, b, A, dt, out, go, gf, init)
    state, grad = init.clone(), gf.clone()
    again, _ = gdr.linear_recurrence(x, a, b, A, dt, state, final_state=state)
    call = gdr.gdr_linear_recurrence_backward if dtype is torch.bfloat16 else \
        gdr.gdr_linear_recurrence_backward_f32
    dx, da, db = (torch.empty_like(x) for _ in range(3))
    dA, ddt = torch.empty_like(A), torch.empty_like(dt)
    call(x, a, b, A, dt, init, out, go, grad, dx, da, db, dA, ddt, grad, None, B, T, C, C, C)
    torch.cuda.synchronize()
    assert torch.equal(again, out) and torch.equal(state, final)
    for name, p, q in zip(NAMES[2:], (dx, da, db, dA, ddt, grad), apart):
        assert torch.equal(p, q), name


@gpu
def test_no_tokens():
    C = 64
    e = torch.empty((2, 0, C), device="cuda", dtype=torch.bfloat16)
    p = torch.zeros(C, device="cuda")
    init, gf = torch.randn(2, C, device="cuda"), torch.randn(2, C, device="cuda")
    out, final = gdr.linear_recurrence(e, e, e, p, p, init)
    g = gdr.linear_recurrence_backward(e, e, e, p, p, out, torch.empty(2, 0, C, device="cuda"),
                                       gf, init)
    torch.cuda.synchronize()
    assert torch.equal(final, init) and torch.equal(g[5], gf)
    assert (g[3] == 0).all() and (g[4] == 0).all()


@gpu
@pytest.mark.parametrize("B,T,C", [(1, 700, 64), (4, 300, 136), (64, 1, 64), (5, 9, 64)])
def test_same_bits_again_alone_and_from_a_graph(B, T, C):
    m = make(B, T, C, seed=B + T)
    args, first = on_gpu(m)
    _, again = on_gpu(m)
    for name, p, q in zip(NAMES, first, again):
        assert torch.equal(p, q), name
    # the first sequence alone
    one = dict(m, x=m["x"][:1], a=m["a"][:1], b=m["b"][:1], go=m["go"][:1], n=1)
    if m["init"] is not None:
        one.update(init=m["init"][:1], gf=m["gf"][:1])
    alone = on_gpu(one)[1]
    U_ = (32 + T / 64) * U
    mag = expected(one)[1]
    diff = (alone[0][0] - first[0][0]).abs().cpu().numpy()
    assert (diff <= 2 * U_ * mag[0][0] + 1e-30).all()
    # captured once, replayed twice on fresh inputs in the same buffers
    init, go, gf = dev(m["init"]), dev(m["go"]), dev(m["gf"])
    out, final = torch.empty_like(first[0]), torch.empty_like(first[1])
    graph, cap = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    cap.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=cap):
        gdr.linear_recurrence(*args, init, out=out, final_state=final, stream=cap)
        grads = gdr.linear_recurrence_backward(*args, out, go, gf, init, stream=cap)
    torch.cuda.current_stream().wait_stream(cap)
    for _ in range(2):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for name, p, q in zip(NAMES, (out, final) + tuple(grads), first):
            assert torch.equal(p, q), name
    assert gdr.gdr_device_status() == gdr.GDR_OK
    del graph


@gpu
def test_two_streams_at_once():
    """calls on two streams without ordering between them: each has its own workspace"""
    ms = [make(2, 400, 136, seed=s) for s in (1, 2)]
    want = [on_gpu(m)[1] for m in ms]
    streams = [torch.cuda.Stream() for _ in ms]
    ready = []
    for m in ms:
        dt = torch.bfloat16
        ready.append(([dev(m[k], dt) for k in ("x", "a", "b")] + [dev(m["A_log"]), dev(m["dt_bias"])],
                      dev(m["init"]), dev(m["go"]), dev(m["gf"])))
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(5):
        for i, s in enumerate(streams):
            args, init, go, gf = ready[i]
            with torch.cuda.stream(s):
                out, final = gdr.linear_recurrence(*args, init)
                got[i] = (out, final) + gdr.linear_recurrence_backward(*args, out, go, gf, init)
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for name, p, q in zip(NAMES, w, g):
            assert torch.equal(p, q), name


# --------------------------------------------------------------------------- refusals (no GPU)

A = 1 << 20  # fake aligned addresses: every call below fails a check before any launch


def _fwd(name="gdr_linear_recurrence", **kw):
    args = dict(x=A, a=A, b=A, A_log=A, dt_bias=A, init_state=None, out=A, final_state=None,
                cu_seqlens=None, B=1, T=16, C=64, ld=64)
    args.update(kw)
    return getattr(gdr, name)(**args, stream=0, check=False)


def _bwd(name="gdr_linear_recurrence_backward", **kw):
    args = dict(x=A, a=A, b=A, A_log=A, dt_bias=A, init_state=None, out=A, grad_out=A,
                grad_final_state=None, grad_x=A, grad_a=A, grad_b=A, grad_A_log=A,
                grad_dt_bias=A, grad_init_state=None, cu_seqlens=None, B=1, T=16, C=64, ld=64,
                ld_grad=64)
    args.update(kw)
    return getattr(gdr, name)(**args, stream=0, check=False)


@pytest.mark.parametrize("call,suffix", [(_fwd, ""), (_fwd, "_f32"), (_bwd, ""), (_bwd, "_f32")])
def test_refusals(call, suffix):
    name = call.__defaults__[0] + suffix
    for p in ("x", "a", "b", "A_log", "dt_bias", "out"):
        assert call(name, **{p: None}) == gdr.GDR_ERR_NULL, p
    for kw in (dict(B=0), dict(T=-1), dict(C=0), dict(C=60), dict(ld=56), dict(ld=68),
               dict(C=64, ld=32), dict(B=1 << 20, T=1 << 12), dict(ld=1 << 40)):
        assert call(name, **kw) == gdr.GDR_ERR_SHAPE, kw
    for p in ("x", "a", "b", "out", "init_state"):
        assert call(name, **{p: A + 8}) == gdr.GDR_ERR_ALIGN, p
    for p in ("A_log", "dt_bias", "cu_seqlens"):
        assert call(name, **{p: A + 2}) == gdr.GDR_ERR_ALIGN, p
    if call is _fwd:
        assert call(name, final_state=A + 8) == gdr.GDR_ERR_ALIGN
    else:
        for p in ("grad_out", "grad_x", "grad_a", "grad_b", "grad_A_log", "grad_dt_bias"):
            assert call(name, **{p: None}) == gdr.GDR_ERR_NULL, p
        for p in ("grad_out", "grad_x", "grad_a", "grad_b", "grad_final_state",
                  "grad_init_state"):
            assert call(name, **{p: A + 8}) == gdr.GDR_ERR_ALIGN, p
        assert call(name, ld_grad=56) == gdr.GDR_ERR_SHAPE
        assert call(name, ld_grad=68) == gdr.GDR_ERR_SHAPE


def test_refusals_of_zero_outer_rows():
    def call(**kw):
        args = dict(x=A, y=A, z=None, cu_seqlens=A, B=2, T=16, row_bytes=64, pitch_bytes=64)
        args.update(kw)
        return gdr.gdr_zero_outer_rows(**args, stream=0, check=False)

    assert call(cu_seqlens=None) == gdr.GDR_ERR_NULL == call(x=None, y=None)
    for kw in (dict(B=0), dict(T=-1), dict(row_bytes=0), dict(row_bytes=24), dict(pitch_bytes=48),
               dict(pitch_bytes=72), dict(pitch_bytes=1 << 33), dict(T=2 ** 32 + 16),
               dict(row_bytes=2 ** 64 + 64)):
        assert call(**kw) == gdr.GDR_ERR_SHAPE, kw
    for p in ("x", "y", "z"):
        assert call(**{p: A + 8}) == gdr.GDR_ERR_ALIGN, p
    assert call(cu_seqlens=A + 2) == gdr.GDR_ERR_ALIGN


@pytest.mark.parametrize("kw", [dict(T=2 ** 32 + 16), dict(C=2 ** 32 + 64), dict(B=2 ** 32 + 1),
                                dict(T=-2 ** 32 + 16)])
def test_sizes_that_would_wrap_to_others_are_refused(kw):
    assert _fwd(**kw) == gdr.GDR_ERR_SHAPE and _bwd(**kw) == gdr.GDR_ERR_SHAPE


def test_binding_refuses_sizes_that_would_wrap():
    p = torch.zeros(8)
    long = torch.zeros(1, 1, 8).expand(1, 2 ** 32 + 4, 8)
    with pytest.raises(ValueError, match="2\\^31"):
        gdr.linear_recurrence(long, long, long, p, p)
    with pytest.raises(ValueError, match="2\\^31"):
        gdr.short_conv_silu_backward(long, p, long)
    wide = torch.zeros(1, 1).expand(1, 2 ** 32 + 8)
    with pytest.raises(ValueError, match="2\\^31"):
        gdr.layer_norm(wide, p)


def test_binding_refuses_cpu_tensors():
    x, p = torch.zeros(1, 4, 8), torch.zeros(8)
    with pytest.raises(ValueError, match="CUDA"):
        gdr.linear_recurrence(x, x, x, p, p)
    with pytest.raises(ValueError, match="CUDA"):
        gdr.linear_recurrence_backward(x, x, x, p, p, x, x)


@gpu
def test_binding_refuses_what_does_not_fit():
    x, p = torch.zeros(2, 4, 64, device="cuda"), torch.zeros(64, device="cuda")
    h = x.half()
    with pytest.raises(ValueError, match="bf16 or fp32"):
        gdr.linear_recurrence(h, h, h, p, p)
    with pytest.raises(ValueError, match="a must be"):
        gdr.linear_recurrence(x, x.bfloat16(), x, p, p)
    with pytest.raises(ValueError, match="shape"):
        gdr.linear_recurrence(x, x, x, p[:8], p)
    with pytest.raises(ValueError, match="layout"):
        gdr.linear_recurrence(x, x.transpose(0, 1).contiguous().transpose(0, 1), x, p, p)
    with pytest.raises(ValueError, match="layout"):
        gdr.linear_recurrence(x, x[:1].expand(2, 4, 64), x, p, p)
    with pytest.raises(ValueError, match="B == 1"):
        gdr.linear_recurrence(x, x, x, p, p, cu_seqlens=torch.zeros(2, device="cuda",
                                                                    dtype=torch.int32))
    with pytest.raises(ValueError, match="together"):
        gdr.linear_recurrence_backward(x, x, x, p, p, x, x, grad_x=x)
    with pytest.raises(gdr.GdrError):
        gdr.linear_recurrence(x[..., :60].contiguous(), x[..., :60].contiguous(),
                              x[..., :60].contiguous(), p[:60], p[:60])
