"""Linear attention with a decay for each head on the GPU, against the recurrence
in 64 bits, token by token.

Bounds.  Beside each value the reference keeps the same sum over absolute values
(``o_abs``, ``S_abs``).  A rounding to bf16 is off by at most 2^-8 of the value, one
to fp32 by 2^-24.
  o, bf16: its own rounding, that of the weights q.k and that of the state it is
    read from: |error| <= 2^-8 |o| + 2 (2^-8 + 2^-16) o_abs.  The roundings being
    independent and of either sign, the norm of the error is below 2^-8 of the
    norm of o (each has a root mean square of at most 2^-8 / sqrt 3).
  states, bf16 inputs: keys with their decays are split into three bf16, what is
    left out below 2^-25 of a term: the bounds of fp32.
  fp32: a sum of T tokens, then of dk channels: |error| <= (T + dk + 64) 2^-24 of the
    sum over absolute values, the 64 for the decays' logarithms and exponentials; in
    norm, roundings of either sign add up like a random walk: 2^-18.
"""
import pytest
import torch

from linear_attention_serving_delta_gb300 import kda

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
NORM_O = {"bf16": 2.0 ** -8, "f32": 2.0 ** -18}
NORM_S = {"bf16": 2.0 ** -18, "f32": 2.0 ** -18}


def log_alpha(g, slope, T, H):
    x = torch.ones(T, H, device="cuda", dtype=torch.float64) if g is None else torch.nn.functional.softplus(g.double())
    return -x if slope is None else -x * slope.double()


def spread(x, H):
    return x.double().repeat_interleave(H // x.shape[1], dim=1)


def walk(q, k, v, loga, S, scale, order):
    """The recurrence over the tokens `order`; o, o over absolute values, states of both kinds."""
    A = S.abs()
    o, oa = [], []
    for t in order:
        a = torch.exp(loga[t])[:, None, None]
        S = a * S + k[t][:, :, None] * v[t][:, None, :]
        A = a * A + k[t].abs()[:, :, None] * v[t].abs()[:, None, :]
        if q is not None:
            o.append(scale * torch.einsum("hd,hde->he", q[t], S))
            oa.append(abs(scale) * torch.einsum("hd,hde->he", q[t].abs(), A))
    return o, oa, S, A


def close(got, want, total, dtype, T, dk, what, state=False):
    got, err = got.double(), (got.double() - want).abs()
    if state:
        lim = (T + 64) * 2.0 ** -24 * total
        norm = NORM_S[dtype]
    elif dtype == "bf16":
        lim, norm = 2.0 ** -8 * want.abs() + 2 * (2.0 ** -8 + 2.0 ** -16) * total, NORM_O[dtype]
    else:
        lim, norm = (T + dk + 64) * 2.0 ** -24 * total, NORM_O[dtype]
    assert torch.isfinite(got).all(), what
    assert bool((err <= lim + 1e-30).all()), (what, float((err / (lim + 1e-30)).max()))
    rel = float(err.norm() / want.norm().clamp(min=1e-30))
    assert rel <= norm, (what, rel)


def inputs(seed, T, H, Hk, dk, dv, dtype, gate, n=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    d = dict(q=rand(T, Hk, dk).to(DT[dtype]), k=rand(T, Hk, dk).to(DT[dtype]), v=rand(T, H, dv).to(DT[dtype]),
             g=None, slope=None)
    if gate in ("g", "both"):
        d["g"] = (rand(T, H) - 2.0).to(DT[dtype])
    if gate == "strong":  # most tokens forget nearly everything, some nothing
        d["g"] = (40.0 * rand(T, H)).to(DT[dtype])
    if gate in ("slope", "both"):
        d["slope"] = 2.0 ** (-8.0 * torch.arange(H, device="cuda") / max(1, H - 1)).float()
    if gate == "keep":  # nothing is forgotten
        d["slope"] = torch.zeros(H, device="cuda")
    d["state"] = None if n is None else rand(n, H, dk, dv)
    return d


def offsets(lens):
    cu = torch.zeros(len(lens) + 1, dtype=torch.int64)
    cu[1:] = torch.tensor(lens).cumsum(0)
    return cu.cuda()


def check_prefill(d, lens, H, dk, dtype, o, final, scale, slots=None, what=""):
    T = d["v"].shape[0]
    loga = log_alpha(d["g"], d["slope"], T, H)
    q, k, v = spread(d["q"], H), spread(d["k"], H), d["v"].double()
    at = 0
    for s, n in enumerate(lens):
        row = s if slots is None else slots[s]
        if row < 0:
            at += n
            continue
        S = torch.zeros(H, dk, v.shape[2], device="cuda", dtype=torch.float64)
        if d["state"] is not None:
            S = d["state"][row].double()
        ro, roa, rS, rA = walk(q, k, v, loga, S, scale, range(at, at + n))
        if n:
            close(o[at:at + n], torch.stack(ro), torch.stack(roa), dtype, n, dk, (what, "o", s))
        if final is not None:
            close(final[row], rS, rA, dtype, n, dk, (what, "state", s), state=True)
        at += n


SIZES = [(16, 16), (32, 32), (64, 64), (128, 128), (256, 256), (128, 64), (64, 128), (16, 256), (256, 16), (32, 128)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", SIZES)
def test_prefill_sizes(dtype, dk, dv):
    H, Hk, lens = 4, 2, [130, 0, 1, 257, 64]
    d = inputs(dk + 7 * dv, sum(lens), H, Hk, dk, dv, dtype, "g", n=len(lens))
    o, final = kda.lin_prefill(d["q"], d["k"], d["v"], offsets(lens), g=d["g"], scale=dk ** -0.5,
                               initial_state=d["state"])
    check_prefill(d, lens, H, dk, dtype, o, final, dk ** -0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", ["g", "slope", "both", "strong", "keep"])
@pytest.mark.parametrize("H,Hk", [(1, 1), (6, 3), (8, 1)])
def test_prefill_gates_and_heads(dtype, gate, H, Hk):
    lens = [1, 2, 127, 128, 129, 3, 300]
    d = inputs(H + 11, sum(lens), H, Hk, 64, 64, dtype, gate)
    o, final = kda.lin_prefill(d["q"], d["k"], d["v"], offsets(lens), g=d["g"], slope=d["slope"])
    check_prefill(d, lens, H, 64, dtype, o, final, 1.0)


def test_prefill_alphas_of_zero_and_one():
    lens, H = [200], 2
    d = inputs(3, 200, H, H, 64, 64, "bf16", "g", n=1)
    d["g"][5, 0] = d["g"][130, 1] = float("inf")     # forget everything
    d["g"][6:9] = float("-inf")                      # keep everything
    o, final = kda.lin_prefill(d["q"], d["k"], d["v"], offsets(lens), g=d["g"], initial_state=d["state"])
    d["g"] = d["g"].double().clamp(-1e4, 1e4)
    check_prefill(d, lens, H, 64, "bf16", o, final, 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_slots_in_place_and_rows_left_alone(dtype):
    lens, H, Hk, dk, dv = [70, 0, 131, 40], 4, 4, 64, 64
    slots = [5, 2, -1, 0]
    T, pad = sum(lens), 9
    d = inputs(21, T + pad, H, Hk, dk, dv, dtype, "g", n=7)
    pool = d["state"].clone()
    o = torch.full((T + pad, H, dv), 7.0, device="cuda", dtype=DT[dtype])
    cu, sl = offsets(lens), torch.tensor(slots, device="cuda", dtype=torch.int32)
    call = kda.LinPrefill(d["q"], d["k"], d["v"], cu, g=d["g"], initial_state=pool, final_state=pool, state_slots=sl, o=o)
    call.run()
    check_prefill(d, lens, H, dk, dtype, o, pool, 1.0, slots)
    assert call.device_status() == 0
    assert bool((o[T:] == 7).all()) and bool((o[70:201] == 7).all())
    for row in (1, 2, 3, 4, 6):
        assert torch.equal(pool[row], d["state"][row])


def test_prefill_without_states():
    lens = [33, 90]
    d = inputs(5, 123, 2, 2, 128, 128, "bf16", "g")
    o, none = kda.lin_prefill(d["q"], d["k"], d["v"], offsets(lens), g=d["g"], final_state=None)
    assert none is None
    check_prefill(d, lens, 2, 128, "bf16", o, None, 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_in_pieces(dtype):
    """A prompt in two calls that share the pool is the prompt in one, and no tokens at all keep the states."""
    lens, H, dk = [700], 4, 64
    d = inputs(8, 700, H, H, dk, dk, dtype, "both", n=1)
    pool = d["state"].clone()
    o = torch.empty_like(d["v"])
    for a, b in ((0, 300), (300, 300), (300, 700)):
        kda.lin_prefill(d["q"][a:b], d["k"][a:b], d["v"][a:b], offsets([b - a]), g=d["g"][a:b], slope=d["slope"],
                        initial_state=pool, final_state=pool, o=o[a:b])
    check_prefill(d, lens, H, dk, dtype, o, pool, 1.0)


def test_prefill_unaligned():
    """Tensors that start in the middle of 16 bytes."""
    lens, H, dk = [150, 20], 2, 64
    d = inputs(9, 170, H, H, dk, dk, "bf16", "g")
    for x in ("q", "k", "v", "g"):
        y = torch.empty(d[x].numel() + 1, device="cuda", dtype=d[x].dtype)[1:].view(d[x].shape)
        d[x] = y.copy_(d[x])
    o = torch.empty(170 * H * dk + 1, device="cuda", dtype=torch.bfloat16)[1:].view(170, H, dk)
    _, final = kda.lin_prefill(d["q"], d["k"], d["v"], offsets(lens), g=d["g"], o=o)
    check_prefill(d, lens, H, dk, "bf16", o, final, 1.0)


@pytest.mark.parametrize("cu,flag,good", [([0, 50, 40, 100], 1, [0]), ([0, 50, 200, 100], 1, [0]), ([3, 50, 60, 100], 1, [1, 2])])
def test_prefill_malformed_offsets(cu, flag, good):
    H, dk = 2, 64
    d = inputs(31, 100, H, H, dk, dk, "bf16", "g")
    cut = torch.tensor(cu, device="cuda")
    final = torch.full((3, H, dk, dk), 7.0, device="cuda")
    call = kda.LinPrefill(d["q"], d["k"], d["v"], cut, g=d["g"], final_state=final).run()
    assert call.device_status() == flag
    loga = log_alpha(d["g"], None, 100, H)
    for s in good:
        _, _, S, A = walk(None, spread(d["k"], H), d["v"].double(), loga,
                          torch.zeros(H, dk, dk, device="cuda", dtype=torch.float64), 1.0, range(cu[s], cu[s + 1]))
        close(final[s], S, A, "bf16", cu[s + 1] - cu[s], dk, s, state=True)
    bad = [s for s in range(3) if cu[s + 1] < cu[s] or cu[s + 1] > 100 or (s == 0 and cu[0])]
    for s in bad:
        assert bool((final[s] == 7).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_values_that_are_not_finite(dtype):
    """From its token on, in its own channel and head; no token before it, no sequence beside it."""
    lens, H, dk, dv = [200, 150], 2, 64, 64
    d = inputs(13, 350, H, H, dk, dv, dtype, "g")
    clean, fc = kda.lin_prefill(d["q"], d["k"], d["v"], offsets(lens), g=d["g"])
    d["v"][60, 0, 5] = float("inf")
    d["v"][150, 0, 9] = float("nan")
    o, final = kda.lin_prefill(d["q"], d["k"], d["v"], offsets(lens), g=d["g"])
    same = torch.ones(350, H, dv, dtype=torch.bool, device="cuda")
    same[60:200, 0, 5] = same[150:200, 0, 9] = False
    assert torch.equal(o[same], clean[same])
    assert not torch.isfinite(o[~same].float()).any()
    cols = torch.ones(2, H, dk, dv, dtype=torch.bool, device="cuda")
    cols[0, 0, :, 5] = cols[0, 0, :, 9] = False
    assert torch.equal(final[cols], fc[cols]) and not torch.isfinite(final[~cols]).any()
    # keys, queries, gates: nothing before the token, nothing in another head or sequence
    for name, x in (("k", (70, 1, 3)), ("q", (70, 1, 3)), ("g", (70, 1))):
        d = inputs(13, 350, H, H, dk, dv, dtype, "g")
        d[name][x] = float("nan")
        o, final = kda.lin_prefill(d["q"], d["k"], d["v"], offsets(lens), g=d["g"])
        same = torch.ones(350, H, dtype=torch.bool, device="cuda")
        same[70:200, 1] = False
        assert torch.equal(o[same], clean[same]), name
        assert not torch.isfinite(o[70, 1].float()).any(), name
        if name == "q":
            assert torch.equal(final, fc) and torch.equal(o[71:], clean[71:])
        else:
            assert torch.equal(final[:, 0], fc[:, 0]) and torch.equal(final[1], fc[1])
            assert not torch.isfinite(final[0, 1]).all()


def test_prefill_same_bits_every_time_and_in_a_graph():
    lens, H = [513, 77, 1200], 8
    d = inputs(17, sum(lens), H, 2, 128, 128, "bf16", "g", n=3)
    call = kda.LinPrefill(d["q"], d["k"], d["v"], offsets(lens), g=d["g"], initial_state=d["state"]).run()
    o, f = call.o.clone(), call.final_state.clone()
    call.o.zero_()
    call.final_state.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call.run(side)
    for _ in range(2):
        call.o.zero_()
        call.final_state.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(call.o, o) and torch.equal(call.final_state, f)
    assert call.device_status() == 0


# Long prompts: cut into segments where the chains would not fill the GPU, and planned in any case
LONG = [([5000], 2, 2, 64, 64, "g"), ([3000, 0, 1, 2500], 2, 1, 128, 128, "slope"), ([4100], 1, 1, 256, 128, "both"),
        ([2600, 1300, 17], 3, 3, 64, 128, "strong"), ([2300, 900], 40, 8, 32, 16, "keep"), ([6000], 4, 4, 128, 64, "g")]


@pytest.mark.parametrize("lens,H,Hk,dk,dv,gate", LONG)
def test_prefill_long(lens, H, Hk, dk, dv, gate):
    d = inputs(60 + dk, sum(lens), H, Hk, dk, dv, "bf16", gate, n=len(lens))
    o, final = kda.lin_prefill(d["q"], d["k"], d["v"], offsets(lens), g=d["g"], slope=d["slope"], scale=dk ** -0.5,
                               initial_state=d["state"])
    check_prefill(d, lens, H, dk, "bf16", o, final, dk ** -0.5)


def test_prefill_long_slots_in_place():
    lens, slots, H, dk = [2500, 40, 1200, 0], [4, -1, 0, 2], 2, 64
    T = sum(lens)
    d = inputs(71, T, H, H, dk, dk, "bf16", "g", n=6)
    pool = d["state"].clone()
    o = torch.full((T, H, dk), 7.0, device="cuda", dtype=torch.bfloat16)
    call = kda.LinPrefill(d["q"], d["k"], d["v"], offsets(lens), g=d["g"], initial_state=pool, final_state=pool, o=o,
                          state_slots=torch.tensor(slots, device="cuda", dtype=torch.int32))
    call.run()
    check_prefill(d, lens, H, dk, "bf16", o, pool, 1.0, slots)
    assert call.device_status() == 0 and bool((o[2500:2540] == 7).all())
    for row in (1, 2, 3, 5):
        assert torch.equal(pool[row], d["state"][row])


def test_prefill_many_sequences():
    """More chains than the CTAs take at once; a long prompt among short ones."""
    lens = [(37 * i) % 300 for i in range(90)] + [2000]
    d = inputs(81, sum(lens), 4, 2, 64, 64, "bf16", "g")
    o, final = kda.lin_prefill(d["q"], d["k"], d["v"], offsets(lens), g=d["g"])
    check_prefill(d, lens, 4, 64, "bf16", o, final, 1.0)


@pytest.mark.parametrize("H", [2, 40])
def test_prefill_long_values_that_are_not_finite(H):
    lens, dk = [2600, 400], 64
    d = inputs(14, 3000, H, H, dk, dk, "bf16", "g")
    clean, fc = kda.lin_prefill(d["q"], d["k"], d["v"], offsets(lens), g=d["g"])
    d["v"][60, 0, 5] = float("inf")
    d["v"][2500, 1, 9] = float("nan")
    o, final = kda.lin_prefill(d["q"], d["k"], d["v"], offsets(lens), g=d["g"])
    same = torch.ones(3000, H, dk, dtype=torch.bool, device="cuda")
    same[60:2600, 0, 5] = same[2500:2600, 1, 9] = False
    assert torch.equal(o[same], clean[same]) and not torch.isfinite(o[~same].float()).any()
    cols = torch.ones(2, H, dk, dk, dtype=torch.bool, device="cuda")
    cols[0, 0, :, 5] = cols[0, 1, :, 9] = False
    assert torch.equal(final[cols], fc[cols]) and not torch.isfinite(final[~cols]).any()


def test_prefill_long_malformed_offsets():
    """What two sequences that overlap between malformed ones add up to is refused past the call's room."""
    H, dk, T = 2, 64, 2560
    d = inputs(32, T, H, H, dk, dk, "bf16", "g")
    cut = torch.tensor([0, T, 100, T, 200, T], device="cuda")
    final = torch.full((5, H, dk, dk), 7.0, device="cuda")
    call = kda.LinPrefill(d["q"], d["k"], d["v"], cut, g=d["g"], final_state=final).run()
    assert call.device_status() == 1
    loga = log_alpha(d["g"], None, T, H)
    _, _, S, A = walk(None, spread(d["k"], H), d["v"].double(), loga,
                      torch.zeros(H, dk, dk, device="cuda", dtype=torch.float64), 1.0, range(T))
    close(final[0], S, A, "bf16", T, dk, 0, state=True)
    assert all(bool((final[s] == 7).all()) for s in (1, 3))


def test_prefill_long_same_bits_every_time_and_in_a_graph():
    lens, H = [2500, 1300], 4
    d = inputs(18, sum(lens), H, 2, 128, 128, "bf16", "both", n=2)
    call = kda.LinPrefill(d["q"], d["k"], d["v"], offsets(lens), g=d["g"], slope=d["slope"], initial_state=d["state"]).run()
    o, f = call.o.clone(), call.final_state.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call.run(side)
    for _ in range(3):
        call.o.zero_()
        call.final_state.zero_()
        call.workspace.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(call.o, o) and torch.equal(call.final_state, f)
    assert call.device_status() == 0


# Token by token, in segments too: every size with and without a second column a lane
@pytest.mark.parametrize("lens,H,Hk,dk,dv,gate", [
    ([1500], 2, 2, 64, 64, "g"), ([700, 0, 1, 33, 400], 2, 1, 128, 128, "slope"), ([900], 1, 1, 256, 128, "both"),
    ([600, 300, 17], 3, 3, 16, 256, "strong"), ([800, 90], 6, 2, 32, 16, "keep"), ([1000], 4, 4, 128, 32, "g")])
def test_prefill_f32_long(lens, H, Hk, dk, dv, gate):
    d = inputs(160 + dk, sum(lens), H, Hk, dk, dv, "f32", gate, n=len(lens))
    o, final = kda.lin_prefill(d["q"], d["k"], d["v"], offsets(lens), g=d["g"], slope=d["slope"], scale=dk ** -0.5,
                               initial_state=d["state"])
    check_prefill(d, lens, H, dk, "f32", o, final, dk ** -0.5)


def test_prefill_f32_long_slots_in_place_and_in_a_graph():
    lens, slots, H, dk = [900, 40, 500, 0], [4, -1, 0, 2], 2, 64
    T = sum(lens)
    d = inputs(171, T, H, H, dk, dk, "f32", "g", n=6)
    pool = d["state"].clone()
    o = torch.full((T, H, dk), 7.0, device="cuda")
    call = kda.LinPrefill(d["q"], d["k"], d["v"], offsets(lens), g=d["g"], initial_state=pool, final_state=pool, o=o,
                          state_slots=torch.tensor(slots, device="cuda", dtype=torch.int32))
    call.run()
    check_prefill(d, lens, H, dk, "f32", o, pool, 1.0, slots)
    assert call.device_status() == 0 and bool((o[900:940] == 7).all())
    for row in (1, 2, 3, 5):
        assert torch.equal(pool[row], d["state"][row])
    first, after = o.clone(), pool.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call.run(side)
    for _ in range(2):
        pool.copy_(d["state"])
        call.workspace.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, first) and torch.equal(pool, after)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_few_of_many_sequences(dtype):
    """More sequences than the plan takes at once, nearly all skipped, three cut into segments."""
    n, H, dk = 1500, 2, 32
    lens = [i % 2 for i in range(n)]
    lens[0], lens[1200], lens[1499] = 2300, 900, 1
    slots = [-1] * n
    slots[0], slots[1200], slots[1499], slots[700] = 3, 0, 1, 2
    T = sum(lens)
    d = inputs(41, T, H, H, dk, dk, dtype, "g", n=4)
    o = torch.full((T, H, dk), 7.0, device="cuda", dtype=DT[dtype])
    pool = d["state"].clone()
    call = kda.LinPrefill(d["q"], d["k"], d["v"], offsets(lens), g=d["g"], initial_state=pool, final_state=pool, o=o,
                          state_slots=torch.tensor(slots, device="cuda", dtype=torch.int32)).run()
    check_prefill(d, lens, H, dk, dtype, o, pool, 1.0, slots)
    at = offsets(lens).tolist()
    assert call.device_status() == 0 and all(bool((o[at[s]:at[s + 1]] == 7).all()) for s in range(n) if slots[s] < 0)


@pytest.mark.parametrize("dtype,T,H,dk,dv", [("bf16", 9000, 1, 64, 64), ("f32", 3000, 1, 32, 32), ("bf16", 3500, 38, 64, 128)])
def test_prefill_most_segments(dtype, T, H, dk, dv):
    d = inputs(43, T, H, 1, dk, dv, dtype, "both", n=1)
    o, final = kda.lin_prefill(d["q"], d["k"], d["v"], offsets([T]), g=d["g"], slope=d["slope"], scale=dk ** -0.5,
                               initial_state=d["state"])
    check_prefill(d, [T], H, dk, dtype, o, final, dk ** -0.5)


@pytest.mark.parametrize("dtype,lens", [("bf16", [130, 7]), ("bf16", [2500, 130]), ("f32", [90]), ("f32", [700, 33])])
def test_prefill_rows_behind_the_last_sequence(dtype, lens):
    H, dk, more = 2, 64, 70
    T = sum(lens)
    d = inputs(23, T + more, H, H, dk, dk, dtype, "g")
    for x in ("q", "k", "v", "g"):
        d[x][T:] = float("nan")
    o = torch.full((T + more, H, dk), 7.0, device="cuda", dtype=DT[dtype])
    call = kda.LinPrefill(d["q"], d["k"], d["v"], offsets(lens), g=d["g"], o=o).run()
    check_prefill({**d, "v": d["v"][:T], "q": d["q"][:T], "k": d["k"][:T], "g": d["g"][:T]}, lens, H, dk, dtype, o[:T],
                  call.final_state, 1.0)
    assert bool((o[T:] == 7).all()) and call.device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefills_at_once_on_two_streams(dtype):
    lens, H, dk = [1500, 400], 4, 64
    calls, want = [], []
    for i in range(2):
        d = inputs(200 + i, sum(lens), H, 2, dk, dk, dtype, "g", n=2)
        calls.append(kda.LinPrefill(d["q"], d["k"], d["v"], offsets(lens), g=d["g"], initial_state=d["state"]))
        calls[i].run()
        want.append((calls[i].o.clone(), calls[i].final_state.clone()))
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(4):
        for c, s in zip(calls, streams):
            c.run(s)
    torch.cuda.synchronize()
    for c, (o, f) in zip(calls, want):
        assert torch.equal(c.o, o) and torch.equal(c.final_state, f)


def test_prefill_long_unaligned():
    lens, H, dk = [1100, 20], 2, 64
    d = inputs(19, sum(lens), H, H, dk, dk, "bf16", "g")
    for x in ("q", "k", "v", "g"):
        y = torch.empty(d[x].numel() + 1, device="cuda", dtype=d[x].dtype)[1:].view(d[x].shape)
        d[x] = y.copy_(d[x])
    o, final = kda.lin_prefill(d["q"], d["k"], d["v"], offsets(lens), g=d["g"])
    check_prefill(d, lens, H, dk, "bf16", o, final, 1.0)


# ------------------------------------------------------------------ single tokens
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", SIZES)
def test_decode_sizes(dtype, dk, dv):
    B, H, Hk = 5, 4, 2
    d = inputs(dk + 3 * dv, B, H, Hk, dk, dv, dtype, "both", n=8)
    slots = [7, 0, -1, 3, 2]
    pool = d["state"].clone()
    o = torch.full((B, H, dv), 7.0, device="cuda", dtype=DT[dtype])
    call = kda.LinDecode(d["q"], d["k"], d["v"], pool, g=d["g"], slope=d["slope"], scale=dk ** -0.5,
                         state_slots=torch.tensor(slots, device="cuda", dtype=torch.int32), o=o).run()
    assert call.device_status() == 0
    loga = log_alpha(d["g"], d["slope"], B, H)
    for r, slot in enumerate(slots):
        if slot < 0:
            assert bool((o[r] == 7).all())
            continue
        ro, roa, S, A = walk(spread(d["q"], H), spread(d["k"], H), d["v"].double(), loga, d["state"][slot].double(),
                             dk ** -0.5, [r])
        # (decode holds everything in fp32: its o is off by its own rounding and fp32's)
        err = (o[r].double() - ro[0]).abs()
        lim = (2.0 ** -8 if dtype == "bf16" else 0.0) * ro[0].abs() + (dk + 65) * 2.0 ** -24 * roa[0] * (1 + 2.0 ** -8)
        assert bool((err <= lim).all())
        close(pool[slot], S, A, "f32", 1, dk, r, state=True)
    for row in (1, 4, 5, 6):
        assert torch.equal(pool[row], d["state"][row])


@pytest.mark.parametrize("gate", ["g", "slope", "strong", "keep"])
def test_decode_follows_a_prompt(gate):
    """Token by token from the prompt's state is the longer prompt; constant decays do not drift."""
    H, dk, T, more = 4, 64, 40, 300
    d = inputs(41, T + more, H, H, dk, dk, "f32", gate)
    _, pool = kda.lin_prefill(d["q"][:T], d["k"][:T], d["v"][:T], offsets([T]), g=None if d["g"] is None else d["g"][:T],
                              slope=d["slope"])
    rows = []
    for t in range(T, T + more):
        rows.append(kda.lin_decode(d["q"][t:t + 1], d["k"][t:t + 1], d["v"][t:t + 1], pool,
                                   g=None if d["g"] is None else d["g"][t:t + 1], slope=d["slope"]))
    o, final = torch.cat(rows), pool
    loga = log_alpha(d["g"], d["slope"], T + more, H)
    ro, roa, S, A = walk(spread(d["q"], H), spread(d["k"], H), d["v"].double(), loga,
                         torch.zeros(H, dk, dk, device="cuda", dtype=torch.float64), 1.0, range(T + more))
    close(o, torch.stack(ro[T:]), torch.stack(roa[T:]), "f32", T + more, dk, "o")
    close(final[0], S, A, "f32", T + more, dk, "state", state=True)


def test_decode_bad_slots_and_empty():
    d = inputs(2, 3, 2, 2, 32, 32, "bf16", "g", n=4)
    pool, o = d["state"].clone(), torch.full((3, 2, 32), 7.0, device="cuda", dtype=torch.bfloat16)
    call = kda.LinDecode(d["q"], d["k"], d["v"], pool, g=d["g"], o=o,
                         state_slots=torch.tensor([1, 4, 1 << 30], device="cuda", dtype=torch.int32)).run()
    assert call.device_status() == 32 and bool((o[1:] == 7).all()) and not bool((o[0] == 7).all())
    for row in (0, 2, 3):
        assert torch.equal(pool[row], d["state"][row])
    empty = kda.lin_decode(d["q"][:0], d["k"][:0], d["v"][:0], pool, g=d["g"][:0])
    assert empty.shape == (0, 2, 32)


# ------------------------------------------------------------------ trees
def make_tree(kind, lens, seed):
    g = torch.Generator().manual_seed(seed)
    par = []
    for n in lens:
        idx = torch.arange(n)
        if kind == "chain":
            par.append(idx - 1)
        elif kind == "star":
            par.append(torch.full((n,), -1))
        else:
            par.append((torch.rand(n, generator=g) * (idx + 1)).long() - 1)
    return torch.cat(par).int() if par else torch.zeros(0, dtype=torch.int32)


def path_of(par, i):
    p = []
    while i >= 0:
        p.insert(0, i)
        i = int(par[i])
    return p


def check_draft(d, lens, par, H, dk, dtype, o, scale, slots=None):
    loga = log_alpha(d["g"], d["slope"], d["v"].shape[0], H)
    q, k, v = spread(d["q"], H), spread(d["k"], H), d["v"].double()
    at = 0
    for s, n in enumerate(lens):
        row = s if slots is None else slots[s]
        if row >= 0 and n:
            want, total = [], []
            for i in range(n):
                x = walk(q, k, v, loga, d["state"][row].double(), scale, [at + j for j in path_of(par[at:at + n], i)])
                want.append(x[0][-1])
                total.append(x[1][-1])
            close(o[at:at + n], torch.stack(want), torch.stack(total), dtype, n, dk, ("draft", s))
        at += n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", SIZES)
def test_draft_and_commit_sizes(dtype, dk, dv):
    H, Hk, lens = 4, 2, [5, 0, 1, 17, 8]
    T = sum(lens)
    d = inputs(5 * dk + dv, T, H, Hk, dk, dv, dtype, "both", n=9)
    par, slots = make_tree("tree", lens, dk + dv), [4, 1, 8, 0, 5]
    sl = torch.tensor(slots, device="cuda", dtype=torch.int32)
    before = d["state"].clone()
    decay = dict(g=d["g"], slope=d["slope"], parents=par.cuda(), state_slots=sl)
    call = kda.LinDraft(d["q"], d["k"], d["v"], offsets(lens), d["state"], scale=dk ** -0.5, **decay).run()
    assert call.device_status() == 0 and torch.equal(before, d["state"])
    check_draft(d, lens, par, H, dk, dtype, call.o, dk ** -0.5, slots)
    last = [4, -1, 0, 11, -1]
    pool = d["state"].clone()
    c = kda.LinCommit(d["k"], d["v"], offsets(lens), torch.tensor(last, device="cuda", dtype=torch.int32), pool, **decay)
    c.run()
    assert c.device_status() == 0
    check_commit(d, lens, par, H, dk, pool, last, slots)


@pytest.mark.parametrize("most,dv", [(30, 32), (60, 64), (60, 128)])
def test_draft_many_requests(most, dv):
    """More CTAs than the small calls' split of a tree's tiles allows."""
    H, dk, n = 8, 64, 40
    lens = [(7 * i + 3) % (most + 1) for i in range(n)]
    d = inputs(most + dv, sum(lens), H, 2, dk, dv, "bf16", "g", n=n)
    par = make_tree("tree", lens, 5)
    o = kda.lin_draft(d["q"], d["k"], d["v"], offsets(lens), d["state"], parents=par.cuda(), g=d["g"], max_seqlen=most)
    check_draft(d, lens, par, H, dk, "bf16", o, 1.0)


def check_commit(d, lens, par, H, dk, pool, last, slots, untouched=True):
    loga = log_alpha(d["g"], d["slope"], d["v"].shape[0], H)
    k, v, at = spread(d["k"], H), d["v"].double(), 0
    for s, n in enumerate(lens):
        if last[s] < 0:
            assert torch.equal(pool[slots[s]], d["state"][slots[s]])
        else:
            path = [at + j for j in path_of(par[at:at + n], last[s])]
            _, _, S, A = walk(None, k, v, loga, d["state"][slots[s]].double(), 1.0, path)
            close(pool[slots[s]], S, A, "f32", len(path), dk, ("commit", s), state=True)
        at += n
    if untouched:
        for row in set(range(pool.shape[0])) - set(slots):
            assert torch.equal(pool[row], d["state"][row])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["chain", "star", "tree"])
@pytest.mark.parametrize("gate,H,Hk", [("g", 3, 3), ("slope", 8, 1), ("strong", 2, 2), ("keep", 2, 1)])
def test_draft_and_commit_trees(dtype, kind, gate, H, Hk):
    lens, dk, dv = [64, 33, 16, 15, 2], 64, 128
    T = sum(lens)
    d = inputs(77, T, H, Hk, dk, dv, dtype, gate, n=5)
    par = make_tree(kind, lens, 3)
    decay = dict(g=d["g"], slope=d["slope"], parents=None if kind == "chain" else par.cuda())
    o = kda.lin_draft(d["q"], d["k"], d["v"], offsets(lens), d["state"], max_seqlen=64, **decay)
    check_draft(d, lens, par, H, dk, dtype, o, 1.0)
    last = [63, 20, -1, 14, 0]
    out = torch.zeros_like(d["state"])
    kda.lin_commit(d["k"], d["v"], offsets(lens), torch.tensor(last, device="cuda", dtype=torch.int32), d["state"],
                   state_out=out, max_seqlen=64, **decay)
    check_commit(d, lens, par, H, dk, out, last, list(range(5)))


@pytest.mark.parametrize("parents,last,lens,most,flag,bad", [
    ([-1, 0, 2, -1, 0, 0], [1, 1], [3, 3], 0, 32, 0),      # a token that follows itself
    ([-1, 0, -2, -1, 0, 0], [1, 1], [3, 3], 0, 32, 0),
    ([-1, 0, 1, -1, 300, 0], [1, 1], [3, 3], 0, 32, 1),    # (300 would be 44 in eight bits)
    ([-1, 0, 1, -1, 256, 0], [1, 1], [3, 3], 0, 32, 1),
    ([-1, 0, 1, -1, -1, 0], [1, 1], [4, 2], 3, 128, 0),     # longer than was said
])
def test_malformed_trees(parents, last, lens, most, flag, bad):
    H, dk, T = 2, 32, 6
    d = inputs(1, T, H, H, dk, dk, "bf16", "g", n=2)
    par, cu = torch.tensor(parents, dtype=torch.int32), offsets(lens)
    o = torch.full((T, H, dk), 7.0, device="cuda", dtype=torch.bfloat16)
    call = kda.LinDraft(d["q"], d["k"], d["v"], cu, d["state"], parents=par.cuda(), g=d["g"], o=o, max_seqlen=most).run()
    assert call.device_status() == flag
    at = [0, lens[0], T]
    assert bool((o[at[bad]:at[bad + 1]] == 7).all())
    one = dict(d, q=d["q"][at[1 - bad]:at[2 - bad]], k=d["k"][at[1 - bad]:at[2 - bad]], v=d["v"][at[1 - bad]:at[2 - bad]],
               g=d["g"][at[1 - bad]:at[2 - bad]], state=d["state"][1 - bad:2 - bad])
    check_draft(one, [lens[1 - bad]], par[at[1 - bad]:at[2 - bad]], H, dk, "bf16", o[at[1 - bad]:at[2 - bad]], 1.0)
    pool = d["state"].clone()
    c = kda.LinCommit(d["k"], d["v"], cu, torch.tensor(last, device="cuda", dtype=torch.int32), pool, parents=par.cuda(),
                      g=d["g"], max_seqlen=most).run()
    assert c.device_status() == flag and torch.equal(pool[bad], d["state"][bad])
    assert not torch.equal(pool[1 - bad], d["state"][1 - bad])


@pytest.mark.parametrize("last,flag", [([3, 0], 32), ([-2, 0], 32), ([-1, 0], 0)])
def test_accepted_tokens_out_of_range(last, flag):
    d = inputs(4, 5, 2, 2, 16, 16, "f32", "g", n=2)
    pool = d["state"].clone()
    c = kda.LinCommit(d["k"], d["v"], offsets([3, 2]), torch.tensor(last, device="cuda", dtype=torch.int32), pool,
                      g=d["g"]).run()
    assert c.device_status() == flag and torch.equal(pool[0], d["state"][0])


def test_drafted_values_that_are_not_finite():
    """A token off the path changes nothing on it, whatever it holds."""
    lens, H, dk = [20], 2, 64
    for dtype in ("bf16", "f32"):
        d = inputs(6, 20, H, H, dk, dk, dtype, "g", n=1)
        par = torch.arange(20, dtype=torch.int32) - 2
        par[0] = par[1] = -1                          # two chains, even and odd tokens
        kw = dict(parents=par.cuda(), g=d["g"])
        clean = kda.lin_draft(d["q"], d["k"], d["v"], offsets(lens), d["state"], **kw)
        for x in ("k", "v"):
            d[x][7, 0, 3] = float("nan")
        d["v"][9, 1, 3] = float("inf")
        o = kda.lin_draft(d["q"], d["k"], d["v"], offsets(lens), d["state"], **kw)
        assert torch.equal(o[0::2], clean[0::2]) and torch.equal(o[1:7:2], clean[1:7:2])
        assert not torch.isfinite(o[7::2, 0, 3].float()).any()
        pool = kda.lin_commit(d["k"], d["v"], offsets(lens), torch.tensor([18], device="cuda").int(), d["state"].clone(), **kw)
        assert torch.isfinite(pool).all()


def test_serving_steps():
    """Prompts into a pool, a draft, its commit, single tokens after it: the recurrence over what was accepted."""
    H, Hk, dk, dv, dtype = 4, 2, 64, 64, "bf16"
    lens, rows = [150, 40, 9], [3, 1, 4]
    sl = torch.tensor(rows, device="cuda", dtype=torch.int32)
    pool = torch.zeros(6, H, dk, dv, device="cuda")
    d = inputs(50, sum(lens), H, Hk, dk, dv, dtype, "both")
    o, _ = kda.lin_prefill(d["q"], d["k"], d["v"], offsets(lens), g=d["g"], slope=d["slope"], initial_state=pool,
                           final_state=pool, state_slots=sl)
    drafts = [6, 8, 3]
    e = inputs(51, sum(drafts), H, Hk, dk, dv, dtype, "both")
    e["slope"] = d["slope"]
    par = make_tree("tree", drafts, 9)
    kw = dict(parents=par.cuda(), g=e["g"], slope=e["slope"], state_slots=sl)
    od = kda.lin_draft(e["q"], e["k"], e["v"], offsets(drafts), pool, **kw)
    last = [4, -1, 2]
    kda.lin_commit(e["k"], e["v"], offsets(drafts), torch.tensor(last, device="cuda", dtype=torch.int32), pool, **kw)
    f = inputs(52, 3, H, Hk, dk, dv, dtype, "both")
    oc = kda.lin_decode(f["q"], f["k"], f["v"], pool, g=f["g"], slope=d["slope"], state_slots=sl)
    at = bt = 0
    for s, n in enumerate(lens):
        path = path_of(par[bt:bt + drafts[s]], last[s]) if last[s] >= 0 else []
        pick = lambda x, y, z: torch.cat([spread(x, H)[at:at + n]] + [spread(y, H)[bt + j:bt + j + 1] for j in path]  # noqa: E731,B023
                                         + [spread(z, H)[s:s + 1]])  # noqa: B023
        q, k, v = pick(d["q"], e["q"], f["q"]), pick(d["k"], e["k"], f["k"]), pick(d["v"], e["v"], f["v"])
        la = lambda x: log_alpha(x["g"], d["slope"], x["v"].shape[0], H)  # noqa: E731
        loga = torch.cat([la(d)[at:at + n]] + [la(e)[bt + j:bt + j + 1] for j in path] + [la(f)[s:s + 1]])
        ro, roa, S, A = walk(q, k, v, loga, torch.zeros(H, dk, dv, device="cuda", dtype=torch.float64), 1.0, range(q.shape[0]))
        got = torch.cat([o[at:at + n]] + [od[bt + j:bt + j + 1] for j in path] + [oc[s:s + 1]])
        close(got, torch.stack(ro), torch.stack(roa), dtype, n, dk, ("o", s))
        close(pool[rows[s]], S, A, dtype, n, dk, ("state", s), state=True)
        at, bt = at + n, bt + drafts[s]
