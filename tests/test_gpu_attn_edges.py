"""Full attention where masks, groups and values that are not finite meet:
corners beside those of test_gpu_attn.py, with its reference and tolerances.
"""
import pytest
import torch

from linear_attention_serving_delta_gb300 import kda
from test_gpu_attn import Pool, check, cu_of, gen, rand, reference

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ one token to a row tile
@pytest.mark.parametrize("D,dtype", [(256, "bf16"), (128, "bf16"), (128, "f32"), (256, "f32")])
@pytest.mark.parametrize("G", [64, 65, 100, 128])
@pytest.mark.parametrize("at", [5, 100])
def test_later_tokens_never_reach_wide_groups(D, dtype, G, at):
    """Groups of more than 64 query heads: a row tile holds one token, its last key tile those behind it too."""
    g = gen(G + at)
    T = 150
    q, k, v = rand(g, T, 2 * G, D, dtype=dtype), rand(g, T, 2, D, dtype=dtype), rand(g, T, 2, D, dtype=dtype)
    clean = kda.attn_prefill(q, k, v, cu_of([T]).cuda())
    v[at] = float("inf")
    v[at + 1:] = float("nan")
    o = kda.attn_prefill(q, k, v, cu_of([T]).cuda())
    check(o[:at], *reference(q[:at], k[:at], v[:at], 0, D ** -0.5, dtype))
    assert torch.equal(o[:at], clean[:at])
    assert torch.isposinf(o[at].float()).all() and torch.isnan(o[at + 1:].float()).all()


@pytest.mark.parametrize("D,dtype", [(256, "bf16"), (128, "bf16"), (128, "f32"), (256, "f32")])
@pytest.mark.parametrize("G", [65, 128])
def test_later_tokens_of_a_chunk_never_reach_wide_groups(D, dtype, G):
    ctx, new, at = 70, 60, 20
    p = Pool([ctx], [new], 1, D, 16, dtype, 7)
    q = rand(gen(G), new, G, D, dtype=dtype)
    cu = cu_of([new]).cuda()
    clean = kda.attn_paged(q, p.k, p.v, p.table, p.lens, cu)
    x = torch.arange(ctx + at, ctx + new)
    slot = (p.table[0].cpu().long()[x // 16] * 16 + x % 16).cuda()
    p.v.view(-1, 1, D)[slot] = float("nan")
    o = kda.attn_paged(q, p.k, p.v, p.table, p.lens, cu)
    check(o[:at], *reference(q[:at], p.K[0][:ctx + at], p.V[0][:ctx + at], ctx, D ** -0.5, dtype))
    assert torch.equal(o[:at], clean[:at]) and torch.isnan(o[at:].float()).all()


# ------------------------------------------------------------------ values that are not finite
def check_classes(o, q, k, v, pos0, scale, dtype):
    """Each output's kind is that of the values its row attends in its channel: NaN for a NaN or both
    infinities, an infinity for one, and otherwise finite, with the tolerance of the same values without
    the others' (zeros in their place)."""
    H, G = q.shape[1], q.shape[1] // v.shape[1]
    last = torch.arange(pos0, pos0 + q.shape[0], device=q.device).clamp(max=v.shape[0] - 1)

    def any_up_to(hit):  # [m, Hkv, D] -> [n, H, D]: one such value at or before the row's position
        return (hit.cumsum(0) > 0)[last].repeat_interleave(G, 1)

    pos, neg = any_up_to(torch.isposinf(v)), any_up_to(torch.isneginf(v))
    nan = any_up_to(torch.isnan(v)) | (pos & neg)
    assert torch.equal(torch.isnan(o), nan)
    assert torch.equal(torch.isposinf(o), pos & ~nan) and torch.equal(torch.isneginf(o), neg & ~nan)
    ref, tol = reference(q, k, torch.where(torch.isfinite(v), v, torch.zeros_like(v)), pos0, scale, dtype)
    finite = torch.isfinite(o)
    check(torch.where(finite, o, torch.zeros_like(o)), torch.where(finite, ref, torch.zeros_like(ref)),
          torch.where(finite, tol, torch.ones_like(tol)))


def strew(v, seed, share):
    """Infinities of both signs and NaN in a share of v's places, in half of the channels."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    where = torch.rand(v.shape, generator=g, device="cuda") < share
    where[..., ::2] = False
    kind = torch.randint(0, 5, v.shape, generator=g, device="cuda")
    for z, x in enumerate(("inf", "inf", "-inf", "-inf", "nan")):
        v[where & (kind == z)] = float(x)


KINDS = [(4, 2, 64, "bf16"), (8, 2, 128, "bf16"), (6, 2, 32, "bf16"), (4, 2, 256, "bf16"), (130, 2, 256, "bf16"),
         (4, 2, 64, "f32"), (8, 2, 128, "f32"), (100, 1, 128, "f32"), (4, 2, 32, "f32"), (4, 1, 256, "f32")]


@pytest.mark.parametrize("H,Hkv,D,dtype", KINDS)
@pytest.mark.parametrize("share", [0.0005, 0.01])
def test_strewn_values_in_prompts(H, Hkv, D, dtype, share):
    g = gen(H + D)
    lens = [330, 1, 95]
    T = sum(lens)
    q, k, v = rand(g, T, H, D, dtype=dtype), rand(g, T, Hkv, D, dtype=dtype), rand(g, T, Hkv, D, dtype=dtype)
    strew(v, H, share)
    cu = cu_of(lens)
    a = kda.AttnPrefill(q, k, v, cu.cuda()).run()
    assert a.device_status() == 0
    for b, e in zip(cu.tolist(), cu.tolist()[1:]):
        check_classes(a.o[b:e], q[b:e], k[b:e], v[b:e], 0, D ** -0.5, dtype)


@pytest.mark.parametrize("H,Hkv,D,dtype", KINDS)
@pytest.mark.parametrize("ctx,new", [([150, 700], [60, 3]), ([5000, 40], [20, 1]), ([3000, 900, 16], [1, 1, 1])])
def test_strewn_values_in_the_cache(H, Hkv, D, dtype, ctx, new):
    p = Pool(ctx, new, Hkv, D, 16, dtype, 3)
    for i, (c, n) in enumerate(zip(ctx, new)):
        strew(p.V[i], i, 0.001)
        x = torch.arange(c + n)
        slot = (p.table[i].cpu().long()[x // 16] * 16 + x % 16).cuda()
        p.v.view(-1, Hkv, D)[slot] = p.V[i]
    cu = cu_of(new)
    q = rand(gen(H), sum(new), H, D, dtype=dtype)
    a = kda.AttnPaged(q, p.k, p.v, p.table, p.lens, cu.cuda(), max_seqlen=max(new)).run()
    assert a.device_status() == 0
    for i, c in enumerate(ctx):
        b, e = int(cu[i]), int(cu[i + 1])
        check_classes(a.o[b:e], q[b:e], p.K[i], p.V[i], c, D ** -0.5, dtype)


@pytest.mark.parametrize("T,D,dtype", [(45_000, 128, "f32"), (45_000, 64, "f32"), (12_000, 256, "f32"),
                                       (45_000, 128, "bf16")])
def test_two_infinities_far_apart(T, D, dtype):
    """One near each end of a long prompt: their rows get them, the call ends without a flag, and the prompt
    beside it is whole."""
    g = gen(D)
    lens = [T, 300]
    n = sum(lens)
    q, k, v = rand(g, n, 1, D, dtype=dtype), rand(g, n, 1, D, dtype=dtype), rand(g, n, 1, D, dtype=dtype)
    v[3, 0, 5] = float("inf")
    v[T - 3, 0, 9] = -float("inf")
    a = kda.AttnPrefill(q, k, v, cu_of(lens).cuda()).run()
    assert a.device_status() == 0
    for b, e in ((0, 70), (T // 2, T // 2 + 70), (T - 70, T)):
        check_classes(a.o[b:e], q[b:e], k[:e], v[:e], b, D ** -0.5, dtype)
    check_classes(a.o[T:], q[T:], k[T:], v[T:], 0, D ** -0.5, dtype)


@pytest.mark.parametrize("scale", [-0.3, 0.125])
@pytest.mark.parametrize("cu", [[-80, 10, 100], [10, 10, 100], [-1000, -90, 5, 100]])
def test_a_malformed_first_sequence_leaves_the_others_whole(cu, scale):
    """The well-formed sequence behind it is attended to its last token, on the CUDA cores and the tensor cores."""
    g = gen(3)
    T, G, D = 100, 64, 64
    q, k, v = rand(g, T, G, D), rand(g, T, 1, D), rand(g, T, 1, D)
    a = kda.AttnPrefill(q, k, v, torch.tensor(cu).cuda(), scale=scale, o=torch.full_like(q, 7.0)).run()
    assert a.device_status() == 1
    b, e = cu[-2:]
    check(a.o[b:e], *reference(q[b:e], k[b:e], v[b:e], 0, scale, "bf16"))
    assert (a.o[:b] == 7).all()


# ------------------------------------------------------------------ rows by themselves
ROWS = [(3, 64, "bf16"), (5, 128, "bf16"), (12, 128, "bf16"), (20, 64, "bf16"), (33, 128, "bf16"), (90, 32, "bf16"),
        (4, 128, "bf16"), (5, 256, "bf16"), (5, 128, "f32"), (20, 64, "f32"), (5, 256, "f32")]


@pytest.mark.parametrize("G,D,dtype", ROWS)
@pytest.mark.parametrize("paged", [False, True])
def test_same_bits_whatever_ran_before(G, D, dtype, paged):
    """Rows of a tile that no token fills hold what an earlier call left in shared memory: it changes nothing."""
    g = gen(G)
    ctx, new = [700, 90], [120, 31]
    T = sum(new)
    q = rand(g, T, G, D, dtype=dtype)
    if paged:
        p = Pool(ctx, new, 1, D, 32, dtype, 5)
        a = kda.AttnPaged(q, p.k, p.v, p.table, p.lens, cu_of(new).cuda())
    else:
        k, v = rand(g, T, 1, D, dtype=dtype), rand(g, T, 1, D, dtype=dtype)
        a = kda.AttnPrefill(q, k, v, cu_of(new).cuda())
    big = rand(g, 3000, 128, D, dtype=dtype)
    kb = rand(g, 3000, 1, D, dtype=dtype)
    first = a.run().o.clone()
    for fill in (3.0, 40.0, float("nan")):
        kda.attn_prefill(big * fill, kb, kb, cu_of([3000]).cuda())
        assert torch.equal(a.run().o, first)


@pytest.mark.parametrize("G,D,dtype", ROWS)
def test_a_query_changes_its_own_rows_only(G, D, dtype):
    """The other tokens' rows keep their bits, whatever the query of one holds."""
    g = gen(G + 1)
    T, at = 700, 431
    q, k, v = rand(g, T, 2 * G, D, dtype=dtype), rand(g, T, 2, D, dtype=dtype), rand(g, T, 2, D, dtype=dtype)
    cu = cu_of([T]).cuda()
    first = kda.attn_prefill(q, k, v, cu)
    for x in (30.0, float("inf"), float("nan")):
        other = q.clone()
        other[at] *= x
        o = kda.attn_prefill(other, k, v, cu)
        assert torch.equal(o[:at], first[:at]) and torch.equal(o[at + 1:], first[at + 1:])


@pytest.mark.parametrize("G,D,dtype", ROWS)
def test_a_later_key_changes_no_earlier_row(G, D, dtype):
    """Keys past a row's position, NaN among them, leave its bits as they were."""
    g = gen(G + 2)
    T, at = 700, 431
    q, k, v = rand(g, T, 2 * G, D, dtype=dtype), rand(g, T, 2, D, dtype=dtype), rand(g, T, 2, D, dtype=dtype)
    cu = cu_of([T]).cuda()
    first = kda.attn_prefill(q, k, v, cu)
    for x in (30.0, float("inf"), float("nan")):
        other = k.clone()
        other[at] *= x
        o = kda.attn_prefill(q, other, v, cu)
        assert torch.equal(o[:at], first[:at])


@pytest.mark.parametrize("scale", [-0.3, 0.125])
@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 256), ("f32", 128)])
@pytest.mark.parametrize("new", [1, 40])
def test_malformed_requests_without_tokens_are_flagged(new, dtype, D, scale):
    """A row outside the pool, or a length that the table cannot hold, of a request that brings no token."""
    for row, length in ((9, 20), (0, 1 << 40)):
        p = Pool([20, 30], [0, new], 2, D, 16, dtype, 2)
        p.lens[0] = length
        q = rand(gen(1), new, 4, D, dtype=dtype)
        a = kda.AttnPaged(q, p.k, p.v, p.table, p.lens, cu_of([0, new]).cuda(), scale=scale, max_seqlen=new,
                          rows=torch.tensor([row, 1], dtype=torch.int32, device="cuda")).run()
        assert a.device_status() == 32
        check(a.o, *reference(q, p.K[1], p.V[1], 30, scale, dtype))
