"""Full attention over packed prompts and over the paged cache, against the
definition in 64 bits.

Tolerances, derived (u = 2^-24, half a step of fp32; h = 2^-8, of bf16).  With
X = max_j scale |q|.|k_j| (products of magnitudes) a logit summed in fp32 is
off by at most d = (D + 4) 2u X, doubled for tensor-core accumulation; a weight then by a factor
e^{2 d}, numerator and denominator both; a sum over n keys by n 2u of
A = sum_j w_j |v_j|.  So |o - o*| <= A (4 d + (n + 16) 2u) in fp32, plus, with
bf16 inputs, h A for the weights and h |o*| for o itself.
"""
import math

import pytest
import torch

from linear_attention_serving_delta_gb300 import kda

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U2 = 2.0 ** -23


def reference(q, k, v, pos0, scale, dtype):
    """o and its tolerance for q [n, H, D] at positions pos0.. over k, v [m, Hkv, D]."""
    n, H, D = q.shape
    m, Hkv = k.shape[:2]
    G = H // Hkv
    qd = q.double().view(n, Hkv, G, D)
    kd, vd = k.double(), v.double()
    if m == 0:
        z = torch.zeros(n, H, D, dtype=torch.float64, device=q.device)
        return z, z
    x = torch.einsum("ihgd,jhd->ihgj", qd, kd) * scale
    seen = torch.arange(m, device=q.device)[None, :] <= torch.arange(pos0, pos0 + n, device=q.device)[:, None]
    x = x.masked_fill(~seen[:, None, None, :], -math.inf)
    w = torch.softmax(x, -1).nan_to_num(0.0)  # rows with no key: zeros
    o = torch.einsum("ihgj,jhd->ihgd", w, vd).reshape(n, H, D)
    mag = (torch.einsum("ihgd,jhd->ihgj", qd.abs(), kd.abs()) * abs(scale)).masked_fill(~seen[:, None, None, :], 0)
    d = (D + 4) * U2 * mag.amax(-1)[..., None]
    A = torch.einsum("ihgj,jhd->ihgd", w, vd.abs())
    tol = (A * (4 * d + (m + 16) * U2)).reshape(n, H, D) + 1e-30
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * (A.reshape(n, H, D) + o.abs())
    return o, tol


def check(o, ref, tol):
    assert not torch.isnan(o).any()
    bad = (o.double() - ref).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} off, worst {float(((o.double() - ref).abs() / tol).max()):.3f} of tolerance"


def rand(g, *shape, dtype="bf16"):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(DT[dtype])


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def cu_of(lens):
    return torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int64)


# ------------------------------------------------------------------ prompts
LENS = [[1], [64], [65, 1, 0, 130], [257, 3, 127, 128, 129], [700, 33]]


def run_prompt(lens, H, Hkv, D, dtype, seed=0, scale=None, sharp=1.0):
    g = gen(seed)
    T = sum(lens)
    q, k, v = rand(g, T, H, D, dtype=dtype) * sharp, rand(g, T, Hkv, D, dtype=dtype), rand(g, T, Hkv, D, dtype=dtype)
    cu = cu_of(lens)
    a = kda.AttnPrefill(q, k, v, cu.cuda(), scale=scale)
    a.run()
    scale = D ** -0.5 if scale is None else scale
    for s in range(len(lens)):
        b, e = int(cu[s]), int(cu[s + 1])
        if b < e:
            check(a.o[b:e], *reference(q[b:e], k[b:e], v[b:e], 0, scale, dtype))
    assert a.device_status() == 0
    return a


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("H,Hkv,D,dtype", [(4, 4, 64, "bf16"), (8, 2, 128, "bf16"), (6, 1, 128, "bf16"),
                                           (10, 2, 64, "bf16"), (4, 2, 32, "bf16"), (2, 1, 16, "bf16"),
                                           (4, 2, 256, "bf16"), (4, 4, 64, "f32"), (8, 2, 128, "f32"),
                                           (3, 1, 256, "f32"), (14, 2, 16, "f32")])
def test_prompts(lens, H, Hkv, D, dtype):
    run_prompt(lens, H, Hkv, D, dtype, seed=len(lens) + H)


@pytest.mark.parametrize("G", [1, 2, 3, 5, 7, 12, 33, 64, 65, 100, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_group_size(G, dtype):
    run_prompt([70, 5], 2 * G, 2, 64, dtype, seed=G)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale,sharp", [(0.0, 1.0), (-0.3, 1.0), (1.0, 4.0), (0.125, 30.0)])
def test_scales_and_sharp_rows(dtype, scale, sharp):
    """Constant logits, a negative scale, and rows whose maximum keeps moving."""
    run_prompt([300, 40], 4, 2, 64, dtype, seed=3, scale=scale, sharp=sharp)


@pytest.mark.parametrize("D,H,Hkv,dtype", [(128, 8, 2, "bf16"), (64, 4, 4, "bf16"), (256, 6, 2, "bf16"),
                                           (128, 8, 2, "f32"), (64, 4, 4, "f32"), (32, 8, 2, "f32"), (256, 6, 2, "f32")])
def test_longer_prompts(D, H, Hkv, dtype):
    run_prompt([2500, 1111], H, Hkv, D, dtype, seed=9)


@pytest.mark.parametrize("D,dtype", [(128, "bf16"), (256, "bf16"), (64, "f32")])
def test_many_short_prompts(D, dtype):
    """More sequences than a CTA plans at once, among them empty ones."""
    lens = [(7 * i) % 5 for i in range(1300)]
    run_prompt(lens, 4, 2, D, dtype, seed=10)


def test_rising_logits():
    """Every key tile raises the running maximum by far: the rescaling of what was accumulated."""
    T, H, D = 1300, 2, 64
    g = gen(5)
    q = torch.ones(T, H, D, device="cuda", dtype=torch.bfloat16)
    k = (torch.arange(T, device="cuda").float() / 24).round()[:, None, None].expand(T, H, D).bfloat16().contiguous()
    v = rand(g, T, H, D)
    o = kda.attn_prefill(q, k, v, cu_of([T]).cuda(), scale=0.125)
    check(o, *reference(q, k, v, 0, 0.125, "bf16"))
    o = kda.attn_prefill(q, k.flip(0).contiguous(), v, cu_of([T]).cuda(), scale=0.125)
    check(o, *reference(q, k.flip(0), v, 0, 0.125, "bf16"))


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_rows_behind_the_last_sequence_stay(dtype, D):
    g = gen(1)
    T, used = 300, [100, 33]
    q, k, v = rand(g, T, 4, D, dtype=dtype), rand(g, T, 2, D, dtype=dtype), rand(g, T, 2, D, dtype=dtype)
    k[sum(used):] = float("nan")
    v[sum(used):] = float("inf")
    o = torch.full_like(q, 7.0)
    kda.attn_prefill(q, k, v, cu_of(used).cuda(), o=o)
    assert (o[sum(used):] == 7).all()
    check(o[100:133], *reference(q[100:133], k[100:133], v[100:133], 0, D ** -0.5, dtype))


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("bf16", 256), ("f32", 128)])
def test_a_neighbour_with_infinities_changes_nothing(dtype, D):
    """A sequence of NaN and infinities between two others."""
    g = gen(2)
    lens = [77, 50, 90]
    T = sum(lens)
    q, k, v = rand(g, T, 4, D, dtype=dtype), rand(g, T, 2, D, dtype=dtype), rand(g, T, 2, D, dtype=dtype)
    k[77:127] = float("nan")
    v[77:127:2] = float("inf")
    v[78:127:2] = float("nan")
    o = kda.attn_prefill(q, k, v, cu_of(lens).cuda())
    for b, e in ((0, 77), (127, 217)):
        check(o[b:e], *reference(q[b:e], k[b:e], v[b:e], 0, D ** -0.5, dtype))


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("bf16", 256), ("f32", 128), ("f32", 256)])
@pytest.mark.parametrize("at", [0, 5, 100, 299])
def test_later_tokens_never_reach_earlier_rows(dtype, D, at):
    """Infinities and NaN from position `at` on: the rows before it are as they were."""
    g = gen(4)
    T = 300
    q, k, v = rand(g, T, 8, D, dtype=dtype), rand(g, T, 2, D, dtype=dtype), rand(g, T, 2, D, dtype=dtype)
    clean = kda.attn_prefill(q, k, v, cu_of([T]).cuda())
    v[at] = float("inf")
    v[at + 1:] = float("nan")
    k[at + 2:] = float("nan")
    o = kda.attn_prefill(q, k, v, cu_of([T]).cuda())
    check(o[:at], *reference(q[:at], k[:at], v[:at], 0, D ** -0.5, dtype))
    assert torch.equal(o[:at], clean[:at])
    assert not torch.isfinite(o[at:].float()).any()


def test_unaligned_tensors():
    """Bases that are only element-aligned."""
    g = gen(6)
    T, H, Hkv, D = 150, 4, 2, 64
    for dtype in ("bf16", "f32"):
        def odd(*shape):
            n = math.prod(shape)
            return rand(g, n + 1, dtype=dtype)[1:].view(*shape)
        q, k, v = odd(T, H, D), odd(T, Hkv, D), odd(T, Hkv, D)
        out = torch.empty(T * H * D + 1, device="cuda", dtype=DT[dtype])[1:].view(T, H, D)
        kda.attn_prefill(q, k, v, cu_of([T]).cuda(), o=out)
        check(out, *reference(q, k, v, 0, D ** -0.5, dtype))


def test_malformed_seqlens_are_flagged():
    g = gen(7)
    for D in (64, 128):
        q, k = rand(g, 100, 4, D), rand(g, 100, 2, D)
        for cu in ([0, 50, 120], [0, 60, 40], [3, 50, 100], [0, -5, 100]):
            a = kda.AttnPrefill(q, k, k, torch.tensor(cu).cuda())
            a.run()
            assert a.device_status() & 1
        a = kda.AttnPrefill(q, k, k, torch.tensor([0, 50, 120]).cuda(), o=torch.full_like(q, 3.0)).run()
        check(a.o[:50], *reference(q[:50], k[:50], k[:50], 0, D ** -0.5, "bf16"))
        assert (a.o[50:] == 3).all()


# ------------------------------------------------------------------ the paged cache
class Pool:
    """Caches of NaN, pages handed out in a shuffled order."""

    def __init__(self, ctx, new, Hkv, D, page, dtype, seed, spare=3, rows=None):
        g = gen(seed)
        self.page, self.dtype = page, dtype
        n = [c + l for c, l in zip(ctx, new)]
        need = [-(-x // page) for x in n]
        num = sum(need) + spare
        perm = torch.randperm(num, generator=torch.Generator().manual_seed(seed)).int()
        self.rows = list(range(len(n))) if rows is None else rows
        R = max(self.rows) + 2
        # entries behind a request's pages are never read
        table = torch.full((R, max(need) + 2), -(1 << 30), dtype=torch.int32)
        table[:, 1::2] = 1 << 30
        lens = torch.zeros(R, dtype=torch.int64)
        self.k = torch.full((num, page, Hkv, D), float("nan"), device="cuda", dtype=DT[dtype])
        self.v = torch.full_like(self.k, float("inf"))
        self.K, self.V = [], []
        at = 0
        for i, x in enumerate(n):
            table[self.rows[i], :need[i]] = perm[at:at + need[i]]
            at += need[i]
            lens[self.rows[i]] = x
            K, V = rand(g, x, Hkv, D, dtype=dtype), rand(g, x, Hkv, D, dtype=dtype)
            where = torch.arange(x)
            slot = (table[self.rows[i]].long()[where // page] * page + where % page).cuda()
            self.k.view(-1, Hkv, D)[slot] = K
            self.v.view(-1, Hkv, D)[slot] = V
            self.K.append(K)
            self.V.append(V)
        self.table, self.lens = table.cuda(), lens.cuda()


def run_paged(ctx, new, H, Hkv, D, page, dtype, seed=0, rows=None, max_seqlen=None, scale=None):
    p = Pool(ctx, new, Hkv, D, page, dtype, seed, rows=rows)
    g = gen(seed + 100)
    cu = cu_of(new)
    q = rand(g, int(cu[-1]), H, D, dtype=dtype)
    r = None if rows is None else torch.tensor(rows, dtype=torch.int32, device="cuda")
    a = kda.AttnPaged(q, p.k, p.v, p.table, p.lens, cu.cuda(), rows=r, scale=scale,
                      max_seqlen=max(new) if max_seqlen is None else max_seqlen)
    a.run()
    assert a.device_status() == 0
    scale = D ** -0.5 if scale is None else scale
    for i in range(len(new)):
        b, e = int(cu[i]), int(cu[i + 1])
        if b < e:
            check(a.o[b:e], *reference(q[b:e], p.K[i], p.V[i], ctx[i], scale, dtype))
    return a


SHAPES = [(8, 2, 128, "bf16"), (4, 4, 64, "bf16"), (12, 2, 128, "bf16"), (16, 1, 64, "bf16"), (5, 1, 128, "bf16"),
          (4, 2, 32, "bf16"), (8, 2, 256, "bf16"), (8, 2, 128, "f32"), (4, 4, 64, "f32"), (3, 1, 256, "f32"),
          (40, 1, 64, "bf16"), (2, 2, 16, "f32")]


@pytest.mark.parametrize("H,Hkv,D,dtype", SHAPES)
@pytest.mark.parametrize("page", [16, 64, 256])
def test_single_tokens(H, Hkv, D, dtype, page):
    run_paged([0, 1, 15, 16, 17, 63, 64, 127, 128, 129, 500, 1024], [1] * 12, H, Hkv, D, page, dtype, seed=page + H)


@pytest.mark.parametrize("H,Hkv,D,dtype", SHAPES)
@pytest.mark.parametrize("ctx,new", [([0, 30, 200], [1, 5, 3]), ([100, 0, 31, 64], [64, 40, 1, 129]),
                                     ([0], [300]), ([1000, 3], [17, 0])])
def test_chunks(H, Hkv, D, dtype, ctx, new):
    run_paged(ctx, new, H, Hkv, D, 32, dtype, seed=sum(new) + D)


@pytest.mark.parametrize("page", [16, 32, 128, 512, 1024])
@pytest.mark.parametrize("new", [1, 2, 4, 9, 33])
def test_long_contexts_of_few_requests(page, new):
    """Few rows over long contexts: the work of a row is cut along its keys."""
    run_paged([5000, 777], [new, 1], 8, 2, 128, page, "bf16", seed=page + new)
    run_paged([4097], [new], 4, 1, 64, page, "bf16", seed=page + new)
    run_paged([2000], [new], 4, 2, 64, page, "f32", seed=page + new)
    run_paged([3000, 100], [new, new], 8, 2, 256, page, "bf16", seed=page + new)
    run_paged([1500, 900], [new, 1], 8, 2, 128, page, "f32", seed=page + new)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 256), ("f32", 128), ("f32", 256)])
def test_a_chunk_beside_decoding_requests(dtype, D):
    run_paged([3000, 17, 900, 2500, 0, 64], [200, 1, 1, 1, 1, 3], 8, 2, D, 32, dtype, seed=D)


@pytest.mark.parametrize("dtype,D,new", [("bf16", 128, 1), ("bf16", 64, 1), ("f32", 64, 1), ("f32", 64, 20)])
def test_many_requests(dtype, D, new):
    """More requests than a CTA plans at once, with skipped and empty ones between."""
    n = 700
    ctx = [(13 * i) % 90 for i in range(n)]
    lens = [0 if i % 7 == 3 else 1 + i % new for i in range(n)]
    run_paged(ctx, lens, 4, 2, D, 16, dtype, seed=new)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_of_the_pool(dtype):
    run_paged([30, 100, 7, 64], [1, 1, 1, 1], 8, 2, 64, 16, dtype, rows=[6, 0, 3, 9])
    run_paged([30, 100, 7, 64], [4, 50, 1, 7], 8, 2, 128, 16, dtype, rows=[6, 0, 3, 9])


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("f32", 64)])
@pytest.mark.parametrize("new", [1, 40])
def test_skipped_and_malformed_requests(dtype, D, new):
    p = Pool([50, 60, 70, 80, 90], [new] * 5, 2, D, 16, dtype, 3)
    g = gen(8)
    q = rand(g, 5 * new, 4, D, dtype=dtype)
    cu = cu_of([new] * 5).cuda()
    rows = torch.tensor([0, -1, 2, 99, 4], dtype=torch.int32, device="cuda")
    p.lens[2] = 1 << 40
    o = torch.full_like(q, 5.0)
    a = kda.AttnPaged(q, p.k, p.v, p.table, p.lens, cu, rows=rows, o=o, max_seqlen=new).run()
    assert a.device_status() == 32
    for i in range(5):
        mine = o[i * new:(i + 1) * new]
        if i in (0, 4):
            x = q[i * new:(i + 1) * new]
            check(mine, *reference(x, p.K[i], p.V[i], [50, 60, 70, 80, 90][i], D ** -0.5, dtype))
        else:
            assert (mine == 5).all()
    # longer than announced
    if new > 1:
        b = kda.AttnPaged(q, p.k, p.v, p.table, p.lens, cu, rows=rows, max_seqlen=1).run()
        assert b.device_status() == 128


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("f32", 64)])
@pytest.mark.parametrize("new", [1, 40])
def test_pages_outside_the_cache_read_as_zeros(dtype, D, new):
    ctx = [200, 40]
    p = Pool(ctx, [new, new], 2, D, 32, dtype, 4)
    q = rand(gen(9), 2 * new, 4, D, dtype=dtype)
    p.table[0, 1], p.table[0, 3] = -1, p.k.shape[0]
    for page in (1, 3):
        p.K[0][32 * page:32 * page + 32] = 0
        p.V[0][32 * page:32 * page + 32] = 0
    a = kda.AttnPaged(q, p.k, p.v, p.table, p.lens, cu_of([new, new]).cuda(), max_seqlen=new).run()
    assert a.device_status() == 32
    for i in range(2):
        check(a.o[i * new:(i + 1) * new], *reference(q[i * new:(i + 1) * new], p.K[i], p.V[i], ctx[i], D ** -0.5, dtype))


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("bf16", 256), ("f32", 64)])
def test_rows_before_the_first_position_are_zero(dtype, D):
    """More new tokens than cached positions: the first rows attend nothing."""
    new, have = [50, 3, 20], [30, 0, 20]
    p = Pool([0, 0, 0], have, 2, D, 16, dtype, 5)
    q = rand(gen(10), sum(new), 4, D, dtype=dtype)
    cu = cu_of(new)
    a = kda.AttnPaged(q, p.k, p.v, p.table, p.lens, cu.cuda()).run()
    assert a.device_status() == 0
    for i in range(3):
        b, e = int(cu[i]), int(cu[i + 1])
        dead = new[i] - have[i]
        assert (a.o[b:b + dead] == 0).all()
        if have[i]:
            check(a.o[b + dead:e], *reference(q[b + dead:e], p.K[i], p.V[i], 0, D ** -0.5, dtype))


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 64), ("f32", 128), ("f32", 256)])
@pytest.mark.parametrize("new", [3, 60])
def test_infinite_values_reach_the_rows_that_attend_them(dtype, D, new):
    """One infinite value, and one NaN, in the cache: their channels in the rows from there on, nothing else."""
    ctx = 150
    p = Pool([ctx], [new], 2, D, 16, dtype, 6)
    q = rand(gen(12), new, 4, D, dtype=dtype)
    cu = cu_of([new]).cuda()

    def put(x, head, c, value):
        page, off = int(p.table[0, x // 16]), x % 16
        p.v[page, off, head, c] = value

    put(ctx + 1, 0, 5, float("inf"))       # among the new tokens
    put(ctx + new - 1, 1, 7, float("nan"))
    p.V[0][ctx + 1, 0, 5] = 0
    p.V[0][ctx + new - 1, 1, 7] = 0
    a = kda.AttnPaged(q, p.k, p.v, p.table, p.lens, cu, max_seqlen=new).run()
    ref, tol = reference(q, p.K[0], p.V[0], ctx, D ** -0.5, dtype)
    o = a.o.clone()
    assert torch.isposinf(o[1:, 0:2, 5]).all() and torch.isfinite(o[0, 0:2, 5]).all()
    assert torch.isnan(o[-1, 2:4, 7]).all() and torch.isfinite(o[:-1, 2:4, 7]).all()
    o[1:, 0:2, 5], o[-1, 2:4, 7] = 0, 0
    tol[1:, 0:2, 5], tol[-1, 2:4, 7] = 1e9, 1e9
    check(o, ref, tol)


@pytest.mark.parametrize("G", [16, 17, 20, 33, 40, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_group_sizes_of_wide_heads(G, dtype):
    """A token's group of heads cut into blocks of 16 or 32 rows."""
    run_prompt([40, 3], G, 1, 256, dtype, seed=G)
    run_paged([100, 7, 900], [1, 1, 1], 2 * G, 2, 256, 16, dtype, seed=G)
    run_paged([100, 7, 900], [1, 2, 1], G, 1, 64, 16, dtype, seed=G)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.0, -0.2, 1e-6])
@pytest.mark.parametrize("new", [1, 30])
def test_scales_over_the_cache(dtype, scale, new):
    run_paged([300, 20], [new, 1], 8, 2, 64, 16, dtype, seed=new, scale=scale)


@pytest.mark.parametrize("bound", [40, 1 << 31, (1 << 32) + 1])
def test_a_loose_bound_on_the_new_tokens(bound):
    run_paged([30, 500], [3, 40], 8, 2, 64, 16, "bf16", seed=5, max_seqlen=bound)


def test_unaligned_cache():
    g = gen(13)
    p = Pool([200, 31], [3, 20], 2, 64, 16, "bf16", 14)
    k = torch.empty(p.k.numel() + 1, device="cuda", dtype=torch.bfloat16)[1:].view(p.k.shape).copy_(p.k)
    v = torch.empty(p.v.numel() + 1, device="cuda", dtype=torch.bfloat16)[1:].view(p.v.shape).copy_(p.v)
    q = rand(g, 23, 8, 64)
    o = kda.attn_paged(q, k, v, p.table, p.lens, cu_of([3, 20]).cuda())
    check(o[:3], *reference(q[:3], p.K[0], p.V[0], 200, 0.125, "bf16"))
    check(o[3:], *reference(q[3:], p.K[1], p.V[1], 31, 0.125, "bf16"))


def test_prompts_in_a_graph():
    """A captured call follows its inputs, lengths among them."""
    for D, dtype in ((64, "bf16"), (128, "bf16"), (256, "bf16"), (64, "f32")):
        g = gen(15)
        T = 900
        q, k, v = rand(g, T, 8, D, dtype=dtype), rand(g, T, 2, D, dtype=dtype), rand(g, T, 2, D, dtype=dtype)
        cu = cu_of([300, 500]).cuda()
        a = kda.AttnPrefill(q, k, v, cu)
        a.run()
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            a.run()
        for lens in ([300, 500], [1, 899], [450, 450], [0, 10]):
            cu.copy_(cu_of(lens))
            v.copy_(rand(g, T, 2, D, dtype=dtype))
            a.o.fill_(9)
            graph.replay()
            b = lens[0]
            for x, y in ((0, b), (b, b + lens[1])):
                if x < y:
                    check(a.o[x:y], *reference(q[x:y], k[x:y], v[x:y], 0, D ** -0.5, dtype))
            assert (a.o[sum(lens):] == 9).all()


def test_slots_past_32_bit_offsets():
    """A cache of more than 2^32 elements, pages at its far end."""
    Hkv, D, page = 8, 128, 64
    pages = (1 << 32) // (page * Hkv * D) + 100
    k = torch.empty(pages, page, Hkv, D, device="cuda", dtype=torch.bfloat16)
    v = torch.empty_like(k)
    g = gen(11)
    table = torch.tensor([[pages - 1, 0, pages - 2, 5, pages - 50]], dtype=torch.int32)
    n = 300
    K, V = rand(g, n, Hkv, D), rand(g, n, Hkv, D)
    where = torch.arange(n)
    slot = (table[0].long()[where // page] * page + where % page).cuda()
    st = kda.KvWrite(K, V, slot, k, v).run()
    assert st.device_status() == 0
    for new in (1, 100):
        q = rand(g, new, 16, D)
        a = kda.AttnPaged(q, k, v, table.cuda(), torch.tensor([n], device="cuda"), cu_of([new]).cuda()).run()
        check(a.o, *reference(q, K, V, n - new, D ** -0.5, "bf16"))


def test_same_call_gives_the_same_bits():
    a = run_paged([3000, 100, 900], [1, 1, 1], 8, 2, 128, 16, "bf16", seed=21)
    first = a.o.clone()
    b = run_prompt([900, 200], 8, 2, 128, "bf16", seed=22)
    second = b.o.clone()
    for _ in range(5):
        assert torch.equal(a.run().o, first) and torch.equal(b.run().o, second)


def test_another_stream_and_two_calls_at_once():
    """Two planned calls with their own workspaces, in flight together on two streams."""
    p = Pool([4000, 300], [1, 1], 2, 128, 16, "bf16", 31)
    q1, q2 = rand(gen(1), 2, 8, 128), rand(gen(2), 2, 8, 128)
    cu = cu_of([1, 1]).cuda()
    a = kda.AttnPaged(q1, p.k, p.v, p.table, p.lens, cu, max_seqlen=1)
    b = kda.AttnPaged(q2, p.k, p.v, p.table, p.lens, cu, max_seqlen=1)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        a.run(s1)
        b.run(s2)
    torch.cuda.synchronize()
    for i in range(2):
        check(a.o[i:i + 1], *reference(q1[i:i + 1], p.K[i], p.V[i], [4000, 300][i], 128 ** -0.5, "bf16"))
        check(b.o[i:i + 1], *reference(q2[i:i + 1], p.K[i], p.V[i], [4000, 300][i], 128 ** -0.5, "bf16"))
    o = kda.attn_paged(q1, p.k, p.v, p.table, p.lens, cu, max_seqlen=1, stream=s1)
    torch.cuda.synchronize()
    assert torch.equal(o, a.o)


def test_empty_calls():
    q, k = torch.empty(0, 4, 64, device="cuda", dtype=torch.bfloat16), torch.empty(0, 2, 64, device="cuda",
                                                                                  dtype=torch.bfloat16)
    assert kda.attn_prefill(q, k, k, torch.zeros(2, dtype=torch.int64, device="cuda")).shape == (0, 4, 64)
    p = Pool([10], [0], 2, 64, 16, "bf16", 0)
    kda.attn_paged(q, p.k, p.v, p.table, p.lens, torch.zeros(2, dtype=torch.int64, device="cuda"))
    torch.cuda.synchronize()
