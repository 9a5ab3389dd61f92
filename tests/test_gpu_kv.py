"""The paged cache's bookkeeping: pages and slots planned on the GPU, pages
released, new rows written, and the whole serving loop with the attention that
reads them.  Whole numbers and moved values have to be equal.
"""
import pytest
import torch

from linear_attention_serving_delta_gb300 import kda
from test_gpu_attn import DT, check, cu_of, gen, rand, reference

pytestmark = pytest.mark.gpu


def plan_by_hand(cu, T, table, lens, free, count, page, rows):
    """The call's definition, request by request; returns table, slots, lens, count, flags."""
    table, lens = table.clone(), lens.clone()
    R, M = table.shape
    slots = torch.full((T,), -1, dtype=torch.int64)
    flags, before, served, seen = 0, 0, 0, set()
    start = lens.clone()
    for s in range(len(cu) - 1):
        r = s if rows is None else int(rows[s])
        L = int(cu[s + 1]) - int(cu[s])
        if r < 0:
            continue
        if r >= R or r in seen:
            flags |= 32
            continue
        seen.add(r)
        c = int(start[r])
        if c < 0 or c + L > M * page:
            flags |= 32
            continue
        have, want = -(-c // page), -(-(c + L) // page)
        need = want - have
        if need and before + need > count:
            flags |= 64
            before += need
            continue
        for j in range(need):
            table[r, have + j] = free[count - 1 - (before + j)]
        before += need
        served += need
        for i in range(L):
            x = c + i
            slots[int(cu[s]) + i] = int(table[r, x // page]) * page + x % page
        lens[r] = c + L
    return table, slots, lens, count - served, flags


def pool(R, M, page, cached, num, seed):
    g = torch.Generator().manual_seed(seed)
    perm = torch.randperm(num, generator=g).int()
    table = torch.full((R, M), -9, dtype=torch.int32)
    lens = torch.tensor(cached, dtype=torch.int64)
    at = 0
    for r, c in enumerate(cached):
        n = -(-max(c, 0) // page) if c <= M * page else 0
        table[r, :n] = perm[at:at + n]
        at += n
    free = torch.full((num,), -5, dtype=torch.int32)
    free[:num - at] = perm[at:]
    return table, lens, free, num - at


def run_plan(cu, T, table, lens, free, count, page, rows, in_place=False):
    d = [x.cuda() for x in (cu, table, lens, free)]
    cnt = torch.tensor([count], dtype=torch.int32, device="cuda")
    kw = {}
    if not in_place:
        kw = dict(kv_lens_out=d[2].clone(), free_count_out=torch.full_like(cnt, -1))
    r = None if rows is None else rows.cuda()
    p = kda.KvPlan(d[0], T, d[1], d[2], d[3], cnt, page_size=page, rows=r, **kw).run()
    want = plan_by_hand(cu, T, table, lens, free, count, page, rows)
    assert torch.equal(d[1].cpu(), want[0])
    assert torch.equal(p.slot_map.cpu(), want[1])
    assert torch.equal(p.kv_lens_out.cpu(), want[2])
    assert int(p.free_count_out) == want[3]
    assert p.device_status() == want[4]
    assert torch.equal(d[3].cpu(), free)
    if not in_place:
        assert torch.equal(d[2].cpu(), lens) and int(cnt) == count
    return p


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("page", [16, 64, 1024])
@pytest.mark.parametrize("n,new,ctx", [(1, 1, 0), (7, 1, 100), (256, 1, 900), (1500, 2, 300), (5, 400, 50),
                                       (3, 5000, 20), (40, 300, 0), (2100, 3, 64)])
def test_plan(n, new, ctx, page, in_place):
    g = torch.Generator().manual_seed(n + new)
    lens = torch.randint(0, new + 1, (n,), generator=g).tolist()
    cached = torch.randint(0, ctx + 1, (n + 3,), generator=g).tolist()
    M = (ctx + new) // page + 2
    table, kv, free, count = pool(n + 3, M, page, cached, sum(-(-(c + new) // page) for c in cached) + 5, n)
    rows = torch.randperm(n + 3, generator=g)[:n].int()
    run_plan(cu_of(lens), sum(lens), table, kv, free, count, page, rows, in_place)


def test_plan_and_release_in_a_large_pool():
    """More rows than the owners found in shared memory; a row named twice."""
    R, page = 9000, 16
    cached = [i % 40 for i in range(R)]
    table, kv, free, count = pool(R, 5, page, cached, sum(-(-c // page) for c in cached) + 60, 8)
    rows = torch.tensor([8999, 5, 4096, 4095, 5, 8191, 7000], dtype=torch.int32)
    run_plan(cu_of([3, 20, 1, 17, 4, 0, 30]), 75, table, kv, free, count, page, rows, in_place=True)
    d = [x.cuda() for x in (rows, table, kv, free)]
    cnt = torch.tensor([count], dtype=torch.int32, device="cuda")
    assert kda.KvRelease(*d, cnt, page_size=page).run().device_status() == 0
    want = free[:count].tolist()
    for r in (8999, 5, 4096, 4095, 8191, 7000):
        want += table[r, :-(-cached[r] // page)].tolist()
    assert int(cnt) == len(want) and d[3][:len(want)].tolist() == want


def test_plan_without_rows_and_with_padding():
    """Request s is row s; the slot map is longer than the batch's tokens."""
    table, kv, free, count = pool(4, 8, 16, [0, 16, 15, 33], 40, 1)
    run_plan(cu_of([5, 0, 20, 1]), 40, table, kv, free, count, 16, None)
    run_plan(cu_of([5, 0, 20, 1]), 5000, table, kv, free, count, 16, None)


@pytest.mark.parametrize("spare", [0, 1, 2, 3, 5, 9])
def test_plan_when_the_free_list_runs_out(spare):
    """Requests that need no page go on; the first that does not fit and those behind it are refused."""
    cached = [10, 30, 0, 16, 5, 47, 100, 3]
    table, kv, free, count = pool(8, 20, 16, cached, sum(-(-c // 16) for c in cached) + spare, 2)
    run_plan(cu_of([1, 40, 20, 1, 2, 1, 64, 13]), 142, table, kv, free, count, 16, None, in_place=spare % 2 == 0)


def test_plan_of_malformed_requests():
    """Rows outside the pool, rows named twice, skipped rows, lengths that do not fit the table."""
    cached = [10, 30, 0, 16, -4, 1 << 50, 79, 3]
    table, kv, free, count = pool(8, 5, 16, cached, 30, 3)
    rows = torch.tensor([3, 0, 3, -1, 8, 4, 5, 6, 0, 7, -2147483648, 2147483647], dtype=torch.int32)
    run_plan(cu_of([2, 3, 4, 5, 6, 7, 8, 1, 2, 60, 1, 1]), 100, table, kv, free, count, 16, rows)
    run_plan(cu_of([2, 3, 4, 5, 6, 7, 8, 2, 2, 90, 1, 1]), 131, table, kv, free, count, 16, rows, in_place=True)


def test_plan_of_malformed_seqlens():
    table, kv, free, count = pool(3, 8, 16, [0, 20, 5], 30, 4)
    cu = torch.tensor([0, 10, 7, 30])
    d = [x.cuda() for x in (cu, table, kv, free)]
    p = kda.KvPlan(d[0], 30, d[1], d[2], d[3], torch.tensor([count], dtype=torch.int32, device="cuda"),
                   page_size=16).run()
    assert p.device_status() & 1
    assert int(p.kv_lens_out[1]) == 20  # the malformed request advanced nothing


def test_plan_flags_bad_free_pages_and_counts():
    table, kv, free, count = pool(2, 8, 16, [0, 0], 10, 5)
    free[count - 2] = 10  # outside the cache
    d = [x.cuda() for x in (cu_of([16, 16]), table, kv, free)]
    p = kda.KvPlan(d[0], 32, d[1], d[2], d[3], torch.tensor([count], dtype=torch.int32, device="cuda"),
                   page_size=16).run()
    assert p.device_status() == 32 and (p.slot_map[16:] == -1).all() and (p.slot_map[:16] >= 0).all()
    for bad in (-1, 11):
        p = kda.KvPlan(d[0], 32, d[1], torch.zeros(2, dtype=torch.int64, device="cuda"), d[3],
                       torch.tensor([bad], dtype=torch.int32, device="cuda"), page_size=16).run()
        assert p.device_status() == 32 | 64 and (p.slot_map == -1).all()


@pytest.mark.parametrize("M", [1, 5, 1500])
def test_release(M):
    page, R = 16, 1600
    g = torch.Generator().manual_seed(M)
    cached = torch.randint(0, 100, (R,), generator=g).tolist()
    table, kv, free, count = pool(R, 8, page, cached, sum(-(-c // page) for c in cached) + 7, 6)
    rows = torch.randperm(R, generator=g)[:M].int()
    d = [x.cuda() for x in (rows, table, kv, free)]
    cnt = torch.tensor([count], dtype=torch.int32, device="cuda")
    a = kda.KvRelease(*d, cnt, page_size=page).run()
    want, lens = free[:count].tolist(), kv.clone()
    for r in rows.tolist():
        want += table[r, :-(-cached[r] // page)].tolist()
        lens[r] = 0
    assert a.device_status() == 0 and int(cnt) == len(want)
    assert d[3][:len(want)].tolist() == want and torch.equal(d[2].cpu(), lens)


def test_release_of_long_rows():
    # more pages than one pass of the threads takes, next to rows of none and of one
    page, R = 16, 5
    cached = [100_000, 0, 1, 70_000, 16 * 1024]
    table, kv, free, count = pool(R, 6250, page, cached, sum(-(-c // page) for c in cached) + 7, 9)
    rows = torch.tensor([3, 1, 4, 0, 2], dtype=torch.int32)
    d = [x.cuda() for x in (rows, table, kv, free)]
    cnt = torch.tensor([count], dtype=torch.int32, device="cuda")
    a = kda.KvRelease(*d, cnt, page_size=page).run()
    want = free[:count].tolist()
    for r in rows.tolist():
        want += table[r, :-(-cached[r] // page)].tolist()
    assert a.device_status() == 0 and int(cnt) == len(want) and d[2].tolist() == [0] * R
    assert d[3][:len(want)].tolist() == want


def test_release_of_malformed_rows():
    table, kv, free, count = pool(5, 8, 16, [20, 40, 1 << 40, 0, 100], 30, 7)
    rows = torch.tensor([1, -1, 1, 9, 2, 3, 0, 1], dtype=torch.int32)
    d = [x.cuda() for x in (rows, table, kv, free)]
    cnt = torch.tensor([count], dtype=torch.int32, device="cuda")
    a = kda.KvRelease(*d, cnt, page_size=16).run()
    assert a.device_status() == 32
    want = free[:count].tolist() + table[1, :3].tolist() + table[0, :2].tolist()
    assert int(cnt) == len(want) and d[3][:len(want)].tolist() == want
    assert d[2].tolist() == [0, 0, 1 << 40, 0, 100]
    # a free list that cannot hold the pages
    kv2 = torch.tensor([20, 40, 60, 0, 100]).cuda()
    cnt.fill_(26)
    a = kda.KvRelease(d[0][5:], d[1], kv2, d[3], cnt, page_size=16).run()   # rows 3, 0, 1: 0 + 2 + 3 pages
    assert a.device_status() == 32 and int(cnt) == 28 and kv2.tolist() == [0, 40, 60, 0, 100]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,Hkv,D", [(1, 1, 16), (7, 3, 32), (300, 8, 128), (2000, 2, 256), (20000, 1, 64)])
@pytest.mark.parametrize("odd", [False, True])
def test_write(dtype, T, Hkv, D, odd):
    g = gen(T)
    pages = (T * 5 // 4) // 16 + 2
    n = T * Hkv * D

    def make(shape, fill=None):
        total = 1
        for x in shape:
            total *= x
        base = rand(g, total + 1, dtype=dtype) if fill is None else torch.full((total + 1,), fill, device="cuda",
                                                                               dtype=DT[dtype])
        return (base[1:] if odd else base[:total]).view(*shape)

    k, v = make((T, Hkv, D)), make((T, Hkv, D))
    kc, vc = make((pages, 16, Hkv, D), 3.0), make((pages, 16, Hkv, D), 4.0)
    slots = torch.randperm(pages * 16, generator=torch.Generator().manual_seed(T))[:T]
    slots[::7] = -1
    want_k, want_v = kc.clone(), vc.clone()
    keep = (slots >= 0).cuda()
    want_k.view(-1, Hkv, D)[slots.cuda()[keep]] = k[keep]
    want_v.view(-1, Hkv, D)[slots.cuda()[keep]] = v[keep]
    a = kda.KvWrite(k, v, slots.cuda(), kc, vc).run()
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v) and a.device_status() == 0
    if T > 1:
        slots[1] = pages * 16
        slots[T - 1] = 1 << 60
        a = kda.KvWrite(k, v, slots.cuda(), kc, vc).run()
        assert torch.equal(kc, want_k) and torch.equal(vc, want_v) and a.device_status() == 32


@pytest.mark.parametrize("dtype,H,Hkv,D,page", [("bf16", 8, 2, 128, 16), ("bf16", 4, 4, 64, 64), ("f32", 4, 2, 32, 16)])
def test_serving_loop(dtype, H, Hkv, D, page):
    """Prompts in chunks of odd sizes beside decoding requests, everything through plan, write and
    attention; each token's output is that of causal attention over its whole sequence.  One request ends,
    gives its pages back, and another takes its row."""
    g = gen(77)
    totals = [301, 97, 160, 45]
    Q = [rand(g, n, H, D, dtype=dtype) for n in totals]
    K = [rand(g, n, Hkv, D, dtype=dtype) for n in totals]
    V = [rand(g, n, Hkv, D, dtype=dtype) for n in totals]
    want = [reference(Q[i], K[i], V[i], 0, D ** -0.5, dtype) for i in range(4)]
    R, M = 3, -(-301 // page)
    # room for the first three and a little more: the fourth needs released pages
    num = sum(-(-n // page) for n in totals[:3]) + 1
    kc = torch.full((num, page, Hkv, D), float("nan"), device="cuda", dtype=DT[dtype])
    vc = torch.full_like(kc, float("nan"))
    table = torch.full((R, M), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(R, dtype=torch.int64, device="cuda")
    free = torch.arange(num, dtype=torch.int32, device="cuda")
    count = torch.tensor([num], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    steps = [{0: 64, 1: 97}, {0: 130}, {0: 1, 2: 33}, {0: 50, 2: 1}, {2: 100, 0: 55}]
    at = [0, 0, 0, 0]
    row_of = {0: 2, 1: 0, 2: 1}

    def step(batch):
        who = list(batch)
        new = [batch[i] for i in who]
        cu = cu_of(new).cuda()
        rows = torch.tensor([row_of[i] for i in who], dtype=torch.int32, device="cuda")
        part = [slice(at[i], at[i] + batch[i]) for i in who]
        q, k, v = (torch.cat([x[i][p] for i, p in zip(who, part)]) for x in (Q, K, V))
        slots = kda.kv_plan(cu, int(cu[-1]), table, lens, free, count, page_size=page, rows=rows, status=status)
        kda.kv_write(k, v, slots, kc, vc, status=status)
        o = kda.attn_paged(q, kc, vc, table, lens, cu, rows=rows, max_seqlen=max(new), status=status)
        pos = 0
        for i, p, n in zip(who, part, new):
            check(o[pos:pos + n], want[i][0][p], want[i][1][p])
            at[i] += n
            pos += n

    for batch in steps:
        step(batch)
    assert at[0] == 300 and at[1] == 97 and at[2] == 134 and int(status) == 0
    kda.kv_release(torch.tensor([0], dtype=torch.int32, device="cuda"), table, lens, free, count, page_size=page,
                   status=status)
    row_of[3] = 0
    step({3: 44, 0: 1})
    step({3: 1, 2: 26})
    assert int(status) == 0 and lens.tolist() == [45, 160, 301]


def test_decode_loop_in_a_graph():
    """A decode step captured once and replayed: every replay takes the next token of each request."""
    H, Hkv, D, page, N, steps = 8, 2, 128, 16, 5, 40
    g = gen(78)
    start = [0, 15, 31, 100, 7]
    Q, K, V = rand(g, steps, N, H, D), rand(g, N, 200, Hkv, D), rand(g, N, 200, Hkv, D)
    num, M = 80, 12
    kc, vc = (torch.full((num, page, Hkv, D), float("nan"), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    table = torch.full((N, M), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(N, dtype=torch.int64, device="cuda")
    free = torch.randperm(num, generator=torch.Generator().manual_seed(1)).int().cuda()
    count = torch.tensor([num], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu0 = cu_of(start).cuda()
    slots = kda.kv_plan(cu0, sum(start), table, lens, free, count, page_size=page, status=status)
    kda.kv_write(torch.cat([K[i, :n] for i, n in enumerate(start)]), torch.cat([V[i, :n] for i, n in enumerate(start)]),
                 slots, kc, vc, status=status)
    q, k, v = (torch.empty_like(x) for x in (Q[0], K[:, 0].contiguous(), V[:, 0].contiguous()))
    cu = torch.arange(N + 1, device="cuda")
    plan = kda.KvPlan(cu, N, table, lens, free, count, page_size=page, status=status)
    write = kda.KvWrite(k, v, plan.slot_map, kc, vc, status=status)
    attn = kda.AttnPaged(q, kc, vc, table, lens, cu, max_seqlen=1, status=status)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        plan.run()
        write.run()
        attn.run()
    for t in range(steps):
        at = [n + t for n in start]
        q.copy_(Q[t])
        for i in range(N):
            k[i], v[i] = K[i, at[i]], V[i, at[i]]
        graph.replay()
        if t % 13 == 0 or t == steps - 1:
            for i in range(N):
                n = at[i] + 1
                check(attn.o[i:i + 1], *reference(Q[t, i:i + 1], K[i, :n], V[i, :n], at[i], D ** -0.5, "bf16"))
    assert int(status) == 0 and lens.tolist() == [n + steps for n in start]
