"""The paged cache's bookkeeping on malformed batches and full lists: what is
refused leaves every pool entry as it was, what is served is whole.
"""
import pytest
import torch

from linear_attention_serving_delta_gb300 import kda
from test_gpu_attn import cu_of
from test_gpu_kv import plan_by_hand, pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R", [3, 4500])
def test_malformed_seqlens_beside_malformed_rows(R):
    """A request with malformed cu_seqlens whose row lies behind the pool, or is another request's: lengths
    that are written apart from those read get nothing from it, nor does what stands around them."""
    cached = [5 + i % 30 for i in range(R)]
    table, kv, free, count = pool(R, 8, 16, cached, sum(-(-c // 16) for c in cached) + 9, 11)
    # what stands behind (and before) the pool's rows, in the lengths read and in those written
    around = torch.arange(40_000, 40_000 + R + 64)
    lens_in, lens_out = around.clone().cuda(), (around + 100_000).cuda()
    lens_in[32:32 + R] = kv.cuda()
    for row in (R, R + 20, 1):  # (the first request's row is 1)
        before_in, before_out = lens_in.clone(), lens_out.clone()
        cu = torch.tensor([0, 20, 15]).cuda()
        cnt = torch.tensor([count], dtype=torch.int32, device="cuda")
        p = kda.KvPlan(cu, 40, table.cuda(), lens_in[32:32 + R], free.cuda(), cnt, page_size=16,
                       rows=torch.tensor([1, row], dtype=torch.int32, device="cuda"),
                       kv_lens_out=lens_out[32:32 + R], free_count_out=torch.full_like(cnt, -1)).run()
        assert p.device_status() == 1 | 32
        before_out[32 + 1] = cached[1] + 20
        assert torch.equal(lens_in, before_in) and torch.equal(lens_out, before_out)
        assert (p.slot_map[:20] >= 0).all() and (p.slot_map[20:] == -1).all()


@pytest.mark.parametrize("n", [1, 1500])
def test_plan_of_lengths_next_to_64_bits(n):
    """Cached lengths to which no new token can be added within 64 bits: refused as any that the table cannot hold."""
    top = 2 ** 63 - 1
    table, kv, free, count = pool(n + 3, 5, 16, [7] * (n + 3), 2 * n + 20, 12)
    bad = torch.tensor([top, top - 1, 5 * 16 + 1])
    kv[n:] = bad
    cu = cu_of([1] * n + [2, 2, 0])
    T = int(cu[-1])
    d = [x.cuda() for x in (cu, table, kv, free)]
    out = torch.full_like(d[2], -3)
    p = kda.KvPlan(d[0], T, d[1], d[2], d[3], torch.tensor([count], dtype=torch.int32, device="cuda"), page_size=16,
                   kv_lens_out=out).run()
    assert p.device_status() == 32 and int(p.free_count_out) == count
    assert torch.equal(d[1].cpu(), table) and torch.equal(out.cpu(), torch.cat([torch.full((n,), 8), bad]))
    assert (p.slot_map[n:] == -1).all() and (p.slot_map[:n] >= 0).all()


@pytest.mark.parametrize("T", [40, 6000])
@pytest.mark.parametrize("cu,good", [([0, 10, 7, 30], 1), ([0, 20, 5, 8, 30], 1), ([0, 4, 9, 41000, 12, 30], 2),
                                     ([0, 16, 32, 31, 40], 2), ([2, 10, 30], 0), ([0, 18, -3, 20], 1)])
def test_nothing_behind_malformed_seqlens_is_planned(cu, good, T):
    """The first malformed request and those behind it are refused; those before it are served whole."""
    n = len(cu) - 1
    table, kv, free, count = pool(n, 8, 16, [3, 20, 5, 0, 17][:n], 30, 4)
    d = [x.cuda() for x in (torch.tensor(cu), table, kv, free)]
    p = kda.KvPlan(d[0], T, d[1], d[2], d[3], torch.tensor([count], dtype=torch.int32, device="cuda"),
                   page_size=16).run()
    want = plan_by_hand(cu[:good + 1] if good else [0], T, table, kv, free, count, 16, None)
    assert p.device_status() == 1
    assert torch.equal(d[1].cpu(), want[0]) and torch.equal(p.slot_map.cpu(), want[1])
    assert torch.equal(d[2].cpu(), want[2]) and int(p.free_count_out) == want[3]


# ------------------------------------------------------------------ a free list that cannot take every page
def release_by_hand(rows, table, kv, free, count, page):
    free, kv, cap = free[:count].tolist(), kv.clone(), len(free)
    refused = False
    for r in rows:
        n = -(-int(kv[r]) // page)
        if len(free) + n > cap:
            refused = True
            continue
        free += table[r, :n].tolist()
        kv[r] = 0
    return free, kv, refused


@pytest.mark.parametrize("M,room", [(3, 4), (40, 25), (1500, 900), (1500, 3700)])
def test_release_into_a_full_list_takes_every_row_that_fits(M, room):
    page = 16
    g = torch.Generator().manual_seed(M)
    cached = torch.randint(0, 6 * page, (M,), generator=g).tolist()
    cached[0] = 6 * page  # the first row is refused where there is no room for it
    num = sum(-(-c // page) for c in cached) + 40
    table, kv, free, _ = pool(M, 8, page, cached, num, 3)
    count = num - room
    free = torch.where(free < 0, torch.arange(num).int(), free)
    rows = torch.arange(M).int()
    want = release_by_hand(rows.tolist(), table, kv, free, count, page)
    d = [x.cuda() for x in (rows, table, kv, free)]
    cnt = torch.tensor([count], dtype=torch.int32, device="cuda")
    a = kda.KvRelease(*d, cnt, page_size=page).run()
    assert want[2] and a.device_status() == 32
    assert int(cnt) == len(want[0]) and d[3][:len(want[0])].tolist() == want[0] and torch.equal(d[2].cpu(), want[1])
