"""The full-attention operators and their paged cache, as workloads to measure.

Four operators: the block tables and slot maps of a batch of requests
(``plan``), the write of new keys and values into the cache (``write``),
causal attention over packed prompts (``prompt``) and attention of new tokens
over the paged cache (``paged``).  ``run`` computes each in a plain form from
elementary torch operations, or, with ``own`` set, through the package.
"""
import math

import torch

own = False

HEADS = [(32, 8), (16, 16), (8, 1), (24, 4), (20, 4), (8, 8), (64, 8), (16, 2), (32, 32)]
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one decode step's plan: 256 running requests, one new token each, small pages
        dict(name="plan_decode_256", op="plan", n=256, lo=1, hi=1, ctx_lo=0, ctx_hi=8191, page=16),
        # the plan of eight prompts of 1k..32k tokens arriving together
        dict(name="plan_prompts_8", op="plan", n=8, lo=1024, hi=32768, uniform=True, ctx_lo=0, ctx_hi=0, page=64),
        # the new keys and values of a decode step of 256 rows
        dict(name="write_decode_256", op="write", t=256, hkv=8, d=128, dtype="bf16"),
        # those of the eight prompts
        dict(name="write_prompts", op="write", t=110353, hkv=8, d=128, dtype="bf16"),
        # a handful of short chat turns, where latency counts
        dict(name="prompt_short_ragged", op="prompt", n=5, lo=1, hi=200, hq=8, hkv=2, d=64, dtype="bf16"),
        # one long prompt
        dict(name="prompt_8k", op="prompt", n=1, lo=8192, hi=8192, hq=32, hkv=8, d=128, dtype="bf16"),
        # eight packed prompts of very different lengths: the largest case
        dict(name="prompt_varlen_8", op="prompt", n=8, lo=1024, hi=32768, uniform=True, hq=32, hkv=8, d=128,
             dtype="bf16"),
        # full-precision check runs of a small model, a key head per query head
        dict(name="prompt_f32", op="prompt", n=2, lo=500, hi=1500, hq=8, hkv=8, d=64, dtype="f32"),
        # one user deep in a long document: a single token over 128k cached ones
        dict(name="decode_1_long", op="paged", n=1, lo=1, hi=1, ctx_lo=131071, ctx_hi=131071, chunk=0, hq=32,
             hkv=8, d=128, page=64, dtype="bf16"),
        # a full decode batch with contexts of all lengths
        dict(name="decode_256", op="paged", n=256, lo=1, hi=1, ctx_lo=64, ctx_hi=8191, chunk=0, hq=32, hkv=8,
             d=128, page=16, dtype="bf16"),
        # chunked prefill: a 512-token piece of a long prompt beside eight decoding requests
        dict(name="chunk_512_mixed", op="paged", n=9, lo=1, hi=1, ctx_lo=1000, ctx_hi=32000, chunk=512, hq=32,
             hkv=8, d=128, page=32, dtype="bf16"),
        # a small full-precision batch with a few tokens each, odd lengths
        dict(name="paged_f32", op="paged", n=7, lo=1, hi=5, ctx_lo=0, ctx_hi=2001, chunk=0, hq=16, hkv=4, d=64,
             page=16, dtype="f32"),
    ]


def _logint(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    op = rng.choice(["plan", "write", "prompt", "prompt", "paged", "paged", "paged"])
    if op == "plan":
        if rng.random() < 0.5:
            return dict(op=op, n=_logint(rng, 1, 1500), lo=1, hi=rng.choice([1, 1, 4]), ctx_lo=0,
                        ctx_hi=_logint(rng, 30, 9000), page=rng.choice([16, 32, 64, 128]))
        hi = _logint(rng, 40, 32768)
        return dict(op=op, n=_logint(rng, 1, 40), lo=max(1, hi // 30), hi=hi, ctx_lo=0,
                    ctx_hi=_logint(rng, 1, 5000), page=rng.choice([16, 32, 64, 128]))
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = rng.choice([32, 64, 64, 128, 128, 128, 256])
    if op == "write":
        return dict(op=op, t=_logint(rng, 1, 60000), hkv=rng.choice([1, 2, 4, 8]), d=d, dtype=dtype)
    hq, hkv = rng.choice(HEADS)
    if op == "prompt":
        n = _logint(rng, 1, 24)
        top = 16000 if dtype == "bf16" and d <= 128 else 5000
        hi = _logint(rng, 2, max(4, int(top / math.sqrt(n * hq / 16))))
        return dict(op=op, n=n, lo=max(1, hi // 20), hi=hi, hq=hq, hkv=hkv, d=d, dtype=dtype)
    n = _logint(rng, 1, 200)
    size = 2.0 * hkv * d * (2 if dtype == "bf16" else 4)  # bytes of a cached token
    hi = _logint(rng, 2, max(4, min(60000, int(3.5e9 / size / n))))
    new = rng.choice([1, 1, 1, 3, 8, 40])
    chunk = rng.choice([0, 0, _logint(rng, 2, 1000)])
    return dict(op=op, n=n, lo=1, hi=new, ctx_lo=hi // 50, ctx_hi=hi, chunk=chunk, hq=hq, hkv=hkv, d=d,
                page=rng.choice([16, 32, 64, 128]), dtype=dtype)


def _lens(case, seed):
    """New tokens and cached tokens of each request, on the host: the same lengths for every seed, in another
    order, so that the sizes of a case stay its own."""
    g = torch.Generator().manual_seed(17)
    n, lo, hi = case["n"], case["lo"], case["hi"]
    if hi >= 8 * lo and not case.get("uniform"):  # a wide range, spread over its logarithm
        new = (lo * torch.exp(torch.rand(n, generator=g, dtype=torch.float64) * math.log((hi + 0.49) / lo))).long()
    else:
        new = torch.randint(lo, hi + 1, (n,), generator=g)
    new = new.clamp(lo, hi)
    ctx = torch.zeros(n, dtype=torch.int64)
    if "ctx_hi" in case:
        ctx = torch.randint(case["ctx_lo"], case["ctx_hi"] + 1, (n,), generator=g)
    if case.get("chunk"):
        new[0] = case["chunk"]
        ctx[0] = case["ctx_hi"]
    order = torch.randperm(n, generator=torch.Generator().manual_seed(seed + 1))
    return new[order], ctx[order]


def _work_lens(case):
    new, ctx = _lens(case, 0)
    return new.double(), ctx.double()


def _cu(new):
    cu = torch.zeros(new.numel() + 1, dtype=torch.int64)
    cu[1:] = new.cumsum(0)
    return cu


def _pages(case, seed, new, ctx, spare):
    """A pool of shuffled pages: the table of what is cached, and the free ones."""
    g = torch.Generator().manual_seed(seed * 7919 + 3)
    p, n = case["page"], new.numel()
    have = (ctx + p - 1) // p
    total = (ctx + new + p - 1) // p
    num = int(total.sum()) + spare
    perm = torch.randperm(num, generator=g).int()
    width = int(total.max()) + 2
    return have, total, num, perm, width


def _inputs(case, seed):
    dev = "cuda"
    op = case["op"]
    g = torch.Generator(device=dev).manual_seed(seed * 104729 + 11)

    def rand(*shape):
        x = torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)
        return x.to(DT[case["dtype"]])

    st = dict(op=op, case=case)
    if op == "write":
        t, hkv, d = case["t"], case["hkv"], case["d"]
        slots = t + t // 2 + 64
        hg = torch.Generator().manual_seed(seed + 5)
        smap = torch.randperm(slots, generator=hg)[:t]
        smap[torch.rand(t, generator=hg) < 0.02] = -1  # padding tokens of the batch
        # the cache is laid out in pages of 16 tokens
        pages = (slots + 15) // 16
        st.update(k=rand(t, hkv, d), v=rand(t, hkv, d), slot_map=smap.to(dev),
                  k_cache=torch.zeros(pages, 16, hkv, d, device=dev, dtype=DT[case["dtype"]]),
                  v_cache=torch.zeros(pages, 16, hkv, d, device=dev, dtype=DT[case["dtype"]]))
    elif op == "plan":
        new, ctx = _lens(case, seed)
        cu = _cu(new)
        have, total, num, perm, width = _pages(case, seed, new, ctx, 40)
        rows_n = case["n"] + 9
        hg = torch.Generator().manual_seed(seed + 6)
        rows = torch.randperm(rows_n, generator=hg)[:case["n"]].int()
        table = torch.full((rows_n, width), -1, dtype=torch.int32)
        lens = torch.zeros(rows_n, dtype=torch.int64)
        at = 0
        for s in range(case["n"]):
            h = int(have[s])
            table[rows[s], :h] = perm[at:at + h]
            lens[rows[s]] = ctx[s]
            at += h
        free = torch.full((num,), -1, dtype=torch.int32)
        free[:num - at] = perm[at:]
        st.update(cu=cu.to(dev), T=int(cu[-1]), table=table.to(dev), lens=lens.to(dev), rows=rows.to(dev),
                  free=free.to(dev), count=torch.tensor([num - at], dtype=torch.int32, device=dev),
                  page=case["page"], lens_out=lens.to(dev), count_out=torch.zeros(1, dtype=torch.int32, device=dev))
    else:
        new, ctx = _lens(case, seed)
        cu = _cu(new)
        T, hq, hkv, d = int(cu[-1]), case["hq"], case["hkv"], case["d"]
        st.update(cu=cu.to(dev), host_cu=cu.tolist(), scale=1.0 / math.sqrt(d), q=rand(T, hq, d))
        # some heads attend sharply, others broadly
        st["q"] *= torch.linspace(0.5, 2.5, hq, device=dev).to(st["q"].dtype)[None, :, None]
        if op == "prompt":
            st.update(k=rand(T, hkv, d), v=rand(T, hkv, d))
        else:
            have, total, num, perm, width = _pages(case, seed, new, ctx, 3)
            table = torch.zeros(case["n"], width, dtype=torch.int32)
            at = 0
            for s in range(case["n"]):
                n_p = int(total[s])
                table[s, :n_p] = perm[at:at + n_p]
                at += n_p
            lens = ctx + new
            st.update(k_cache=rand(num, case["page"], hkv, d), v_cache=rand(num, case["page"], hkv, d),
                      table=table.to(dev), lens=lens.to(dev), host_lens=lens.tolist(),
                      max_new=int(new.max()))
    return st


def prepare(case, seed):
    st, op = _inputs(case, seed), case["op"]
    if own:
        from linear_attention_serving_delta_gb300 import kda
        if op == "write":
            st["call"] = kda.KvWrite(st["k"], st["v"], st["slot_map"], st["k_cache"], st["v_cache"])
        elif op == "plan":
            st["call"] = kda.KvPlan(st["cu"], st["T"], st["table"], st["lens"], st["free"], st["count"],
                                    page_size=st["page"], rows=st["rows"], kv_lens_out=st["lens_out"],
                                    free_count_out=st["count_out"])
        elif op == "prompt":
            st["call"] = kda.AttnPrefill(st["q"], st["k"], st["v"], st["cu"], scale=st["scale"])
        else:
            st["call"] = kda.AttnPaged(st["q"], st["k_cache"], st["v_cache"], st["table"], st["lens"], st["cu"],
                                       scale=st["scale"], max_seqlen=st["max_new"])
    return st


# ------------------------------------------------------------------ plain forms
def _plain_plan(st):
    cu, page, T = st["cu"], st["page"], st["T"]
    rows = st["rows"].long()
    new = cu[1:] - cu[:-1]
    ctx = st["lens"][rows]
    have = (ctx + page - 1) // page
    need = (ctx + new + page - 1) // page - have
    end = need.cumsum(0)
    count = st["count"].long()
    served = (need == 0) | (end <= count)
    table = st["table"].clone()
    take = torch.where(served, need, torch.zeros_like(need))
    # one entry for each new page
    seq = torch.repeat_interleave(torch.arange(rows.numel(), device=cu.device), take)
    first = end - need
    j = torch.arange(seq.numel(), device=cu.device) - (take.cumsum(0) - take)[seq]
    table[rows[seq], have[seq] + j] = st["free"][count - 1 - (first[seq] + j)]
    # one slot for each new token
    tok = torch.arange(T, device=cu.device)
    ts = torch.searchsorted(cu, tok, right=True) - 1
    pos = ctx[ts] + tok - cu[ts]
    slot = table[rows[ts], pos // page].long() * page + pos % page
    slot = torch.where(served[ts], slot, torch.full_like(slot, -1))
    lens = st["lens"].clone()
    lens[rows] = torch.where(served, ctx + new, ctx)
    left = (count - take.sum()).int()
    return table, slot, lens, left


def _plain_write(st):
    hkv, d = st["case"]["hkv"], st["case"]["d"]
    keep = st["slot_map"] >= 0
    slots = st["slot_map"][keep]
    st["k_cache"].view(-1, hkv, d)[slots] = st["k"][keep]
    st["v_cache"].view(-1, hkv, d)[slots] = st["v"][keep]
    return st["k_cache"], st["v_cache"]


def _plain_rows(q, k, v, pos0, scale, out):
    """Causal attention of q [n, hq, d] at positions pos0.. over k, v [m, hkv, d], by blocks of rows."""
    n, hq, d = q.shape
    m, hkv = k.shape[0], k.shape[1]
    grp = hq // hkv
    kf, vf = k.float().permute(1, 2, 0), v.float().permute(1, 0, 2)
    step = max(16, min(1024, int(2.5e8 / max(1, hq * m))))
    for a in range(0, n, step):
        b = min(n, a + step)
        keys = min(m, pos0 + b)
        if keys <= 0:
            out[a:b] = 0
            continue
        qb = q[a:b].float().reshape(b - a, hkv, grp, d).permute(1, 2, 0, 3).reshape(hkv, grp * (b - a), d)
        s = torch.matmul(qb, kf[:, :, :keys]) * scale
        s = s.view(hkv, grp, b - a, keys)
        dead = torch.arange(keys, device=q.device)[None, :] > pos0 + torch.arange(a, b, device=q.device)[:, None]
        s.masked_fill_(dead, float("-inf"))
        top = s.amax(-1, keepdim=True)
        s = torch.exp(s - torch.where(torch.isinf(top), torch.zeros_like(top), top))
        den = s.sum(-1, keepdim=True)
        r = torch.matmul(s.view(hkv, -1, keys), vf[:, :keys]).view(hkv, grp, b - a, d)
        r = r / torch.where(den == 0, torch.ones_like(den), den)
        out[a:b] = r.permute(2, 0, 1, 3).reshape(b - a, hq, d).to(out.dtype)


def _plain_attention(st):
    q, cu = st["q"], st["host_cu"]
    out = torch.zeros_like(q)
    for s in range(len(cu) - 1):
        a, b = cu[s], cu[s + 1]
        if a == b:
            continue
        if st["op"] == "prompt":
            _plain_rows(q[a:b], st["k"][a:b], st["v"][a:b], 0, st["scale"], out[a:b])
        else:
            m, page = st["host_lens"][s], st["case"]["page"]
            pages = st["table"][s, :(m + page - 1) // page].long()
            k = st["k_cache"][pages].flatten(0, 1)[:m]
            v = st["v_cache"][pages].flatten(0, 1)[:m]
            _plain_rows(q[a:b], k, v, m - (b - a), st["scale"], out[a:b])
    return out


def run(st):
    op = st["op"]
    if own:
        c = st["call"].run()
        if op == "write":
            return st["k_cache"], st["v_cache"]
        if op == "plan":
            return st["table"], c.slot_map, c.kv_lens_out, c.free_count_out
        return c.o
    if op == "write":
        return _plain_write(st)
    if op == "plan":
        return _plain_plan(st)
    return _plain_attention(st)


# ------------------------------------------------------------------ work and definition
def _pairs(case):
    new, ctx = _work_lens(case)
    return float((new * ctx + new * (new + 1) / 2).sum())


def work(case):
    op = case["op"]
    if op == "write":
        b = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 4.0 * case["t"] * case["hkv"] * case["d"] * b + 8.0 * case["t"], "flops": 0.0}
    new, ctx = _work_lens(case)
    if op == "plan":
        pages = float(((ctx + new + case["page"] - 1) // case["page"] - (ctx + case["page"] - 1) // case["page"]).sum())
        # a slot for each token, a page read and written for each new one, lengths and offsets of each request
        return {"bytes": 8.0 * float(new.sum()) + 8.0 * pages + 28.0 * case["n"], "flops": 0.0}
    b = 2 if case["dtype"] == "bf16" else 4
    rows = float(new.sum())
    kv = rows if op == "prompt" else float((ctx + new).sum())
    return {"bytes": b * case["d"] * (2.0 * rows * case["hq"] + 2.0 * kv * case["hkv"]),
            "flops": 4.0 * case["d"] * case["hq"] * _pairs(case)}


def exact(case, seed):
    """The attention's definition in 64 bits, a key head at a time; the cache's rows, one scatter for each tensor."""
    if case["op"] == "plan" or (case["op"] != "write" and 4.0 * case["d"] * case["hq"] * _pairs(case) > 4e12):
        return None
    if case["op"] == "write":
        st = _inputs(case, seed)
        where = torch.nonzero(st["slot_map"] + 1).flatten()
        res = []
        for cache, rows in ((st["k_cache"], st["k"]), (st["v_cache"], st["v"])):
            full = cache.double().flatten(0, 1)
            full.index_copy_(0, st["slot_map"].index_select(0, where), rows.index_select(0, where).double())
            res.append(full.view(cache.shape))
        return tuple(res)
    st = _inputs(case, seed)
    q, cu, grp = st["q"], st["host_cu"], case["hq"] // case["hkv"]
    res = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    for s in range(len(cu) - 1):
        n = cu[s + 1] - cu[s]
        if n == 0:
            continue
        if case["op"] == "prompt":
            m, idx, ks, vs = n, slice(cu[s], cu[s + 1]), st["k"], st["v"]
        else:
            m, page = st["host_lens"][s], case["page"]
            where = torch.arange(m, device=q.device)
            idx = st["table"][s].long()[where // page] * page + where % page
            ks, vs = st["k_cache"].flatten(0, 1), st["v_cache"].flatten(0, 1)
        for h in range(case["hkv"]):
            kh, vh = ks[idx, h].double(), vs[idx, h].double()
            for a in range(0, n, 2048):
                b = min(n, a + 2048)
                keys = m - n + b
                x = q[cu[s] + a:cu[s] + b, h * grp:(h + 1) * grp].double()
                logit = torch.einsum("tgd,jd->tgj", x, kh[:keys]) * st["scale"]
                at = torch.arange(m - n + a, m - n + b, device=q.device)
                seen = torch.arange(keys, device=q.device)[None, :] <= at[:, None]
                w = torch.softmax(logit.masked_fill(~seen[:, None, :], -torch.inf), dim=-1)
                res[cu[s] + a:cu[s] + b, h * grp:(h + 1) * grp] = torch.einsum("tgj,jd->tgd", w, vh[:keys])
    return res
