"""Linear attention with a decay for each head, as workloads to measure.

Four operators over fixed-size states S (dk x dv, fp32) of every head,
S_t = a_t S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t, log a_t = -slope softplus(g_t):
packed prompts (``prompt``), one token a row over a pool of states
(``decode``), trees of drafted tokens that leave the states as they are
(``draft``), and the states moved on along the accepted path (``commit``).
``run`` computes each in a plain form from elementary torch operations, or,
with ``own`` set, through the package.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
# heads of v, o and the states; heads of q and k
HEADS = [(32, 32), (16, 16), (8, 8), (24, 24), (32, 8), (16, 1), (20, 4), (64, 64), (4, 4), (1, 1)]
WIDTHS = [(64, 64), (128, 128), (128, 128), (128, 128), (128, 64), (64, 128), (32, 32), (256, 256), (128, 256)]


def listed():
    return [
        # a handful of short chat turns, where latency counts
        dict(name="prompt_short_ragged", op="prompt", n=5, lo=1, hi=200, h=8, hk=8, dk=64, dv=64, gate="g", init=False,
             dtype="bf16"),
        # one long prompt
        dict(name="prompt_8k", op="prompt", n=1, lo=8192, hi=8192, h=32, hk=32, dk=128, dv=128, gate="g", init=False,
             dtype="bf16"),
        # eight packed prompts of very different lengths that go on from saved states, a constant decay for each
        # head: the largest case
        dict(name="prompt_varlen_8", op="prompt", n=8, lo=1024, hi=32768, uniform=True, h=32, hk=32, dk=128, dv=128,
             gate="slope", init=True, dtype="bf16"),
        # heads that share queries and keys, narrow values, decays from both
        dict(name="prompt_shared", op="prompt", n=6, lo=300, hi=5000, h=32, hk=8, dk=128, dv=64, gate="both", init=True,
             dtype="bf16"),
        # full-precision check runs of a small model
        dict(name="prompt_f32", op="prompt", n=2, lo=500, hi=1500, h=8, hk=8, dk=64, dv=64, gate="g", init=False,
             dtype="f32"),
        # one user's next token
        dict(name="decode_1", op="decode", n=1, h=32, hk=32, dk=128, dv=128, gate="g", dtype="bf16"),
        # a full decode batch
        dict(name="decode_256", op="decode", n=256, h=32, hk=32, dk=128, dv=128, gate="g", dtype="bf16"),
        # a small full-precision batch, odd sizes
        dict(name="decode_f32", op="decode", n=33, h=20, hk=4, dk=64, dv=128, gate="both", dtype="f32"),
        # a batch of requests with trees of eight drafted tokens
        dict(name="draft_64", op="draft", n=64, lo=8, hi=8, h=32, hk=32, dk=128, dv=128, gate="g", dtype="bf16"),
        # trees of very different sizes
        dict(name="draft_ragged", op="draft", n=9, lo=1, hi=60, h=16, hk=4, dk=128, dv=64, gate="both", dtype="bf16"),
        # the accepted paths of that batch
        dict(name="commit_64", op="commit", n=64, lo=8, hi=8, h=32, hk=32, dk=128, dv=128, gate="g", dtype="bf16"),
        # and of trees of very different sizes, full precision
        dict(name="commit_f32", op="commit", n=9, lo=1, hi=60, h=16, hk=16, dk=64, dv=64, gate="slope", dtype="f32"),
    ]


def _logint(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "prompt", "decode", "decode", "draft", "commit"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    dk, dv = rng.choice(WIDTHS)
    h, hk = rng.choice(HEADS)
    case = dict(op=op, h=h, hk=hk, dk=dk, dv=dv, gate=rng.choice(["g", "slope", "both"]), dtype=dtype)
    if op == "prompt":
        n = _logint(rng, 1, 24)
        # tokens of the longest, by the operations of all
        top = 2.0e12 if dtype == "bf16" else 1.0e11
        top = int(min(60000, top / (n * h * (dk * dv + 64 * (dk + dv)) * 4.0)))
        hi = _logint(rng, 2, max(4, top))
        return dict(case, n=n, lo=max(1, hi // 20), hi=hi, init=rng.random() < 0.5)
    most = int(1.0e9 / (h * dk * dv * 4.0))  # requests whose states take a gigabyte
    if op == "decode":
        return dict(case, n=_logint(rng, 1, min(600, most)))
    hi = rng.choice([3, 8, 8, 16, 64])
    return dict(case, n=_logint(rng, 1, min(200, most)), lo=rng.choice([1, hi]), hi=hi)


def _lens(case, seed):
    """Tokens of each request, on the host: the same lengths for every seed, in another order, so that the sizes of
    a case stay its own."""
    g = torch.Generator().manual_seed(17)
    n, lo, hi = case["n"], case["lo"], case["hi"]
    if hi >= 8 * lo and not case.get("uniform"):  # a wide range, spread over its logarithm
        new = (lo * torch.exp(torch.rand(n, generator=g, dtype=torch.float64) * math.log((hi + 0.49) / lo))).long()
    else:
        new = torch.randint(lo, hi + 1, (n,), generator=g)
    return new.clamp(lo, hi)[torch.randperm(n, generator=torch.Generator().manual_seed(seed + 1))]


def _inputs(case, seed):
    dev, op = "cuda", case["op"]
    g = torch.Generator(device=dev).manual_seed(seed * 104729 + 11)
    host = torch.Generator().manual_seed(seed * 7919 + 3)
    n, h, hk, dk, dv, dt = (case[x] for x in ("n", "h", "hk", "dk", "dv", "dtype"))

    def rand(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)

    st = dict(op=op, case=case, scale=dk ** -0.5)
    if op == "decode":
        t = n
    else:
        new = _lens(case, seed)
        cu = torch.zeros(n + 1, dtype=torch.int64)
        cu[1:] = new.cumsum(0)
        t = int(cu[-1])
        st.update(cu=cu.to(dev), host_cu=cu.tolist(), max_new=int(new.max()))
    if op != "commit":
        st["q"] = rand(t, hk, dk).to(DT[dt])
    st.update(k=rand(t, hk, dk).to(DT[dt]), v=rand(t, h, dv).to(DT[dt]), g=None, slope=None)
    if case["gate"] == "slope":  # heads from short to long memory
        st["slope"] = 2.0 ** (-8.0 * torch.arange(1, h + 1, device=dev).float() / h)
    elif case["gate"] == "both":  # steps of a few hundredths, rates of 0.5 to 8
        st["slope"] = 0.5 * 16.0 ** torch.rand(h, generator=g, device=dev)
        st["g"] = (rand(t, h) - 4.0).to(DT[dt])
    else:
        st["g"] = (rand(t, h) - 3.0).to(DT[dt])
    if op == "prompt":
        st["init"] = rand(n, h, dk, dv) if case["init"] else None
        return st
    # a pool of states with some rows to spare, the requests' rows in any order
    st["slots"] = torch.randperm(n + 3, generator=host)[:n].int().to(dev)
    st["state"] = rand(n + 3, h, dk, dv)
    if op != "draft":
        st["state_out"] = torch.zeros_like(st["state"])
    if op == "decode":
        return st
    # trees: most tokens follow the one before, the others an earlier one (-1: the state itself)
    parents = []
    for s in range(n):
        ln = int(new[s])
        idx = torch.arange(ln)
        other = (torch.rand(ln, generator=host) * (idx + 1)).long() - 1
        parents.append(torch.where(torch.rand(ln, generator=host) < 0.6, idx - 1, other))
    par = torch.cat(parents).int()
    st.update(parents=par.to(dev), host_parents=par.tolist())
    if op == "commit":
        last = (torch.rand(n, generator=host) * (new + 1)).long() - 1  # -1: nothing was accepted
        st.update(last=last.int().to(dev), host_last=last.tolist())
    return st


def prepare(case, seed):
    st, op = _inputs(case, seed), case["op"]
    if own:
        from linear_attention_serving_delta_gb300 import kda
        decay = dict(g=st["g"], slope=st["slope"])
        if op == "prompt":
            st["call"] = kda.LinPrefill(st["q"], st["k"], st["v"], st["cu"], scale=st["scale"], initial_state=st["init"],
                                        **decay)
        elif op == "decode":
            st["call"] = kda.LinDecode(st["q"], st["k"], st["v"], st["state"], scale=st["scale"],
                                       state_out=st["state_out"], state_slots=st["slots"], **decay)
        elif op == "draft":
            st["call"] = kda.LinDraft(st["q"], st["k"], st["v"], st["cu"], st["state"], scale=st["scale"],
                                      parents=st["parents"], state_slots=st["slots"], max_seqlen=st["max_new"], **decay)
        else:
            st["call"] = kda.LinCommit(st["k"], st["v"], st["cu"], st["last"], st["state"], parents=st["parents"],
                                       state_out=st["state_out"], state_slots=st["slots"], max_seqlen=st["max_new"],
                                       **decay)
    return st


# ------------------------------------------------------------------ plain forms
def _log_decay(st, t0, t1):
    """log a of tokens t0..t1 in 64 bits (sums over long stretches follow), [t, H]."""
    h = st["case"]["h"]
    x = torch.ones(t1 - t0, h, device=st["k"].device, dtype=torch.float64)
    if st["g"] is not None:
        x = torch.nn.functional.softplus(st["g"][t0:t1].double())
    return -x if st["slope"] is None else -x * st["slope"].double()


def _heads_first(x, h):
    """[t, heads, d] -> [h, t, d] in fp32, shared heads repeated."""
    return x.float().repeat_interleave(h // x.shape[1], dim=1).transpose(0, 1)


def _plain_prompt(st):
    case, cu = st["case"], st["host_cu"]
    h, dk, dv = case["h"], case["dk"], case["dv"]
    dev, c = st["q"].device, 128
    o = torch.zeros(st["v"].shape, device=dev, dtype=st["v"].dtype)
    final = torch.zeros(case["n"], h, dk, dv, device=dev)
    lower = torch.ones(c, c, device=dev, dtype=torch.bool).tril()
    for s in range(case["n"]):
        state = torch.zeros(h, dk, dv, device=dev) if st["init"] is None else st["init"][s].clone()
        for a in range(cu[s], cu[s + 1], c):
            b = min(cu[s + 1], a + c)
            q, k, v = (_heads_first(st[x][a:b], h) for x in "qkv")
            gsum = _log_decay(st, a, b).cumsum(0).t()  # [h, t]
            w = torch.exp((gsum[:, :, None] - gsum[:, None, :]).masked_fill(~lower[:b - a, :b - a], float("-inf")))
            att = torch.matmul(q, k.transpose(1, 2)) * w.float()
            part = torch.matmul(att, v) + torch.exp(gsum).float()[:, :, None] * torch.matmul(q, state)
            o[a:b] = (part * st["scale"]).transpose(0, 1).to(o.dtype)
            tail = torch.exp(gsum[:, -1:] - gsum).float()
            state = torch.exp(gsum[:, -1]).float()[:, None, None] * state + torch.matmul(
                (k * tail[:, :, None]).transpose(1, 2), v)
        final[s] = state
    return o, final


def _plain_decode(st):
    case, rows = st["case"], st["slots"].long()
    n, h = case["n"], case["h"]
    rep = h // case["hk"]
    q, k = (st[x].float().repeat_interleave(rep, dim=1) for x in "qk")
    decay = torch.exp(_log_decay(st, 0, n)).float()
    o = torch.empty(st["v"].shape, device=q.device, dtype=st["v"].dtype)
    step = max(1, int(2.5e8 / (h * case["dk"] * case["dv"])))
    for a in range(0, n, step):
        r = slice(a, min(n, a + step))
        new = decay[r][:, :, None, None] * st["state"][rows[r]] + k[r][..., None] * st["v"][r].float()[:, :, None, :]
        st["state_out"][rows[r]] = new
        o[r] = (torch.matmul(q[r][:, :, None, :], new)[:, :, 0] * st["scale"]).to(o.dtype)
    return o, st["state_out"]


def _plain_draft(st):
    case, cu, par = st["case"], st["host_cu"], st["host_parents"]
    h = case["h"]
    o = torch.zeros(st["v"].shape, device=st["q"].device, dtype=st["v"].dtype)
    for s in range(case["n"]):
        a, b = cu[s], cu[s + 1]
        seen = torch.zeros(b - a, b - a)
        for i in range(b - a):
            if par[a + i] >= 0:
                seen[i] = seen[par[a + i]]
            seen[i, i] = 1
        seen = seen.to(o.device)
        gsum = torch.matmul(seen.double(), _log_decay(st, a, b)).t()  # [h, t], along each path
        q, k, v = (_heads_first(st[x][a:b], h) for x in "qkv")
        w = (gsum[:, :, None] - gsum[:, None, :]).masked_fill(seen == 0, float("-inf"))
        att = torch.matmul(q, k.transpose(1, 2)) * torch.exp(w).float()
        state = st["state"][st["slots"][s].long()]
        part = torch.matmul(att, v) + torch.exp(gsum).float()[:, :, None] * torch.matmul(q, state)
        o[a:b] = (part * st["scale"]).transpose(0, 1).to(o.dtype)
    return o


def _plain_commit(st):
    case, cu, par = st["case"], st["host_cu"], st["host_parents"]
    h = case["h"]
    for s in range(case["n"]):
        path, i = [], st["host_last"][s]
        while i >= 0:
            path.insert(0, cu[s] + i)
            i = par[cu[s] + i]
        row = st["slots"][s].long()
        state = st["state"][row]
        if path:
            idx = torch.tensor(path, device=state.device)
            gsum = _log_decay(st, cu[s], cu[s + 1])[idx - cu[s]].cumsum(0).t()
            k, v = (_heads_first(st[x][idx], h) for x in "kv")
            tail = torch.exp(gsum[:, -1:] - gsum).float()
            state = torch.exp(gsum[:, -1]).float()[:, None, None] * state + torch.matmul(
                (k * tail[:, :, None]).transpose(1, 2), v)
        st["state_out"][row] = state
    return st["state_out"]


def run(st):
    op = st["op"]
    if own:
        c = st["call"].run()
        if op == "prompt":
            return c.o, c.final_state
        if op == "decode":
            return c.o, c.state_out
        return c.o if op == "draft" else c.state_out
    return {"prompt": _plain_prompt, "decode": _plain_decode, "draft": _plain_draft, "commit": _plain_commit}[op](st)


# ------------------------------------------------------------------ work and definition
def work(case):
    op, n, h, hk, dk, dv = (case[x] for x in ("op", "n", "h", "hk", "dk", "dv"))
    b = 2.0 if case["dtype"] == "bf16" else 4.0
    t = float(n if op == "decode" else _lens(case, 0).sum())
    state = 4.0 * n * h * dk * dv
    gate = (b * t * h if case["gate"] != "slope" else 0.0) + (4.0 * h if case["gate"] != "g" else 0.0)
    qk, vo = b * t * hk * dk, b * t * h * dv
    if op == "prompt":
        return {"bytes": 2 * qk + 2 * vo + gate + state * (2 if case["init"] else 1), "flops": 4.0 * t * h * dk * dv}
    if op == "decode":
        return {"bytes": 2 * qk + 2 * vo + gate + 2 * state, "flops": 4.0 * t * h * dk * dv}
    if op == "draft":
        return {"bytes": 2 * qk + 2 * vo + gate + state, "flops": 2.0 * t * h * (dk * dv + dk + dv)}
    # about half of the tokens are on the path, at most
    return {"bytes": 2 * state + 0.25 * (qk + vo), "flops": 0.5 * t * h * dk * dv}


def exact(case, seed):
    """The definition in 64 bits, one head at a time; prompts and paths by blocks, weights from the logarithms."""
    if case["op"] == "prompt":
        tokens = float(_lens(case, 0).sum())
        if tokens * case["h"] * (case["dk"] * case["dv"] + 256 * (case["dk"] + case["dv"])) * 4.0 > 8e12:
            return None
    st = _inputs(case, seed)
    h, hk, n, dev = case["h"], case["hk"], case["n"], st["k"].device
    val = st["v"].double()
    loga = torch.full((val.shape[0], h), -1.0, dtype=torch.float64, device=dev)
    if st["g"] is not None:
        x = st["g"].double()
        loga = -(torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs())))
    if st["slope"] is not None:
        loga = loga * st["slope"].double()[None, :]
    grp = h // hk
    if case["op"] == "decode":
        out, states = torch.zeros_like(val), st["state_out"].double()
        for r in range(n):
            row = int(st["slots"][r])
            old = st["state"][row].double()
            kk = st["k"][r].double()[torch.arange(h, device=dev) // grp]
            qq = st["q"][r].double()[torch.arange(h, device=dev) // grp]
            states[row] = torch.exp(loga[r])[:, None, None] * old + torch.einsum("hi,hj->hij", kk, val[r])
            out[r] = st["scale"] * torch.einsum("hij,hi->hj", states[row], qq)
        return out, states

    def paths(s):
        """Ancestors of each token of request s, itself included, in order."""
        a = st["host_cu"][s]
        res = []
        for i in range(st["host_cu"][s + 1] - a):
            up = st["host_parents"][a + i]
            res.append((res[up] if up >= 0 else []) + [i])
        return res

    if case["op"] == "draft":
        out = torch.zeros_like(val)
        for s in range(n):
            a, b = st["host_cu"][s], st["host_cu"][s + 1]
            anc = paths(s)
            old = st["state"][int(st["slots"][s])].double()
            on = torch.zeros(b - a, b - a, dtype=torch.float64)
            for i, p in enumerate(anc):
                on[i, p] = 1.0
            on = on.to(dev)
            total = torch.einsum("ij,jh->ih", on, loga[a:b])
            for x in range(h):
                kk, qq = st["k"][a:b, x // grp].double(), st["q"][a:b, x // grp].double()
                weight = torch.where(on > 0, torch.exp(torch.where(on > 0, total[:, x, None] - total[None, :, x], 0.0)), 0.0)
                res = torch.einsum("ij,jd->id", weight * torch.einsum("id,jd->ij", qq, kk), val[a:b, x])
                out[a:b, x] = st["scale"] * (res + torch.exp(total[:, x, None]) * (qq @ old[x]))
        return out
    if case["op"] == "commit":
        states = st["state_out"].double()
        for s in range(n):
            a, row = st["host_cu"][s], int(st["slots"][s])
            states[row] = st["state"][row].double()
            if st["host_last"][s] < 0:
                continue
            for i in paths(s)[st["host_last"][s]]:  # token by token
                kk = st["k"][a + i].double()[torch.arange(h, device=dev) // grp]
                states[row] = torch.exp(loga[a + i])[:, None, None] * states[row] + torch.einsum("hi,hj->hij", kk, val[a + i])
        return states
    out = torch.zeros_like(val)
    final = torch.zeros(n, h, case["dk"], case["dv"], dtype=torch.float64, device=dev)
    for s in range(n):
        if st["init"] is not None:
            final[s] = st["init"][s].double()
        for a in range(st["host_cu"][s], st["host_cu"][s + 1], 256):
            b = min(st["host_cu"][s + 1], a + 256)
            since = torch.cumsum(loga[a:b], 0)
            idx = torch.arange(b - a, device=dev)
            later = idx[:, None] >= idx[None, :]
            for x0 in range(0, h, 8):  # (eight heads at a time)
                x1 = min(h, x0 + 8)
                at = torch.arange(x0, x1, device=dev)
                kk, qq = st["k"][a:b].double()[:, at // grp], st["q"][a:b].double()[:, at // grp]
                lag = since[:, None, x0:x1] - since[None, :, x0:x1]
                weight = torch.exp(torch.where(later[:, :, None], lag, -torch.inf))
                score = torch.einsum("ihd,jhd->ijh", qq, kk) * weight
                fresh = torch.einsum("ijh,jhd->ihd", score, val[a:b, x0:x1])
                old = torch.einsum("ihd,hde->ihe", qq * torch.exp(since[:, x0:x1])[:, :, None], final[s, x0:x1])
                out[a:b, x0:x1] = st["scale"] * (fresh + old)
                left = torch.exp(since[-1:, x0:x1] - since[:, x0:x1])
                final[s, x0:x1] = torch.exp(since[-1, x0:x1])[:, None, None] * final[s, x0:x1] + torch.einsum(
                    "jhd,jhe->hde", kk * left[:, :, None], val[a:b, x0:x1])
    return out, final
