"""Cases of the paged K/V cache (write, read back), of chunk attention over it, and of cross attention.

``own`` false: the operators in their plain form, elementary torch operations in 32 bits.
``own`` true: the same passes through the entry points of ``block_sparse_video_int8_b200``.

Cache: pages [n_pages, Hkv, page_size, d], INT8 codes with an fp32 scale per (token, head), s = fl32(amax / 127),
code = rint_half_even(fl32(x / s)); or plain bf16 pages. Sequence s has kv_len[s] tokens, the last
q_start[s+1] - q_start[s] of them new; token t of it lies in page page_table[s, t // page_size].
"""
import math
import random

import torch

own = False


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one generated token of each of 16 sequences enters the cache and is read back: pure latency
        dict(name="store_token", op="store", S=16, new=1, kv=700, Hkv=8, d=128, page=16, pages="int8", layout=1, whole=False),
        # ragged chunks (one of them empty) at odd lengths, small heads, whole sequences read back
        dict(name="store_ragged", op="store", S=7, new=419, kv=1003, Hkv=12, d=64, page=32, pages="int8", layout=2, whole=True),
        # a prompt of two latent slices of 48 x 84 tokens for each of 4 sequences, 40 heads: bandwidth
        dict(name="store_slices", op="store", S=4, new=8064, kv=8064, Hkv=40, d=128, page=128, pages="int8", layout=3, whole=True),
        # one token of one sequence against a short context: pure latency
        dict(name="decode_one", op="attend", S=1, new=1, kv=1003, Hq=40, Hkv=8, d=128, page=16, pages="int8", layout=4, window=0, lse=False, tail=0),
        # a serving batch, one token each, contexts of all lengths
        dict(name="decode_batch", op="attend", S=32, new=1, kv=16384, Hq=40, Hkv=8, d=128, page=64, pages="int8", layout=5, window=0, lse=False, tail=0),
        # one token each over very long contexts, every query head with its own key head
        dict(name="decode_long", op="attend", S=2, new=1, kv=131000, Hq=40, Hkv=40, d=128, page=128, pages="int8", layout=6, window=0, lse=False, tail=0),
        # a frame of 32 x 48 tokens joins 7 earlier ones, bf16 pages
        dict(name="chunk_frame", op="attend", S=1, new=1536, kv=12288, Hq=12, Hkv=12, d=128, page=128, pages="bf16", layout=7, window=0, lse=True, tail=0),
        # a long prompt in chunks: 2048 new tokens of a 32760-token context
        dict(name="chunk_long", op="attend", S=1, new=2048, kv=32760, Hq=40, Hkv=8, d=128, page=64, pages="int8", layout=8, window=0, lse=True, tail=0),
        # mixed batch: empty, single-token and longer chunks, sliding window, 7 query heads a key head, rows behind the last sequence
        dict(name="chunk_mixed", op="attend", S=9, new=300, kv=5000, Hq=14, Hkv=2, d=64, page=32, pages="int8", layout=9, window=1000, lse=True, tail=5),
        # video tokens (21 x 30 x 52) to 512 text tokens, 40 heads
        dict(name="cross_video", op="cross", B=1, Lq=32760, Lk=512, Hq=40, Hkv=40, d=128, ragged=False, layout=10, lse=False),
        # padded text of several lengths, one empty; shared key heads, odd sizes
        dict(name="cross_ragged", op="cross", B=3, Lq=1003, Lk=77, Hq=12, Hkv=4, d=64, ragged=True, layout=11, lse=True),
        # one decoder token of each of 16 sequences to its encoder's states
        dict(name="cross_token", op="cross", B=16, Lq=1, Lk=1500, Hq=12, Hkv=12, d=64, ragged=True, layout=12, lse=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["store", "attend", "attend", "cross"])
    d, layout = rng.choice([64, 128]), rng.randrange(1 << 20)
    Hkv, G = rng.choice([1, 2, 4, 8, 12, 40]), rng.choice([1, 1, 2, 3, 4, 5, 7, 8])
    page, pages = rng.choice([16, 32, 64, 128]), rng.choice(["int8", "int8", "bf16"])
    if op == "store":
        S, kv = _log(rng, 1, 32), _log(rng, 1, 8064)
        new = _log(rng, 1, kv)
        while S * kv * Hkv * d > 4 * 8064 * 40 * 128:
            S, Hkv = max(1, S // 2), max(1, Hkv // 2)
        return dict(op=op, S=S, new=new, kv=kv, Hkv=Hkv, d=d, page=page, pages=pages, layout=layout, whole=rng.random() < 0.6)
    if op == "attend":
        S, kv = _log(rng, 1, 32), _log(rng, 1, 131000)
        new = 1 if rng.random() < 0.4 else _log(rng, 1, min(kv, 2048))
        Hkv = min(Hkv, 40 // G)
        while S * kv * Hkv * d > 2 * 131000 * 40 * 128 or S * new * kv * Hkv * G > 2048 * 32760 * 40:
            S, new, Hkv = max(1, S // 2), max(1, new // 2), max(1, (Hkv + 1) // 2)
        return dict(op=op, S=S, new=new, kv=kv, Hq=Hkv * G, Hkv=Hkv, d=d, page=page, pages=pages, layout=layout,
                    window=rng.choice([0, 0, 0, _log(rng, 1, kv)]), lse=rng.random() < 0.5, tail=rng.choice([0, 0, 3]))
    B, Lq, Lk = _log(rng, 1, 16), 1 if rng.random() < 0.25 else _log(rng, 1, 32760), _log(rng, 1, 1500)
    Hkv = min(Hkv, 40 // G)
    while B * Lq * Lk * Hkv * G > 32760 * 512 * 40 or B * Lq * Hkv * G > 32760 * 40:
        B, Lq = max(1, B // 2), max(1, Lq // 2)
    return dict(op=op, B=B, Lq=Lq, Lk=Lk, Hq=Hkv * G, Hkv=Hkv, d=d, ragged=rng.random() < 0.5, layout=layout, lse=rng.random() < 0.5)


def _lengths(case):
    """(new tokens, total tokens) of each sequence. The first has the case's sizes; chunks of several sequences vary,
    the third one is empty."""
    rng, out = random.Random(case["layout"]), []
    for s in range(case["S"]):
        kv = case["kv"] if s == 0 else rng.randint(max(1, case["kv"] // 8), case["kv"])
        new = case["new"] if s == 0 or case["new"] in (1, case["kv"]) else rng.randint(1, case["new"])
        if s == 2 and case["new"] > 1 and case["new"] != case["kv"]:
            new = 0
        if case["new"] == case["kv"]:
            new = kv = case["kv"] if s % 2 == 0 else kv
        out.append((min(new, kv), kv))
    return out


def _key_lengths(case):
    rng = random.Random(case["layout"])
    if not case["ragged"]:
        return [case["Lk"]] * case["B"]
    return [case["Lk"] if b == 0 else 0 if b == 2 and case["Lq"] > 1 else rng.randint(1, case["Lk"]) for b in range(case["B"])]


# ----------------------------------------------------------------------------------------------- inputs
def _states(gen, rows, heads, d, dev):
    """Keys or values as a layer gives them, bf16 [rows, heads, d]: normal, some channels and tokens larger."""
    x = torch.randn((rows, heads, d), generator=gen, device=dev)
    x *= torch.exp(0.5 * torch.randn((rows, heads, 1), generator=gen, device=dev))
    x *= 1 + 3 * (torch.rand((heads, d), generator=gen, device=dev) < 0.05)
    return x.to(torch.bfloat16)


def _quantise(x):
    """Codes (as fp32) and scales of the rows of x."""
    x = x.float()
    s = x.abs().amax(-1) / 127.0
    c = torch.round(x / torch.where(s > 0, s, 1.0).unsqueeze(-1))
    return c, s


def _made(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=dev).manual_seed(seed)
    st = dict(case=case)
    if case["op"] == "cross":
        B, Lq, Lk, d = case["B"], case["Lq"], case["Lk"], case["d"]
        st["q"] = torch.randn((B, case["Hq"], Lq, d), generator=gen, device=dev).to(torch.bfloat16)
        for n in "kv":
            st[n] = _states(gen, B * Lk, case["Hkv"], d, dev).view(B, Lk, case["Hkv"], d).transpose(1, 2).contiguous()
        st["k_len"] = torch.tensor(_key_lengths(case), dtype=torch.int32, device=dev)
        return st
    S, Hkv, d, ps = case["S"], case["Hkv"], case["d"], case["page"]
    lens = _lengths(case)
    per = (case["kv"] + ps - 1) // ps
    used = sum((kv + ps - 1) // ps for _, kv in lens)
    n_pages = used + 3
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table, at, starts = torch.full((S, per), -1, dtype=torch.int32), 0, [0]
    for s, (new, kv) in enumerate(lens):
        n = (kv + ps - 1) // ps
        table[s, :n] = order[at:at + n]
        at += n
        starts.append(starts[-1] + new)
    st["table"] = table.to(dev)
    st["q_start"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    st["kv_len"] = torch.tensor([kv for _, kv in lens], dtype=torch.int32, device=dev)
    st["max_q"], st["max_kv"] = max(n for n, _ in lens), max(kv for _, kv in lens)
    for n in "kv":      # what earlier tokens left in the pages
        x = _states(gen, n_pages * ps, Hkv, d, dev).view(n_pages, ps, Hkv, d).transpose(1, 2).contiguous()
        if case["pages"] == "int8":
            c, sc = _quantise(x)
            st["p" + n], st["s" + n] = c.to(torch.int8), sc
        else:
            st["p" + n] = x
    T = starts[-1] + case.get("tail", 0)
    if case["op"] == "store":
        # one projection's output, keys and values side by side for each token
        kv = torch.cat([_states(gen, T, Hkv, d, dev), _states(gen, T, Hkv, d, dev)], 1)
        st["k"], st["v"] = kv[:, :Hkv], kv[:, Hkv:]
        first = [0 if case["whole"] else kv_ - new for new, kv_ in lens]
        st["first"] = torch.tensor(first, dtype=torch.int32, device=dev)
        st["L"] = max(kv_ - f for f, (_, kv_) in zip(first, lens))
    else:
        st["q"] = torch.randn((T, case["Hq"], d), generator=gen, device=dev).to(torch.bfloat16)
        st["out"] = torch.zeros_like(st["q"])
        st["lse"] = torch.zeros((T, case["Hq"]), device=dev) if case["lse"] else None
    return st


def prepare(case, seed):
    st = _made(case, seed)
    if own:     # the handles that a serving program keeps: the cache over its pages, the batch's plan, the workspace
        import block_sparse_video_int8_b200 as bsva
        if case["op"] == "cross":
            st["ws"] = bsva.new_cross_attn_workspace(st["q"], st["k"])
        else:
            st["cache"] = bsva.PagedKVCache.over(st["pk"], st["pv"], st.get("sk"), st.get("sv"))
            st["batch"] = bsva.PagedBatch(st["q_start"], st["kv_len"], st["table"], st["max_q"], st["max_kv"])
            st["ws"] = st["cache"].new_workspace(st["batch"], case.get("Hq", case["Hkv"]), st["q" if "q" in st else "k"].shape[0])
    return st


# ---------------------------------------------------------------------------------------------- passes
def _gathered(pages, scales, table, n):
    """The first n tokens of every sequence, fp32 [S, Hkv, n, d] (rows of missing pages are page 0's)."""
    ps = pages.shape[2]
    t = torch.arange(n, device=pages.device)
    page = table.long().clamp(min=0)[:, t // ps]
    x = pages[page, :, t % ps].float()
    if scales is not None:
        x = x * scales[page, :, t % ps].unsqueeze(-1)
    return x.transpose(1, 2)


def _softmax_av(q, k, v, allowed, scale):
    """Rows q [.., m, d] over keys k, v [.., n, d] where allowed: (output, log-sum-exp) in fp32."""
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(scale)
    x.masked_fill_(~allowed, -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    o = torch.matmul(x, v) / torch.where(l > 0, l, 1.0)
    return o, (m + torch.log(l)).squeeze(-1)


def _plain_store(st):
    case = st["case"]
    ps, qs, kl = case["page"], st["q_start"].long(), st["kv_len"].long()
    t = torch.arange(st["k"].shape[0], device=qs.device)
    s = torch.searchsorted(qs[1:], t, right=True)
    pos = kl[s] - qs[s + 1] + t
    page = st["table"].long()[s, pos // ps]
    for n in "kv":
        if case["pages"] == "int8":
            c, sc = _quantise(st[n])
            st["p" + n][page, :, pos % ps] = c.to(torch.int8)
            st["s" + n][page, :, pos % ps] = sc
        else:
            st["p" + n][page, :, pos % ps] = st[n]
    # read back tokens first .. kv_len of each sequence, zeros behind them
    r = torch.arange(st["L"], device=qs.device) + st["first"].long()[:, None]
    live = r < kl[:, None]
    r = torch.where(live, r, 0)
    page = st["table"].long().gather(1, r // ps)
    out = []
    for n in "kv":
        x = st["p" + n][page, :, r % ps].float()
        if case["pages"] == "int8":
            x = x * st["s" + n][page, :, r % ps].unsqueeze(-1)
        out.append(torch.where(live[:, :, None, None], x, 0.0).to(torch.bfloat16).transpose(1, 2).contiguous())
    return tuple(out)


def _plain_attend(st):
    case = st["case"]
    S, Hq, Hkv, d = case["S"], case["Hq"], case["Hkv"], case["d"]
    G, mq, mk = Hq // Hkv, st["max_q"], st["max_kv"]
    qs, kl = st["q_start"].long(), st["kv_len"].long()
    new = qs[1:] - qs[:-1]
    i = torch.arange(mq, device=qs.device)
    rows = (qs[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)
    q = st["q"][rows].float().view(S, mq, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(S, Hkv, G * mq, d)
    t = torch.arange(mk, device=qs.device)
    live = (t < kl[:, None])[:, None, :, None]
    k = _gathered(st["pk"], st.get("sk"), st["table"], mk)
    v = torch.where(live, _gathered(st["pv"], st.get("sv"), st["table"], mk), 0.0)
    pos = (kl - new)[:, None] + i
    ok = t <= pos[:, :, None]
    if case["window"]:
        ok &= t > pos[:, :, None] - case["window"]
    ok = ok[:, None, None].expand(S, 1, G, mq, mk).reshape(S, 1, G * mq, mk)
    o, lse = _softmax_av(q, k, v, ok, 1.0 / math.sqrt(d))
    o = o.view(S, Hkv, G, mq, d).permute(0, 3, 1, 2, 4).reshape(S, mq, Hq, d)
    have = i < new[:, None]
    st["out"][rows[have]] = o[have].to(torch.bfloat16)
    if st["lse"] is None:
        return st["out"]
    st["lse"][rows[have]] = lse.view(S, Hkv, G, mq).permute(0, 3, 1, 2).reshape(S, mq, Hq)[have]
    return st["out"], st["lse"]


def _plain_cross(st):
    case = st["case"]
    B, Lq, Lk, Hkv, d = case["B"], case["Lq"], case["Lk"], case["Hkv"], case["d"]
    live = torch.arange(Lk, device=st["q"].device) < st["k_len"][:, None]
    q = st["q"].float().view(B, Hkv, -1, d)
    v = torch.where(live[:, None, :, None], st["v"].float(), 0.0)
    o, lse = _softmax_av(q, st["k"].float(), v, live[:, None, None, :], 1.0 / math.sqrt(d))
    o = o.view(B, case["Hq"], Lq, d).to(torch.bfloat16)
    return (o, lse.view(B, case["Hq"], Lq)) if case["lse"] else o


def run(state):
    case = state["case"]
    if own:
        import block_sparse_video_int8_b200 as bsva
        if case["op"] == "store":
            state["cache"].write(state["k"], state["v"], state["batch"], workspace=state["ws"])
            return state["cache"].read(state["batch"], first=state["first"], length=state["L"], workspace=state["ws"])
        if case["op"] == "attend":
            return state["cache"].attend(state["q"], state["batch"], window=case["window"], with_lse=case["lse"],
                                         out=state["out"], lse=state["lse"], workspace=state["ws"])
        return bsva.cross_attn_fwd(state["q"], state["k"], state["v"], k_len=state["k_len"], with_lse=case["lse"],
                                   workspace=state["ws"])
    return {"store": _plain_store, "attend": _plain_attend, "cross": _plain_cross}[case["op"]](state)


# ------------------------------------------------------------------------------------------------ work
def work(case):
    d, Hkv = case["d"], case["Hkv"]
    if case["op"] == "cross":
        kl, rows = sum(_key_lengths(case)), case["Hq"] * case["Lq"]
        return {"bytes": 4 * case["B"] * rows * d + 4 * kl * Hkv * d + (4 * case["B"] * rows if case["lse"] else 0),
                "flops": 4 * rows * kl * d}
    lens = _lengths(case)
    held = 2 * Hkv * (d + 4 if case["pages"] == "int8" else 2 * d)     # keys and values of one token in the cache
    new = sum(n for n, _ in lens)
    if case["op"] == "store":
        back = [kv if case["whole"] else n for n, kv in lens]
        return {"bytes": new * (4 * Hkv * d + held) + sum(back) * held + len(back) * max(back) * 4 * Hkv * d,
                "flops": 4 * new * Hkv * d + 2 * sum(back) * Hkv * d}
    pairs = keys = 0
    for n, kv in lens:
        w = case["window"] or kv
        pairs += sum(min(p + 1, w) for p in range(kv - n, kv))
        keys += min(kv, w + n - 1) if n else 0
    return {"bytes": keys * held + 4 * new * case["Hq"] * d + (4 * new * case["Hq"] if case["lse"] else 0),
            "flops": 4 * pairs * case["Hq"] * d}


# ----------------------------------------------------------------------------------------------- exact
def _exact_rows(q, k, v, ok):
    x = (q @ k.T) / math.sqrt(q.shape[1])
    x[~ok] = -math.inf
    m = x.max(1, keepdim=True).values
    m[m == -math.inf] = 0
    p = (x - m).exp()
    l = p.sum(1, keepdim=True)
    return (p @ v) / torch.where(l == 0, 1, l), (m + l.log())[:, 0]


def _exact_token(st, n, s, t):
    """Cached tokens t of sequence s, float64 [Hkv, len(t), d]."""
    ps = st["case"]["page"]
    page = st["table"][s].long()[t // ps]
    x = st["p" + n][page, :, t % ps].double()
    return (x * st["s" + n][page, :, t % ps].double().unsqueeze(-1) if "s" + n in st else x).transpose(0, 1)


def exact(case, seed):
    st = _made(case, seed)
    dev, d, Hkv = st.get("q", st.get("k")).device, case["d"], case["Hkv"]
    f64 = dict(dtype=torch.float64, device=dev)
    if case["op"] == "cross":
        o = torch.zeros((case["B"], case["Hq"], case["Lq"], d), **f64)
        lse = torch.full(o.shape[:3], -math.inf, **f64)
        G = case["Hq"] // Hkv
        for b, n in enumerate(_key_lengths(case)):
            for h in range(case["Hq"] if n else 0):
                k, v = st["k"][b, h // G, :n].double(), st["v"][b, h // G, :n].double()
                o[b, h], lse[b, h] = _exact_rows(st["q"][b, h].double(), k, v, torch.ones((case["Lq"], n), dtype=torch.bool, device=dev))
        return (o, lse) if case["lse"] else o
    lens, starts = _lengths(case), st["q_start"].tolist()
    if case["op"] == "store":
        outs = []
        for n in "kv":
            o = torch.zeros((case["S"], Hkv, st["L"], d), **f64)
            for s, (new, kv) in enumerate(lens):
                f = int(st["first"][s])
                x = st[n][starts[s]:starts[s] + new].double()
                if case["pages"] == "int8":     # the codes are defined through two quotients rounded to fp32
                    sc = (x.abs().amax(-1, keepdim=True) / 127).float().double()
                    x = torch.where(sc > 0, (x / torch.where(sc > 0, sc, 1)).float().double().round() * sc, 0)
                old = _exact_token(st, n, s, torch.arange(f, kv - new, device=dev))
                o[s, :, :kv - f] = torch.cat([old, x.transpose(0, 1)], 1)
            outs.append(o)
        return tuple(outs)
    T, G = st["q"].shape[0], case["Hq"] // Hkv
    o, lse = torch.zeros((T, case["Hq"], d), **f64), torch.zeros((T, case["Hq"]), **f64)
    for s, (new, kv) in enumerate(lens):
        if new == 0:
            continue
        t = torch.arange(kv, device=dev)
        k, v = _exact_token(st, "k", s, t), _exact_token(st, "v", s, t)
        pos = torch.arange(kv - new, kv, device=dev)[:, None]
        ok = (t <= pos) & (t > pos - (case["window"] or kv))
        for h in range(case["Hq"]):
            r = slice(starts[s], starts[s] + new)
            o[r, h], lse[r, h] = _exact_rows(st["q"][r, h].double(), k[h // G], v[h // G], ok)
    return (o, lse) if case["lse"] else o
