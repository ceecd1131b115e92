"""Workloads of the operators that serve chunks of new tokens on the paged FP8 (E4M3) cache, and of the
per-head normalisation with rotation in front of it: their inputs, their plain forms in elementary torch
operations, their definitions in 64 bits, and what each cannot do without in bytes and operations.

    qk_norm_rope, qk_norm_rope_bwd   RMS norm of every query and key head, then the position rotation
    paged_append_fp8                 quantise a chunk of new tokens into the pages of their sequences
    paged_gather_fp8                 read a range of cached tokens back as bf16
    paged_index_scores_fp8           block scores of every new token against the cached index keys
    block_topk                       the selection from those scores
    paged_sparse_attn_fp8            attention of the new tokens over their selected pages
"""
import math

import torch

own = False

F8 = torch.float8_e4m3fn
BF = torch.bfloat16
INF = math.inf


def _case(name, op, **kw):
    c = {"op": op, **kw}
    return {"name": name, **c} if name else c


def listed():
    hd = dict(Hq=32, Hkv=4, dh=128)
    pg = dict(Hkv=4, dh=128, di=64, Bk=128)
    return [
        # one decode step of 64 sequences: a row of queries and keys each, half of the head rotated
        _case("norm_rope_decode", "rope", T=64, rot=64, far=131072, bwd=False, **hd),
        # a training step's forward and backward on one long packed batch, the whole head rotated
        _case("norm_rope_train", "rope", T=32768, rot=128, far=32768, bwd=True, **hd),
        # the cache write of a decode step
        _case("append_decode", "append", S=64, T=64, ctx=4000, **pg),
        # the cache write of a step that mixes prefill chunks of seven sequences
        _case("append_chunks", "append", S=7, T=8192, ctx=5000, **pg),
        # the prefixes of five sequences read back, as for moving them into a bf16 cache
        _case("gather_prefixes", "gather", S=5, T=65536, ctx=3000, **pg),
        # single tokens of 32 sequences against their whole index caches: bound by the cache's bytes
        _case("scores_decode", "scores", S=32, T=32, ctx=32700, **pg),
        # a chunk of two long prompts: bound by the products
        _case("scores_chunk", "scores", S=2, T=4096, ctx=61000, **pg),
        # the selection of those single tokens, and of a chunk at a 128K context
        _case("topk_decode", "topk", T=32, Hkv=4, blocks=257, Bk=128, k=16),
        _case("topk_chunk", "topk", T=4096, Hkv=4, blocks=1024, Bk=128, k=16),
        # attention of single tokens, of a few ragged chunks, and of a chunk of two long prompts
        _case("attend_decode", "attend", S=48, T=48, ctx=16000, Hq=32, Hkv=4, dh=128, Bk=128, k=16),
        _case("attend_ragged", "attend", S=5, T=777, ctx=9000, Hq=32, Hkv=4, dh=128, Bk=128, k=16),
        _case("attend_chunk", "attend", S=2, T=4096, ctx=61000, Hq=32, Hkv=4, dh=128, Bk=128, k=16),
    ]


def _log(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, n))


def draw(rng):
    """One more case: an operator, a head layout, and sizes over their whole range."""
    op = rng.choice(["rope", "rope", "append", "gather", "scores", "scores", "topk", "attend", "attend", "attend"])
    if op == "rope":
        dh = rng.choice([32, 64, 128])
        Hkv = rng.choice([1, 2, 4, 8])
        return _case(None, op, T=_log(rng, 1, 8192), rot=16 * rng.randint(0, dh // 16), far=_log(rng, 100, 1 << 20),
                     bwd=rng.random() < 0.5, Hq=Hkv * rng.choice([1, 2, 4, 7, 8]), Hkv=Hkv, dh=dh)
    if op == "topk":
        return _case(None, op, T=_log(rng, 1, 4096), Hkv=rng.choice([1, 2, 4]), blocks=_log(rng, 1, 1024),
                     Bk=rng.choice([64, 128]), k=rng.randint(1, 32))
    pg = dict(Hkv=rng.choice([1, 2, 4, 8]), dh=rng.choice([64, 128]), Bk=rng.choice([64, 128]))
    if op in ("append", "gather"):
        T = _log(rng, 1, 8192 if op == "append" else 40000)
        return _case(None, op, S=min(T, rng.randint(1, 40)), T=T, ctx=_log(rng, 10, 3000), di=rng.choice([64, 128]), **pg)
    if op == "scores":
        pg["Hkv"] = min(pg["Hkv"], 4)
        T = _log(rng, 1, 2000)
        return _case(None, op, S=min(T, rng.randint(1, 6)), T=T, ctx=_log(rng, 10, 20000), di=64, **pg)
    G = rng.choice([1, 2, 4, 8, 8, 16]) if pg["Hkv"] < 8 else rng.choice([1, 2, 4])
    T = _log(rng, 1, 1500)
    return _case(None, op, S=min(T, rng.randint(1, 24)), T=T, ctx=_log(rng, 10, 20000), Hq=G * pg["Hkv"],
                 k=rng.randint(1, 20), **pg)


# ---------------------------------------------------------------------------------------------- inputs


def _lengths(case, g):
    """(new tokens, cached tokens) of each sequence: single tokens where T == S, else ragged chunks."""
    S, T, ctx = case["S"], case["T"], case["ctx"]
    if T == S:
        new = torch.ones(S, dtype=torch.int64)
    else:
        cut = torch.sort(torch.randperm(T - 1, generator=g)[: S - 1] + 1).values
        new = torch.diff(torch.cat([torch.zeros(1, dtype=torch.int64), cut, torch.tensor([T])]))
    have = torch.randint(ctx // 2, ctx + 1, (S,), generator=g)
    have[0] = ctx
    return new, have


def _pages(case, g, new, have, index_only=False):
    """The pool, its page table and the offsets; every token's rows N(0, 1), quantised."""
    S, Bk, Hkv = case["S"], case["Bk"], case["Hkv"]
    need = (new + have + Bk - 1) // Bk
    # sized for any split of the chunk: a pool and a table are allocated once
    max_pages = -(-(case["ctx"] + case["T"]) // Bk)
    n_pages = (S * case["ctx"] + case["T"]) // Bk + S + 3
    free = torch.randperm(n_pages, generator=g)
    table = torch.zeros(S, max_pages, dtype=torch.int32)
    live = torch.arange(max_pages)[None, :] < need[:, None]
    table[live] = free[: int(need.sum())].to(torch.int32)
    gg = torch.Generator("cuda").manual_seed(int(torch.randint(1 << 40, (1,), generator=g)))

    def rows(*shape):
        x = torch.randn(*shape, generator=gg, device="cuda")
        s = x.abs().amax(-1) / 448
        return (x / s[..., None]).to(F8).view(torch.uint8), s

    st = {"table": table.cuda(), "S": S, "Bk": Bk}
    st["cu"] = torch.cat([torch.zeros(1, dtype=torch.int64), new.cumsum(0)]).to(torch.int32).cuda()
    st["len"] = have.to(torch.int32).cuda()
    if not index_only:
        st["kp"], st["ks"] = rows(n_pages, Bk, Hkv, case["dh"])
        st["vp"], st["vs"] = rows(n_pages, Bk, Hkv, case["dh"])
    if "di" in case:
        st["ip"], st["is"] = rows(n_pages, Bk, case["di"])
    return st, gg


def prepare(case, seed):
    g = torch.Generator().manual_seed(int(seed) * 7919 + 13)
    op = case["op"]
    if op == "rope":
        gg = torch.Generator("cuda").manual_seed(int(seed) + 101)
        T, Hq, Hk, d = case["T"], case["Hq"], case["Hkv"], case["dh"]

        def r(*shape):
            return torch.randn(*shape, generator=gg, device="cuda")

        st = {"q": (2 * r(T, Hq, d)).to(BF), "k": (3 * r(T, Hk, d)).to(BF), "wq": (1 + 0.2 * r(d)).to(BF),
              "wk": (1 + 0.2 * r(d)).to(BF), "rot": case["rot"], "theta": 5e6, "eps": 1e-6,
              "pos": torch.randint(0, case["far"], (T,), generator=gg, device="cuda", dtype=torch.int32)}
        if case["bwd"]:
            st["dq"], st["dk"] = r(T, Hq, d).to(BF), r(T, Hk, d).to(BF)
    elif op == "topk":
        gg = torch.Generator("cuda").manual_seed(int(seed) + 202)
        T, H, B = case["T"], case["Hkv"], case["blocks"]
        top = case["blocks"] * case["Bk"]
        first = max(0, top - T) if T > 64 else 0  # a chunk's positions follow one another; single tokens' do not
        pos = torch.arange(T, device="cuda") + first if T > 64 else torch.randint(0, top, (T,), generator=gg, device="cuda")
        pos = pos.clamp(max=top - 1).to(torch.int32)
        x = torch.randn(T, H, B, generator=gg, device="cuda")
        x[..., 0] += 2.0
        late = torch.arange(B, device="cuda")[None, None, :] >= (pos // case["Bk"])[:, None, None]
        st = {"scores": x.masked_fill_(late, -INF), "pos": pos, "Bk": case["Bk"], "k": case["k"]}
    else:
        new, have = _lengths(case, g)
        if op == "gather":
            start = torch.randint(0, case["ctx"] // 2 + 1, (case["S"],), generator=g)
            st, gg = _pages(case, g, new, start)
        else:
            st, gg = _pages(case, g, new, have, index_only=op == "scores")
        T = case["T"]
        st["T"] = T

        def rb(*shape):
            return torch.randn(*shape, generator=gg, device="cuda").to(BF)

        if op == "append":
            st.update(k=rb(T, case["Hkv"], case["dh"]), v=rb(T, case["Hkv"], case["dh"]), ki=rb(T, case["di"]))
        elif op == "scores":
            st["q"] = rb(T, case["Hkv"], case["di"])
        elif op == "attend":
            st["q"] = rb(T, case["Hq"], case["dh"])
            # selections as scored ones come out: the sink and the recent blocks more often than the others
            seq, pos = _where(st)
            B = st["table"].shape[1]
            ownb = (pos // case["Bk"])[:, None, None]
            b = torch.arange(B, device="cuda")[None, None, :]
            x = torch.randn(T, case["Hkv"], B, generator=gg, device="cuda") + 2.0 * (b == 0) + 1.5 * (ownb - b < 4)
            x = torch.where(b == ownb, INF, torch.where(b > ownb, -INF, x))
            n = min(case["k"], B)
            v, i = x.topk(n, -1)
            i = torch.where(v == -INF, B, i).sort(-1).values
            i = torch.where(i == B, -1, i)
            st["idx"] = torch.cat([i, i.new_full((T, case["Hkv"], case["k"] - n), -1)], -1).to(torch.int32)
    st["op"] = op
    return st


# ---------------------------------------------------------------------------------------------- plain forms


def _where(st):
    """Every new token's sequence and position."""
    t = torch.arange(st["T"], device="cuda")
    seq = torch.searchsorted(st["cu"][1:].long(), t, right=True)
    return seq, st["len"].long()[seq] + t - st["cu"].long()[seq]


def _rotate(x, cos, sin, n):
    a, b = x[..., :n], x[..., n : 2 * n]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., 2 * n :]], -1)


def _turns(st):
    n = st["rot"] // 2
    f = st["theta"] ** (-torch.arange(n, device="cuda", dtype=torch.float64) * 2 / max(1, st["rot"]))
    a = (st["pos"].double()[:, None] * f)[:, None, :]
    return a.cos().float(), a.sin().float(), n


def _rope(x, w, turns, eps):
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + eps)
    return _rotate(x * r * w.float(), *turns).to(BF)


def _rope_bwd(x, w, dy, turns, eps):
    cos, sin, n = turns
    x, w = x.float(), w.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + eps)
    g = _rotate(dy.float(), cos, -sin, n)
    nx = x * r
    wg = w * g
    dx = r * (wg - nx * (wg * nx).mean(-1, keepdim=True))
    return dx.to(BF), (g * nx).sum((0, 1))


def _quantise(x):
    x = x.float()
    amax = x.abs().amax(-1)
    s = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
    return (x / s[..., None]).to(F8).view(torch.uint8), s


def _run_rope(st):
    if own:
        import block_sparse_gqa_idx_b200 as msa

        kw = dict(rot_dim=st["rot"], theta=st["theta"], eps=st["eps"])
        out = list(msa.qk_norm_rope(st["q"], st["k"], st["wq"], st["wk"], st["pos"], **kw))
        if "dq" in st:
            out += msa.qk_norm_rope_bwd(st["q"], st["k"], st["wq"], st["wk"], st["pos"], st["dq"], st["dk"], **kw)
        return out
    turns = _turns(st)
    out = [_rope(st["q"], st["wq"], turns, st["eps"]), _rope(st["k"], st["wk"], turns, st["eps"])]
    if "dq" in st:
        dq, dwq = _rope_bwd(st["q"], st["wq"], st["dq"], turns, st["eps"])
        dk, dwk = _rope_bwd(st["k"], st["wk"], st["dk"], turns, st["eps"])
        out += [dq, dk, dwq, dwk]
    return out


def _run_append(st):
    if own:
        import block_sparse_gqa_idx_b200 as msa

        msa.paged_append_fp8(st["k"], st["v"], st["ki"], st["kp"], st["ks"], st["vp"], st["vs"], st["ip"], st["is"],
                             st["table"], st["cu"], st["len"])
    else:
        seq, pos = _where(st)
        page, slot = st["table"][seq, pos // st["Bk"]].long(), pos % st["Bk"]
        st["kp"][page, slot], st["ks"][page, slot] = _quantise(st["k"])
        st["vp"][page, slot], st["vs"][page, slot] = _quantise(st["v"])
        st["ip"][page, slot], st["is"][page, slot] = _quantise(st["ki"])
    return [st["kp"].view(F8), st["ks"], st["vp"].view(F8), st["vs"], st["ip"].view(F8), st["is"]]


def _run_gather(st):
    if own:
        import block_sparse_gqa_idx_b200 as msa

        return msa.paged_gather_fp8(st["kp"], st["ks"], st["vp"], st["vs"], st["ip"], st["is"], st["table"], st["cu"],
                                    st["len"], st["T"])
    seq, pos = _where(st)
    page, slot = st["table"][seq, pos // st["Bk"]].long(), pos % st["Bk"]
    return [(p[page, slot].view(F8).float() * s[page, slot][..., None]).to(BF)
            for p, s in ((st["kp"], st["ks"]), (st["vp"], st["vs"]), (st["ip"], st["is"]))]


def _run_scores(st):
    if own:
        import block_sparse_gqa_idx_b200 as msa

        return msa.paged_index_scores_fp8(st["q"], st["ip"], st["is"], st["table"], st["cu"], st["len"])
    T, H, d = st["q"].shape
    S, B, Bk = st["S"], st["table"].shape[1], st["Bk"]
    seq, pos = _where(st)
    t = torch.arange(T, device="cuda") - st["cu"].long()[seq]
    most = int((st["cu"][1:] - st["cu"][:-1]).max())
    q = torch.zeros(S, most, H, d, device="cuda")
    q[seq, t] = st["q"].float()
    page = st["table"].long()
    keys = (st["ip"][page].view(F8).float() * st["is"][page][..., None]).view(S, B * Bk, d)
    m = torch.bmm(q.view(S, most * H, d), keys.transpose(1, 2)).view(S, most, H, B, Bk).amax(-1)
    m = m[seq, t] / math.sqrt(d)
    return m.masked_fill(torch.arange(B, device="cuda")[None, None, :] >= (pos // Bk)[:, None, None], -INF)


def _run_topk(st):
    if own:
        import block_sparse_gqa_idx_b200 as msa

        return msa.block_topk(st["scores"], st["pos"], st["Bk"], st["k"])
    x, k = st["scores"], st["k"]
    T, H, B = x.shape
    ownb = (st["pos"].long() // st["Bk"])[:, None, None]
    b = torch.arange(B, device="cuda")[None, None, :]
    x = torch.where(b == ownb, INF, torch.where(b > ownb, -INF, x))
    v, i = torch.sort(x, dim=-1, descending=True, stable=True)
    v, i = v[..., :k], i[..., :k]
    i = torch.where(v == -INF, B, i).sort(-1).values
    i = torch.where(i == B, -1, i)
    return torch.cat([i, i.new_full((T, H, max(0, k - B)), -1)], -1).to(torch.int32)


def _run_attend(st):
    if own:
        import block_sparse_gqa_idx_b200 as msa

        return msa.paged_sparse_attn_fp8(st["q"], st["idx"], st["kp"], st["ks"], st["vp"], st["vs"], st["table"],
                                         st["cu"], st["len"])
    T, Hq, d = st["q"].shape
    H, k, Bk = st["ks"].shape[2], st["idx"].shape[2], st["Bk"]
    seq, pos = _where(st)
    idx = st["idx"].long()
    page = st["table"].long()[seq[:, None, None], idx.clamp(min=0)]
    head = torch.arange(H, device="cuda")[None, :, None]
    j = idx[..., None] * Bk + torch.arange(Bk, device="cuda")
    seen = ((idx >= 0)[..., None] & (j <= pos[:, None, None, None])).view(T, H, 1, k * Bk)

    def rows(p, s):
        x = p.permute(0, 2, 1, 3)[page, head].view(F8).float()
        return x.mul_(s.permute(0, 2, 1)[page, head][..., None]).view(T, H, k * Bk, d)

    q = st["q"].float().view(T, H, Hq // H, d)
    x = torch.matmul(q, rows(st["kp"], st["ks"]).transpose(2, 3)).mul_(1 / math.sqrt(d)).masked_fill_(~seen, -INF)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -INF, 0.0, top)
    p = (x - top).exp()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, rows(st["vp"], st["vs"])) / torch.where(total > 0, total, 1.0)
    return [o.view(T, Hq, d).to(BF), (top + total.log()).view(T, Hq)]


def run(state):
    return _RUN[state["op"]](state)


_RUN = {"rope": _run_rope, "append": _run_append, "gather": _run_gather, "scores": _run_scores, "topk": _run_topk,
        "attend": _run_attend}


# ---------------------------------------------------------------------------------------------- work


def _blocks(case):
    """(cached tokens over all sequences, new tokens of each): their mean over the seeds."""
    per = case["ctx"] * 0.75
    return case["ctx"] + (case["S"] - 1) * per, case["T"] / case["S"]


def work(case):
    op, T = case["op"], case["T"]
    if op == "rope":
        n = T * (case["Hq"] + case["Hkv"]) * case["dh"]
        return {"bytes": n * 2 * (5 if case["bwd"] else 2) + 4 * T, "flops": n * (24 if case["bwd"] else 8)}
    if op == "topk":
        # positions are the last ones of the blocks for a chunk, spread over them for single tokens
        B = case["blocks"] if T > 64 else case["blocks"] / 2
        return {"bytes": T * case["Hkv"] * (B + case["k"]) * 4, "flops": T * case["Hkv"] * B}
    row8 = 2 * case["Hkv"] * (case["dh"] + 4) + case.get("di", -4) + 4
    row16 = 2 * (2 * case["Hkv"] * case["dh"] + case.get("di", 0))
    if op in ("append", "gather"):
        return {"bytes": T * (row8 + row16), "flops": T * row16}
    ctx, new = _blocks(case)
    seen = case["S"] and ctx / case["S"] + new / 2
    if op == "scores":
        out = T * case["Hkv"] * -(-(case["ctx"] + T) // case["Bk"]) * 4
        return {"bytes": (ctx + T) * (case["di"] + 4) + T * case["Hkv"] * case["di"] * 2 + out,
                "flops": 2 * T * case["Hkv"] * seen * case["di"]}
    # attention: the keys that a token sees, and each page that any token of its sequence selects once
    keys = min(case["k"] * case["Bk"], seen)
    pages = min(ctx + T, T * keys) * case["Hkv"] * 2 * (case["dh"] + 4)
    return {"bytes": pages + T * case["Hq"] * (case["dh"] * 4 + 4) + T * case["Hkv"] * case["k"] * 4,
            "flops": 4 * T * case["Hq"] * keys * case["dh"]}


# ---------------------------------------------------------------------------------------------- 64 bits


def _e4m3(code):
    """The E4M3 values of uint8 codes, from the format's definition."""
    c = code.long()
    e, m = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e > 0, (1 + m / 8) * torch.pow(2.0, (e - 7).double()), m * 2.0**-9)
    mag = torch.where((c & 127) == 127, math.nan, mag)
    return torch.where(c >= 128, -mag, mag)


def _to_e4m3(x):
    """The nearest E4M3 values (ties to even) of numbers up to 448 in magnitude."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0**-30))).clamp(min=-6)
    step = torch.pow(2.0, e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _each(st):
    """(sequence, first row, rows, position of the first row) of every sequence."""
    cu, have = st["cu"].tolist(), st["len"].tolist()
    return [(s, cu[s], cu[s + 1] - cu[s], have[s]) for s in range(len(have))]


def _exact_rope(st):
    n, eps = st["rot"] // 2, st["eps"]
    rate = torch.tensor([math.pow(st["theta"], -2.0 * j / st["rot"]) for j in range(n)], dtype=torch.float64, device="cuda")
    angle = st["pos"].double()[:, None, None] * rate
    z = torch.polar(torch.ones_like(angle), angle)  # the rotation as a complex factor of each pair

    def turn(x, z):
        y = x.clone()
        c = torch.complex(x[..., :n].contiguous(), x[..., n : 2 * n].contiguous()) * z
        y[..., :n], y[..., n : 2 * n] = c.real, c.imag
        return y

    out, grads, sums = [], [], []
    for x, w, dy in (("q", "wq", "dq"), ("k", "wk", "dk")):
        x, w = st[x].double(), st[w].double()
        inv = (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + eps).pow(-0.5)
        out.append(turn(x * inv * w, z))
        if dy in st:
            g = turn(st[dy].double(), z.conj())
            sums.append((g * x * inv).flatten(0, 1).sum(0))
            dot = (g * w * x).sum(-1, keepdim=True) / x.shape[-1]
            grads.append(g * w * inv - x * dot * inv.pow(3))
    return out + grads + sums


def _exact_append(st):
    out = []
    for new, pool, scale in (("k", "kp", "ks"), ("v", "vp", "vs"), ("ki", "ip", "is")):
        val, sc = _e4m3(st[pool]), st[scale].double()
        x = st[new].double()
        most = x.abs().amax(-1)
        s = torch.where(most > 0, (most / 448).float().double(), 1.0)
        code = _to_e4m3((x / s[..., None]).float().double())  # the rule rounds the quotient to 32 bits first
        for q, row, n, at in _each(st):
            where = torch.arange(at, at + n, device="cuda")
            page, slot = st["table"][q].long()[where // st["Bk"]], where % st["Bk"]
            val[page, slot], sc[page, slot] = code[row : row + n], s[row : row + n]
        out += [val, sc]
    return out


def _exact_gather(st):
    out = []
    for pool, scale in (("kp", "ks"), ("vp", "vs"), ("ip", "is")):
        parts = []
        for q, _, n, at in _each(st):
            where = torch.arange(at, at + n, device="cuda")
            page, slot = st["table"][q].long()[where // st["Bk"]], where % st["Bk"]
            parts.append(_e4m3(st[pool][page, slot]) * st[scale][page, slot].double()[..., None])
        out.append(torch.cat(parts))
    return out


def _exact_scores(st):
    T, H, d = st["q"].shape
    B, Bk = st["table"].shape[1], st["Bk"]
    out = torch.full((T, H, B), -INF, dtype=torch.float64, device="cuda")
    for q, row, n, at in _each(st):
        full = (at + n - 1) // Bk  # blocks that any row of the sequence may score
        page = st["table"][q, :full].long()
        keys = (_e4m3(st["ip"][page]) * st["is"][page].double()[..., None]).reshape(full * Bk, d)
        for a in range(0, n, 256):
            b = min(n, a + 256)
            x = torch.einsum("thd,jd->thj", st["q"][row + a : row + b].double(), keys) * d**-0.5
            x = x.reshape(b - a, H, full, Bk).max(-1).values if full else x.reshape(b - a, H, 0)
            late = torch.arange(full, device="cuda") >= ((at + torch.arange(a, b, device="cuda")) // Bk)[:, None, None]
            out[row + a : row + b, :, :full] = torch.where(late, -INF, x)
    return out


def _exact_topk(st):
    x = st["scores"].cpu().numpy()
    pos = st["pos"].cpu().numpy()
    T, H, _ = x.shape
    out = torch.full((T, H, st["k"]), -1, dtype=torch.int32)
    for t in range(T):
        mine = int(pos[t]) // st["Bk"]
        order = (-x[t, :, :mine]).argsort(-1, kind="stable")[:, : st["k"] - 1]
        for h in range(H):
            got = sorted(int(b) for b in order[h] if x[t, h, b] > -INF) + [mine]
            out[t, h, : len(got)] = torch.tensor(got, dtype=torch.int32)
    return out


def _exact_attend(st):
    T, Hq, d = st["q"].shape
    H, k, Bk = st["ks"].shape[2], st["idx"].shape[2], st["Bk"]
    G = Hq // H
    o = torch.zeros(T, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((T, Hq), -INF, dtype=torch.float64, device="cuda")
    for s, row, n, at in _each(st):
        for h in range(H):
            live = st["table"][s, : (at + n + Bk - 1) // Bk].long()
            K = (_e4m3(st["kp"][live][:, :, h]) * st["ks"][live][:, :, h].double()[..., None]).reshape(-1, d)
            V = (_e4m3(st["vp"][live][:, :, h]) * st["vs"][live][:, :, h].double()[..., None]).reshape(-1, d)
            for a in range(row, row + n, 128):
                b = min(row + n, a + 128)
                pick = st["idx"][a:b, h].long()
                j = (pick.clamp(min=0)[..., None] * Bk + torch.arange(Bk, device="cuda")).reshape(b - a, k * Bk)
                ok = (pick >= 0).repeat_interleave(Bk, -1) & (j <= (at + torch.arange(a - row, b - row, device="cuda"))[:, None])
                j = torch.where(ok, j, 0)
                q = st["q"][a:b, h * G : (h + 1) * G].double()
                x = torch.einsum("tgd,tjd->tgj", q, K[j]) * d**-0.5
                x = torch.where(ok[:, None], x, -INF)
                z = torch.logsumexp(x, -1)
                w = torch.where(ok[:, None], torch.exp(x - torch.where(z == -INF, 0.0, z)[..., None]), 0.0)
                o[a:b, h * G : (h + 1) * G] = torch.einsum("tgj,tjd->tgd", w, V[j])
                lse[a:b, h * G : (h + 1) * G] = z
    return [o, lse]


_EXACT = {"rope": _exact_rope, "append": _exact_append, "gather": _exact_gather, "scores": _exact_scores,
          "topk": _exact_topk, "attend": _exact_attend}


def exact(case, seed):
    st = prepare(case, seed)
    return _EXACT[case["op"]](st)
