"""Workloads of the paged history cache: attention of new events over it, and the
operators that move its rows and pages.

A user's history grows by a few events per request.  Its keys, values and
timestamps live in pages (`kv` [L, pages, 2, H, page, 64], `timestamps` [pages,
page]), found through a block table; forks of a user share pages by reference
count.  Five operators are timed:

  attn     Eq. 2 for the last c_u events of every user over all n_u cached ones:
           AV_i = sum_j phi2(q_i.k_j + rab_pos[h, min(i-j, P-1)]
                             + rab_time[h, bt(t_i - t_j)]) v_j / n_u
           over visible j <= i; with a window W, j > i - W or j < sinks;
           phi2 = softmax replaces phi2 and 1/n_u by a row-wise softmax
  append   the new events' K and V rows into their pages
  gather   whole users out of their pages into dense rows [L, T, 2, H, 64]
  branch   drop the last request's branches, fork new ones, reserve pages for
           their new events (copying the shared partial last page)
  compact  move the live pages into the lowest ids and rewrite the block table

`run` computes them with elementary torch operations, or with `own` set through
the package's entry points.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
TS_BASE = 1_700_000_000


# --------------------------------------------------------------------------- cases

def _attn(name, **kw):
    c = dict(op="attn", name=name, layers=1, window=0, sinks=0, P=4096, Tb=128, gaps="exp", phi2="silu")
    c.update(kw)
    return c


def listed():
    return [
        # one new event of one user with a short history: launch latency counts
        _attn("attn-one-event", dtype="bf16", batch=1, heads=4, page=16, ctx_lo=301, ctx_hi=301,
              new_lo=1, new_hi=1, P=512, shape=1),
        # a serving batch, one new event each, ragged histories: cache bandwidth counts
        _attn("attn-step-64-users", dtype="fp16", batch=64, heads=8, page=64, ctx_lo=700, ctx_hi=4096,
              new_lo=1, new_hi=1, shape=2),
        # softmax ablation, a handful of events since the last request
        _attn("attn-few-softmax", dtype="bf16", batch=24, heads=8, page=32, ctx_lo=100, ctx_hi=4096,
              new_lo=1, new_hi=37, phi2="softmax", shape=3),
        # lifelong histories read through a window with a profile prefix that stays visible
        _attn("attn-window", dtype="fp16", batch=16, heads=8, page=64, ctx_lo=9000, ctx_hi=16000,
              new_lo=64, new_hi=200, window=2048, sinks=100, P=8192, gaps="lognormal", shape=4),
        # a day's events of the long-sequence users (8192 events, 8 heads, log-normal gaps)
        _attn("attn-long-chunk", dtype="bf16", batch=8, heads=8, page=128, ctx_lo=8192, ctx_hi=8192,
              new_lo=512, new_hi=512, P=8192, gaps="lognormal", shape=5),
        # fp32 layers: small, one head
        _attn("attn-fp32", dtype="fp32", batch=12, heads=2, page=16, ctx_lo=30, ctx_hi=700,
              new_lo=1, new_hi=50, P=64, Tb=32, shape=6),
        # one event of every user of a serving batch
        dict(op="append", name="append-step", dtype="fp16", batch=64, heads=8, page=64, layers=4,
             ctx_lo=700, ctx_hi=4096, new_lo=1, new_hi=1, shape=7),
        # freshly encoded histories go into the cache
        dict(op="append", name="append-history", dtype="fp16", batch=8, heads=8, page=32, layers=2,
             ctx_lo=5000, ctx_hi=8192, new_lo=5000, new_hi=8192, shape=8),
        # histories out of the cache for candidate scoring (16 users, 4 layers)
        dict(op="gather", name="gather-history", dtype="fp16", batch=16, heads=8, page=64, layers=4,
             ctx_lo=2000, ctx_hi=4096, new_lo=0, new_hi=0, shape=9),
        # a few what-if branches of one user
        dict(op="branch", name="branch-one-user", dtype="fp16", batch=1, kids=4, heads=4, page=16, layers=2,
             ctx_lo=301, ctx_hi=301, new_lo=1, new_hi=3, shape=10),
        # eight branches of each user of a batch, 4 layers
        dict(op="branch", name="branch-batch", dtype="bf16", batch=32, kids=8, heads=8, page=64, layers=4,
             ctx_lo=500, ctx_hi=4096, new_lo=1, new_hi=90, shape=11),
        # a pool of which half the pages were freed here and there
        dict(op="compact", name="compact-pool", dtype="fp16", batch=48, heads=8, page=64, layers=4,
             ctx_lo=500, ctx_hi=4096, new_lo=0, new_hi=0, spare=1.0, shape=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn"] * 6 + ["append", "gather", "branch", "branch", "compact"])
    c = dict(op=op, dtype=rng.choice(["bf16", "fp16", "fp16"]), page=rng.choice([16, 32, 64, 128]),
             heads=rng.randint(1, 8), shape=rng.randint(100, 10**9))
    if op == "attn":
        fp32 = rng.random() < 0.15
        hi = _log_int(rng, 60, 600) if fp32 else _log_int(rng, 100, 12000)
        new = _log_int(rng, 1, min(hi, 600))
        pairs = 2.0e8 / (hi * new * c["heads"])  # below the long chunk's work
        c.update(layers=1, batch=max(1, min(_log_int(rng, 1, 64), int(pairs))), ctx_hi=hi,
                 ctx_lo=rng.randint(max(1, hi // 4), hi), new_hi=new, new_lo=rng.randint(1, new),
                 window=0, sinks=0, P=_log_int(rng, 16, 8192), Tb=rng.choice([32, 64, 128]),
                 gaps=rng.choice(["exp", "lognormal"]), phi2=rng.choice(["silu", "silu", "softmax", "relu"]))
        if fp32:
            c["dtype"] = "fp32"
        if rng.random() < 0.3:
            c.update(window=_log_int(rng, 1, hi), sinks=rng.choice([0, rng.randint(1, 200)]))
        return c
    hi = _log_int(rng, 50, 4096)
    c.update(layers=rng.randint(1, 4), batch=_log_int(rng, 1, 24), ctx_hi=hi,
             ctx_lo=rng.randint(max(1, hi // 4), hi), new_lo=0, new_hi=0)
    if op == "append":
        c.update(new_hi=_log_int(rng, 1, hi))
        c["new_lo"] = rng.randint(0, c["new_hi"])
    if op == "branch":
        c.update(kids=rng.randint(1, 8), new_lo=0, new_hi=_log_int(rng, 1, 200))
    if op == "compact":
        c.update(spare=rng.uniform(0.2, 2.0))
    return c


def _lengths(case):
    """(context lengths including the new events, new events) of every user, from the case alone."""
    r = random.Random(case["shape"])
    n = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["batch"])]
    if case["op"] == "branch":
        new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"] * case["kids"])]
    else:
        new = [min(a, r.randint(case["new_lo"], case["new_hi"])) for a in n]
    return n, new


def _offsets(counts):
    out = [0]
    for x in counts:
        out.append(out[-1] + x)
    return out


# --------------------------------------------------------------------------- inputs

def _relu_normal(shape, dtype, gen):
    """Rows of f1's output: ReLU of pre-activations of standard deviation 0.63 (Xavier weights)."""
    x = torch.empty(shape, dtype=dtype, device=DEV)
    x.normal_(0.0, 0.63, generator=gen)
    return x.clamp_(min=0.0)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed * 7919 + case["shape"])
    dt, H, ps, L = TYPES[case["dtype"]], case["heads"], case["page"], case["layers"]
    n, new = _lengths(case)
    B = case["batch"]
    blocks = [-(-x // ps) for x in n]
    kids = case.get("kids", 0)
    grown = max([0] + [n[c // kids] + x for c, x in enumerate(new)]) if kids else max(n)
    max_blocks = -(-max(max(n), grown) // ps) + 1
    used = sum(blocks)
    extra = sum(-(-(n[c // kids] + x) // ps) - blocks[c // kids] + 1 for c, x in enumerate(new)) if kids else 0
    pages = used + extra + 3 + int(case.get("spare", 0.0) * used)
    seqs = B * (1 + kids)
    # pages in no order, as a cache that has lived for a while has them
    perm = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((seqs, max_blocks), -1, dtype=torch.int32, device=DEV)
    at = 0
    for u, b in enumerate(blocks):
        table[u, :b] = perm[at:at + b]
        at += b
    ref = torch.zeros(pages, dtype=torch.int32, device=DEV)
    ref[perm[:used].long()] = 1
    st = {"case": dict(case), "kv": _relu_normal((L, pages, 2, H, ps, 64), dt, gen), "table": table, "ref": ref,
          "lengths": torch.tensor(n + [0] * (seqs - B), dtype=torch.int32, device=DEV),
          "offsets": torch.tensor(_offsets(new), dtype=torch.int64, device=DEV), "total": sum(new),
          "max_new": max([0] + new), "max_context": max(n)}
    # event times: increasing within a user, from its last event backwards through its pages
    nmax = max(n)
    gaps = torch.empty((B, nmax), dtype=torch.float64, device=DEV)
    if case.get("gaps", "exp") == "exp":
        gaps.exponential_(1.0 / 3600.0, generator=gen)
    else:
        gaps.log_normal_(7.0, 2.0, generator=gen)
    times = TS_BASE + gaps.cumsum(1).floor().to(torch.int64)
    ts = torch.zeros((pages, ps), dtype=torch.int64, device=DEV)
    b_i = torch.arange(nmax, device=DEV) // ps
    inside = torch.arange(nmax, device=DEV)[None, :] < st["lengths"][:B, None]
    page = table[:B].long().gather(1, b_i[None, :].expand(B, nmax))
    slot = (torch.arange(nmax, device=DEV) % ps)[None, :].expand(B, nmax)
    ts[page[inside], slot[inside]] = times[inside]
    st["timestamps"] = ts
    T = st["total"]
    counts = torch.tensor(new, device=DEV)
    row_user = torch.repeat_interleave(torch.arange(len(new), device=DEV), counts)
    r_in = torch.arange(T, device=DEV) - st["offsets"][:-1][row_user]
    if kids:
        st["src"] = torch.arange(B, dtype=torch.int32, device=DEV).repeat_interleave(kids)
        st["dst"] = torch.arange(B, seqs, dtype=torch.int32, device=DEV)
        last = times.gather(1, (st["lengths"][:B].long() - 1)[:, None])[:, 0]
        st["new_ts"] = last[st["src"].long()[row_user]] + 60 * (1 + r_in)
    else:
        pos = st["lengths"][:B].long()[row_user] - counts[row_user] + r_in
        st["new_ts"] = times[row_user, pos]
    if case["op"] == "attn":
        P, Tb = case["P"], case["Tb"]
        st["q"] = _relu_normal((T, H * 64), dt, gen)
        st["rab_pos"] = 0.02 * torch.randn((H, P), generator=gen, device=DEV)
        st["rab_time"] = 0.02 * torch.randn((H, Tb), generator=gen, device=DEV)
    if case["op"] == "append":
        # K and V as columns of one row buffer, as the projection leaves them
        st["rows"] = [_relu_normal((T, 2 * H * 64), dt, gen) for _ in range(L)]
    if case["op"] == "gather":
        st["all_offsets"] = torch.tensor(_offsets(n), dtype=torch.int64, device=DEV)
        st["all_total"] = sum(n)
    if case["op"] == "compact":
        st["table0"], st["ref0"] = table.clone(), ref.clone()
    return st


# --------------------------------------------------------------------------- plain forms

def _rows(st):
    """(user, position within the context) of every new row."""
    o = st["offsets"]
    T = st["total"]
    r = torch.arange(T, device=DEV)
    u = torch.searchsorted(o, r, right=True) - 1
    n, c = st["lengths"].long(), o[1:] - o[:-1]
    return u, n[u] - c[u] + (r - o[u])


def _attn_plain(st):
    case = st["case"]
    H, ps, P, Tb, nmax, cmax = case["heads"], case["page"], case["P"], case["Tb"], st["max_context"], st["max_new"]
    B, W, sinks = case["batch"], case["window"], case["sinks"]
    n, o = st["lengths"].long(), st["offsets"]
    c = o[1:] - o[:-1]
    j = torch.arange(nmax, device=DEV)
    page = st["table"].long()[:, j // ps].clamp(min=0)
    slot = (j % ps)[None, :].expand(B, nmax)
    k = st["kv"][0, :, 0].transpose(1, 2)[page, slot].float()  # [B, n, H, 64]
    v = st["kv"][0, :, 1].transpose(1, 2)[page, slot].float()
    t_k = st["timestamps"][page, slot]
    r = torch.arange(cmax, device=DEV)
    row = (o[:-1, None] + r[None, :]).clamp(max=st["total"] - 1)
    live = r[None, :] < c[:, None]
    q = st["q"].view(-1, H, 64)[row].float()  # [B, c, H, 64]
    i = n[:, None] - c[:, None] + r[None, :]
    t_q = st["new_ts"][row]
    dt = (t_q[:, :, None] - t_k[:, None, :]).clamp(min=0)
    bt = (torch.log(dt.double() + 1.0) / 0.301).floor().long().clamp(0, Tb - 1)
    dpos = i[:, :, None] - j
    s = torch.matmul(q.permute(0, 2, 1, 3), k.permute(0, 2, 3, 1))  # [B, H, c, n]
    s = s + st["rab_pos"][:, dpos.clamp(0, P - 1)].transpose(0, 1) + st["rab_time"][:, bt].transpose(0, 1)
    vis = (dpos >= 0) & live[:, :, None]
    if W:
        vis = vis & ((dpos < W) | (j < sinks))
    vis = vis[:, None]
    if case["phi2"] == "softmax":
        s = torch.where(vis, s, -math.inf)
        m = s.amax(-1, keepdim=True)
        e = torch.exp(s - torch.where(torch.isinf(m), 0.0, m))
        p = e / e.sum(-1, keepdim=True).clamp(min=1e-30)
    else:
        p = s / (1.0 + torch.exp(-s)) if case["phi2"] == "silu" else s.clamp(min=0.0)
        p = torch.where(vis, p, 0.0) / n[:, None, None, None].float()
    av = torch.matmul(p, v.transpose(1, 2)).transpose(1, 2)  # [B, c, H, 64]
    u, pos = _rows(st)
    return av[u, pos - (n[u] - c[u])].reshape(st["total"], H * 64).to(st["q"].dtype)


def _append_plain(st):
    ps, H = st["case"]["page"], st["case"]["heads"]
    u, pos = _rows(st)
    page, slot = st["table"].long()[u, pos // ps], pos % ps
    for l, rows in enumerate(st["rows"]):
        k, v = rows.view(-1, 2, H, 64).unbind(1)
        st["kv"][l, :, 0].transpose(1, 2)[page, slot] = k
        st["kv"][l, :, 1].transpose(1, 2)[page, slot] = v
    return st["kv"]


def _gather_plain(st):
    ps, H, L = st["case"]["page"], st["case"]["heads"], st["case"]["layers"]
    o, T = st["all_offsets"], st["all_total"]
    r = torch.arange(T, device=DEV)
    u = torch.searchsorted(o, r, right=True) - 1
    pos = r - o[u]
    page, slot = st["table"].long()[u, pos // ps], pos % ps
    return st["kv"].permute(0, 1, 4, 2, 3, 5)[:, page, slot].reshape(L, T, 2 * H * 64), st["timestamps"][page, slot]


def _branch_plain(st):
    ps = st["case"]["page"]
    table, ref, lens, kv, ts = st["table"], st["ref"], st["lengths"], st["kv"], st["timestamps"]
    src, dst = st["src"].long(), st["dst"].long()
    pages = ref.numel()
    # release the branches of the last request
    old = table[dst]
    ref.index_add_(0, old.clamp(min=0).flatten().long(), -(old >= 0).flatten().int())
    table[dst] = -1
    # fork: share every page
    rows = table[src]
    ref.index_add_(0, rows.clamp(min=0).flatten().long(), (rows >= 0).flatten().int())
    n = lens[src].long()
    # reserve: a private copy of a shared partial last page, then new pages, lowest free ids first
    c = st["offsets"][1:] - st["offsets"][:-1]
    have, want, fill = (n + ps - 1) // ps, (n + c + ps - 1) // ps, n % ps
    last = rows.gather(1, (have - 1).clamp(min=0)[:, None])[:, 0].long().clamp(min=0)
    cow = (c > 0) & (fill > 0) & (ref[last] > 1)
    need = want - have + cow.long()
    first = need.cumsum(0) - need
    free = torch.argsort((ref != 0).to(torch.int8), stable=True)
    b = torch.arange(rows.shape[1], device=DEV)[None, :]
    take = ((b >= have[:, None]) & (b < want[:, None])) | (cow[:, None] & (b == have[:, None] - 1))
    k = first[:, None] + b - have[:, None] + cow[:, None].long()
    given = free[k.clamp(0, pages - 1)]
    table[dst] = torch.where(take, given.int(), rows)
    ref.index_add_(0, given.flatten(), take.flatten().int())
    ref.index_add_(0, last, -cow.int())
    new = torch.where(cow, free[first.clamp(max=pages - 1)], last)
    keep = (torch.arange(ps, device=DEV)[None, :] < fill[:, None]) & cow[:, None]
    # rows that are not copied keep their value (a page that is no copy is copied onto itself)
    kv[:, new] = torch.where(keep[None, :, None, None, :, None], kv[:, last], kv[:, new])
    ts[new] = torch.where(keep, ts[last], ts[new])
    lens[dst] = (n + c).int()
    u = torch.repeat_interleave(torch.arange(dst.numel(), device=DEV), c, output_size=st["total"])
    pos = n[u] + torch.arange(st["total"], device=DEV) - st["offsets"][:-1][u]
    ts[table[dst].long()[u, pos // ps], pos % ps] = st["new_ts"]
    return {"table": table, "ref": ref, "lengths": lens, "kv": kv, "timestamps": ts}


def _compact_plain(st):
    table, ref, kv, ts = st["table"], st["ref"], st["kv"], st["timestamps"]
    table.copy_(st["table0"])
    ref.copy_(st["ref0"])
    pages = ref.numel()
    live, ids = ref > 0, torch.arange(pages, device=DEV)
    count = live.sum()
    moves, holes = live & (ids >= count), ~live & (ids < count)
    m = moves.sum()
    # the k-th live page past the end goes to the k-th hole; the others stay
    src = torch.argsort((~moves).to(torch.int8), stable=True)
    dst = torch.argsort((~holes).to(torch.int8), stable=True)
    to = torch.arange(pages + 1, device=DEV)
    to[torch.where(ids < m, src, pages)] = dst
    src = torch.where(ids < m, src, dst)
    kv[:, dst] = kv[:, src]
    ts[dst] = ts[src]
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].int(), table))
    ref[dst] = ref[src]
    ref.masked_fill_(ids >= count, 0)
    return {"table": table, "ref": ref, "kv": kv, "timestamps": ts, "live": count.int().view(1)}


# --------------------------------------------------------------------------- one pass

def _run_own(st):
    from hstu_sequential_transduction_jagged_b200 import hstu as M
    case = st["case"]
    cache = M.PagedCache(st["kv"], st["timestamps"], st["ref"], st["table"], st["lengths"])
    chunk = M.Jagged(st["offsets"], st["new_ts"], st["max_new"], st["total"])
    if case["op"] == "attn":
        cfg = M.LayerConfig(64 * case["heads"], case["heads"], case["P"], case["Tb"], phi2=case["phi2"],
                            dtype=case["dtype"])
        return M.paged_attn_fwd(cfg, cache, 0, chunk, st["q"], st["rab_pos"], st["rab_time"], st["max_context"],
                                window=case["window"], sinks=case["sinks"])
    if case["op"] == "append":
        hv = case["heads"] * 64
        for l, rows in enumerate(st["rows"]):
            M.cache_append(cache, l, chunk, rows[:, :hv], rows[:, hv:])
        return st["kv"]
    if case["op"] == "gather":
        return M.cache_gather(cache, st["all_offsets"], st["all_total"])
    if case["op"] == "branch":
        M.cache_release(cache, st["dst"])
        M.cache_fork(cache, st["src"], st["dst"])
        M.cache_reserve(cache, chunk, seq_ids=st["dst"])
        return {"table": st["table"], "ref": st["ref"], "lengths": st["lengths"], "kv": st["kv"],
                "timestamps": st["timestamps"]}
    st["table"].copy_(st["table0"])
    st["ref"].copy_(st["ref0"])
    live = M.cache_compact(cache)
    return {"table": st["table"], "ref": st["ref"], "kv": st["kv"], "timestamps": st["timestamps"], "live": live}


def run(state):
    if own:
        return _run_own(state)
    return {"attn": _attn_plain, "append": _append_plain, "gather": _gather_plain, "branch": _branch_plain,
            "compact": _compact_plain}[state["case"]["op"]](state)


# --------------------------------------------------------------------------- what a pass cannot do without

def _visible(n, c, W, sinks):
    """(visible pairs, keys that some row sees) of the last c of n events."""
    if not W:
        return sum(range(n - c + 1, n + 1)), n
    pairs = sum(min(W, i + 1) + min(sinks, max(0, i + 1 - W)) for i in range(n - c, n))
    lo = max(0, n - c + 1 - W)
    return pairs, n - lo + min(sinks, lo)


def work(case):
    n, new = _lengths(case)
    H, ps, L = case["heads"], case["page"], case["layers"]
    e = 4 if case["dtype"] == "fp32" else 2
    row = H * 64 * e
    if case["op"] == "attn":
        vis = [_visible(a, c, case["window"], case["sinks"]) for a, c in zip(n, new) if c]
        keys, rows = sum(k for _, k in vis), sum(new)
        return {"bytes": keys * (2 * row + 8) + rows * (2 * row + 8) + 4 * H * (case["P"] + case["Tb"]),
                "flops": 4 * 64 * H * sum(p for p, _ in vis)}
    if case["op"] == "append":
        return {"bytes": 4 * row * L * sum(new), "flops": 0}
    if case["op"] == "gather":
        return {"bytes": (4 * row * L + 16) * sum(n), "flops": 0}
    if case["op"] == "branch":
        kids = case["kids"]
        fill = sum(n[c // kids] % ps for c, x in enumerate(new) if x)
        tables = sum(-(-x // ps) for x in n) * kids
        return {"bytes": fill * (4 * row * L + 16) + 16 * sum(new) + 16 * tables, "flops": 0}
    used = sum(-(-x // ps) for x in n)
    pages = used + 3 + int(case["spare"] * used)
    moved = used - used * used / pages  # as many of the lowest ids are free, on average
    return {"bytes": moved * (4 * row * L * ps + 16 * ps) + 8 * used + 8 * pages, "flops": 0}


# --------------------------------------------------------------------------- from the definition, in 64 bits

def _user_rows(st, u, what):
    """All of a user's rows of `what(page)` ([..., page, x] per page), page after page."""
    ps, n = st["case"]["page"], int(st["lengths"][u])
    return torch.cat([what(int(p)) for p in st["table"][u, :-(-n // ps)].tolist()], -2)[..., :n, :]


def exact(case, seed):
    st = prepare(case, seed)
    H, ps = case["heads"], case["page"]
    n, new = _lengths(case)
    off = _offsets(new)
    if case["op"] == "attn":
        edges = torch.tensor([math.expm1(0.301 * k) for k in range(1, case["Tb"])], dtype=torch.float64, device=DEV)
        out = torch.zeros((sum(new), H, 64), dtype=torch.float64, device=DEV)
        for u, (a, c) in enumerate(zip(n, new)):
            kv = _user_rows(st, u, lambda p: st["kv"][0, p]).double()  # [2, H, n, 64]
            t = _user_rows(st, u, lambda p: st["timestamps"][p][:, None])[:, 0]
            for r0 in range(0, c, 128):
                r1 = min(c, r0 + 128)
                i = torch.arange(a - c + r0, a - c + r1, device=DEV)[:, None]
                j = torch.arange(a, device=DEV)[None, :]
                seen = j <= i
                if case["window"]:
                    seen &= (j > i - case["window"]) | (j < case["sinks"])
                bt = torch.bucketize((t[i] - t[j]).double(), edges, right=True)
                bp = (i - j).clamp(0, case["P"] - 1)
                for h in range(H):
                    q = st["q"][off[u] + r0:off[u] + r1, h * 64:h * 64 + 64].double()
                    s = q @ kv[0, h].T + st["rab_pos"][h].double()[bp] + st["rab_time"][h].double()[bt]
                    if case["phi2"] == "softmax":
                        w = torch.softmax(s.masked_fill(~seen, -math.inf), 1)
                    else:
                        w = (s * torch.sigmoid(s) if case["phi2"] == "silu" else torch.relu(s)) * seen / a
                    out[off[u] + r0:off[u] + r1, h] = w @ kv[1, h]
        return out.view(-1, H * 64)
    if case["op"] == "append":
        for u, (a, c) in enumerate(zip(n, new)):
            ids = st["table"][u].tolist()
            at = a - c
            while at < a:  # the rows of one page at a time
                take = min(ps - at % ps, a - at)
                r = off[u] + at - (a - c)
                for l, rows in enumerate(st["rows"]):
                    part = rows[r:r + take].view(take, 2, H, 64).permute(1, 2, 0, 3)
                    st["kv"][l, ids[at // ps], :, :, at % ps:at % ps + take] = part
                at += take
        return st["kv"].double()
    if case["op"] == "gather":
        users = [_user_rows(st, u, lambda p: st["kv"][:, p]) for u in range(case["batch"])]  # [L, 2, H, n, 64]
        rows = torch.cat([x.permute(0, 3, 1, 2, 4).reshape(case["layers"], -1, 2 * H * 64) for x in users], 1)
        return rows.double(), None
    # page numbers and copies of whole rows: nothing is computed
    return None
