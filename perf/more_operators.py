"""Several continuations of one context over the paged 8-bit KV cache, as they are measured:
window attention that reads a group's shared prefix once, and the pages behind it: forking
requests, reserving room (with a copy of a page that others hold too), freeing, compacting.

A case is a dict of plain values; `prepare` makes its inputs on the GPU from a seed, `run` is
one pass: with `own` false in elementary torch operations, with `own` true through
`speculative_decoding_verify_temp_gb300.tsverify`. `exact` gives the same results in 64 bits.

Definitions (n(b) = ceil(seq_len[b] / page) table entries of request b; refcount[p] holders of
page p, free where it is not above 0; entries outside [0, pages) name no page):
  attention  of each window over its cached tokens and, causally or by a tree, over itself.
             Group g is the requests group_indptr[g] .. group_indptr[g+1] - 1; the whole pages
             among the first shared_lens[g] tokens are the same pages in all of its tables
  fork       request i of the result is a continuation of request sources[i]: its n entries
             (-1 behind them) and its length; each entry counts as one holder more
  reserve    room for new_lens[b] tokens. A request that grows and whose last page is partly
             filled and held more than once gets a copy of that page (codes of its tokens, and
             scales), unless every holder is such a request of this call and it is the last of
             them: that one keeps the page. Pages are given out in request order, the copy
             first, lowest free page first. A request is served iff the pages asked for up to
             and including it are there (or it asks for none and keeps no page in that way);
             one that is not served stays as it was. reserved[b]: new_lens[b], or seq_len[b]
  free       the entries of the released requests count one holder less
  compact    with n live pages, the k-th lowest live page at or above n moves to the k-th
             lowest free page below n; entries follow (-1: no live page, or behind the n(b))
"""
import math

import numpy as np
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
_F8 = torch.float8_e4m3fn


def listed():
    return [
        # latency: four answers to one short question
        dict(name="shared small", kind="attn", groups=1, n=4, T=1, ragged=False, Hq=8, Hkv=2, D=64,
             S=500, L=21, page=16, dtype="bf16", mask="chain"),
        # plain decoding of eight questions, up to sixteen answers each
        dict(name="shared answers", kind="attn", groups=8, n=16, T=1, ragged=False, Hq=32, Hkv=8, D=128,
             S=8200, L=501, page=16, dtype="bf16", mask="chain"),
        # drafted trees of up to 16 nodes, small heads
        dict(name="shared trees", kind="attn", groups=4, n=8, T=16, ragged=True, Hq=16, Hkv=4, D=64,
             S=20011, L=300, page=32, dtype="fp16", mask="tree"),
        # one very long document, many users, drafted chains
        dict(name="shared document", kind="attn", groups=1, n=32, T=8, ragged=False, Hq=64, Hkv=8, D=128,
             S=131071, L=700, page=64, dtype="bf16", mask="chain"),
        # two requests into four
        dict(name="fork small", kind="fork", B=2, n=4, L=90, page=16, share=1),
        # a full batch chosen anew from itself, long contexts in small pages
        dict(name="fork batch", kind="fork", B=512, n=512, L=30011, page=16, share=8),
        # four answers begin to differ
        dict(name="reserve small", kind="reserve", B=4, L=90, page=16, share=4, extra=5, Hkv=2, D=64),
        # many answers of many prompts begin to differ: hundreds of copies
        dict(name="reserve batch", kind="reserve", B=512, L=4007, page=64, share=8, extra=64, Hkv=8, D=128),
        # a few requests end
        dict(name="free small", kind="free", B=8, L=90, page=16, share=2),
        # half of a large batch ends
        dict(name="free batch", kind="free", B=512, L=30011, page=16, share=4),
        # a small pool
        dict(name="compact small", kind="compact", B=6, L=100, page=16, share=2, Hkv=2, D=64, hold=0.5),
        # a third of a large pool was freed
        dict(name="compact pool", kind="compact", B=64, L=8009, page=32, share=2, Hkv=8, D=128, hold=0.66),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))

    kind = rng.choice(("attn", "attn", "attn", "fork", "reserve", "free", "compact"))
    page = rng.choice((16, 32, 64, 128))
    if kind == "attn":
        c = dict(kind=kind, groups=log(1, 16), n=log(1, 64), T=log(1, 32), ragged=rng.random() < 0.4,
                 Hkv=rng.choice((1, 2, 4, 8)), D=rng.choice((64, 128)), S=log(1, 131071), L=log(1, 2000),
                 page=page, dtype=rng.choice(("bf16", "fp16")), mask=rng.choice(("none", "chain", "tree")))
        c["Hq"] = c["Hkv"] * rng.choice((1, 2, 4, 5, 7, 8))
        while c["groups"] * c["n"] * c["T"] * c["Hq"] * c["L"] > 2 ** 28:
            c[max(("groups", "n", "T"), key=lambda k: c[k])] //= 2
        while c["groups"] * c["n"] * c["T"] * c["Hq"] * c["S"] * c["D"] > 2 ** 37 or \
                c["groups"] * c["S"] * c["Hkv"] * c["D"] > 2 ** 28:
            c["S"] //= 2
        return c
    c = dict(kind=kind, B=log(1, 512), L=log(1, 30000), page=page, share=rng.choice((1, 2, 3, 4, 8)))
    if kind == "fork":
        c["n"] = log(1, 512)
    if kind in ("reserve", "compact"):
        c.update(Hkv=rng.choice((1, 2, 4, 8)), D=rng.choice((64, 128)))
        if kind == "reserve":
            c.update(extra=log(1, 300), short=rng.random() < 0.3)
        else:
            c["hold"] = rng.choice((0.2, 0.5, 0.8, 0.95))
        # the pool at most as large as the largest listed one
        while c["B"] * (c["L"] + 2 * page) * c["Hkv"] * c["D"] > 2 ** 28:
            c["L" if c["L"] > 300 else "B"] //= 2
    return c


# ---- sizes that follow from a case alone ------------------------------------------------

def _groups(c):
    """Requests of each group: between half of n and n."""
    return [c["n"] - (g * 5) % ((c["n"] + 1) // 2) for g in range(c["groups"])]


def _shared(c):
    """Tokens of each group's common context: between half of S and S."""
    return [c["S"] - (g * 7919) % (c["S"] // 2 + 1) for g in range(c["groups"])]


def _lens(c):
    """Cached tokens of each request."""
    if c["kind"] != "attn":  # `share` requests next to each other continue one context
        return [c["L"] - (b // c["share"] * 7919) % (c["L"] // 2 + 1) for b in range(c["B"])]
    of = [s for s, n in zip(_shared(c), _groups(c)) for _ in range(n)]
    return [s + c["L"] - (b * 7919) % (c["L"] // 2 + 1) for b, s in enumerate(of)]


def _windows(c):
    return [c["T"] - ((b * 13) % c["T"] if c["ragged"] else 0) for b in range(sum(_groups(c)))]


def _new_lens(c):
    """Half of the requests ask for a token, the others for up to `extra`; one in nine for none."""
    return [x + (0 if b % 9 == 8 else 1 if b % 2 else 1 + b * 31 % c["extra"]) for b, x in enumerate(_lens(c))]


def _ceil(a, b):
    return -(-a // b)


def _pool(c):
    """Pages held by the case's tables, pages of the pool, entries a table has room for."""
    n = c["page"]
    rows = [_ceil(x, n) for x in _lens(c)]
    wide = max(rows)
    if c["kind"] == "attn":
        whole = [s // n for s in _shared(c)]
        of = [s for s, k in zip(whole, _groups(c)) for _ in range(k)]
        held = sum(whole) + sum(r - s for r, s in zip(rows, of))
        return held, held + 3, wide
    held = sum(rows[::c["share"]])
    if c["kind"] == "reserve":
        new = [_ceil(x, n) for x in _new_lens(c)]
        most = sum(a - b for a, b in zip(new, rows)) + len(rows)
        return held, held + (most // 4 if c.get("short") else most + 3), max(new) + 1  # short: not enough for all
    if c["kind"] == "compact":
        return held, max(held, int(held / c["hold"])) + 1, wide
    return held, held + held // 4 + 3, wide


# ---- inputs -----------------------------------------------------------------------------

def _ints(v):
    return torch.tensor(np.asarray(v, np.int32), dtype=torch.int32, device="cuda")


def _indptr(v):
    return _ints([0] + list(np.cumsum(v)))


def _tables(c, seed):
    """Page tables in random order, and the holders of each page."""
    r = np.random.default_rng(seed)
    _, pages, wide = _pool(c)
    ids = r.permutation(pages).astype(np.int32)
    lens, n = _lens(c), c["page"]
    t = np.full((len(lens), wide), -1, np.int32)
    used = 0
    if c["kind"] == "attn":
        first = 0
        for s, k in zip(_shared(c), _groups(c)):
            t[first:first + k, : s // n] = ids[used:used + s // n]
            used += s // n
            for b in range(first, first + k):
                more = _ceil(lens[b], n) - s // n
                t[b, s // n: s // n + more] = ids[used:used + more]
                used += more
            first += k
    else:
        for b in range(0, len(lens), c["share"]):
            k = _ceil(lens[b], n)
            t[b:b + c["share"], :k] = ids[used:used + k]
            used += k
    count = np.bincount(t[t >= 0], minlength=pages)
    return _ints(t), _ints(count)


def _parents(c, windows, seed):
    """Drafted trees, packed: a node hangs on one of the few before it."""
    r = np.random.default_rng(seed)
    out = [np.maximum(np.arange(t) - 1 - (r.random(t) ** 2 * np.minimum(np.arange(t), 4)).astype(np.int64), 0) for t in windows]
    for p in out:
        p[0] = -1
    return _ints(np.concatenate(out))


def prepare(case, seed):
    c = case
    g = torch.Generator("cuda").manual_seed(seed)
    _, pages, _ = _pool(c)
    s = {"case": c, "seq_lens": _ints(_lens(c))}
    s["page_table"], s["refcount"] = _tables(c, seed)
    Hkv, D = c.get("Hkv", 1), c.get("D", 64)
    for name in ("k", "v"):
        x = torch.randn((pages, Hkv, c["page"], D), generator=g, device="cuda", dtype=torch.float16)
        s[name + "_cache"] = (x * 64).clamp_(-448, 448).to(_F8)
        s[name + "_scale"] = torch.exp2(torch.randint(-8, -4, (pages, Hkv), generator=g, device="cuda").float())
    if c["kind"] == "attn":
        dt, w = _DTYPES[c["dtype"]], _windows(c)
        n = sum(w)
        s["q"] = (torch.randn((n, c["Hq"], D), generator=g, device="cuda") * 1.5).to(dt)
        s["k_new"] = torch.randn((n, Hkv, D), generator=g, device="cuda").to(dt)
        s["v_new"] = torch.randn((n, Hkv, D), generator=g, device="cuda").to(dt)
        s["qo_indptr"], s["group_indptr"] = _indptr(w), _indptr(_groups(c))
        s["shared_lens"] = _ints(_shared(c))
        if c["mask"] == "tree":
            s["parents"] = _parents(c, w, seed)
        return s
    s["refcount_out"] = torch.empty_like(s["refcount"])
    r = np.random.default_rng(seed + 1)
    if c["kind"] == "fork":  # some sources more often than others, some not at all
        s["sources"] = _ints(np.minimum(r.random(c["n"]) ** 2 * c["B"], c["B"] - 1))
    elif c["kind"] == "reserve":
        s["new_lens"] = _ints(_new_lens(c))
    elif c["kind"] == "free":
        s["release"] = _ints(r.random(c["B"]) < 0.5)
    if c["kind"] in ("reserve", "compact"):
        s["table_out"] = torch.empty_like(s["page_table"])
    return s


# ---- the framework's calls --------------------------------------------------------------

def _run_own(s):
    from speculative_decoding_verify_temp_gb300 import tsverify as tv

    c = s["case"]
    cache = (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["page_table"], s["seq_lens"])
    if c["kind"] == "attn":
        new = {} if c["mask"] == "none" else dict(k_new=s["k_new"], v_new=s["v_new"])
        return tv.shared_attention(s["q"], *cache, group_indptr=s["group_indptr"], shared_lens=s["shared_lens"],
                                   qo_indptr=s["qo_indptr"], parents=s.get("parents"), lse=True, **new)
    counts = dict(refcount=s["refcount"], refcount_out=s["refcount_out"])
    if c["kind"] == "fork":
        return tv.kv_fork(*cache, sources=s["sources"], **counts)
    if c["kind"] == "free":
        return {"refcount": tv.kv_free(*cache, release=s["release"], **counts)}
    if c["kind"] == "reserve":
        out = tv.kv_reserve(*cache, new_lens=s["new_lens"], page_table_out=s["table_out"], **counts)
    else:
        out = tv.kv_compact(*cache, page_table_out=s["table_out"], **counts)
    return {**out, **{n: s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")}}


# ---- the plain forms --------------------------------------------------------------------

def _take8(x, pages):
    return x.view(torch.uint8)[pages].view(_F8).float()


def _gathered(s, name, pages):
    """Pages in the order of a [N, P] table, 32 bits: [N, Hkv, tokens, D]."""
    pages = pages.clamp(min=0)
    x = _take8(s[name + "_cache"], pages) * s[name + "_scale"][pages][..., None, None]
    N, P, H, n, D = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(N, H, P * n, D)


def _part(q, k, v, seen):
    """Softmax attention without its quotient: outputs, references, sums. seen: [N, rows, tokens]."""
    x = torch.matmul(q, k.transpose(2, 3)).masked_fill_(~seen[:, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-1e38)
    x = torch.exp_(x.sub_(m))
    return torch.matmul(x, v), m, x.sum(-1, keepdim=True)


def _plain_attn(s):
    c = s["case"]
    Hkv, D, G, n = c["Hkv"], c["D"], c["Hq"] // c["Hkv"], c["page"]
    dev = s["q"].device
    qo, gp = s["qo_indptr"].long(), s["group_indptr"].long()
    B = qo.numel() - 1
    q = s["q"].float().view(-1, Hkv, G, D).permute(1, 0, 2, 3) * (1.0 / math.sqrt(D))   # [Hkv, rows, G, D]

    def rows_of(first, count, most):
        """Rows of N windows or groups, [N, most], and which there are."""
        t = torch.arange(most, device=dev)
        inside = t < count[:, None]
        return (first[:, None] + t).clamp(max=q.shape[1] - 1), inside

    def packed(x, inside):
        """[N, Hkv, most * G, E] -> [Hkv, rows, G, E]"""
        N, _, _, E = x.shape
        return x.view(N, Hkv, -1, G, E).transpose(1, 2)[inside].transpose(0, 1)

    # the shared pages, once a group, for all rows of its requests
    whole = s["shared_lens"].long() // n                                        # pages
    most = max(_shared(c)) // n
    first, count = qo[gp[:-1]], qo[gp[1:]] - qo[gp[:-1]]
    at, inside = rows_of(first, count, c["n"] * c["T"])
    table = s["page_table"].long()
    there = (torch.arange(most * n, device=dev) < whole[:, None] * n)[:, None]
    pages = table[gp[:-1], :most]
    o0, m0, l0 = _part(q[:, at].permute(1, 0, 2, 3, 4).flatten(2, 3), _gathered(s, "k", pages),
                       _gathered(s, "v", pages), there) if most else (None, None, None)
    # the request's own pages, and its window
    group = torch.searchsorted(gp, torch.arange(B, device=dev), right=True) - 1
    skip = whole[group]
    T, wide = c["T"], c["L"] // n + 2
    cols = skip[:, None] + torch.arange(wide, device=dev)
    pages = table.gather(1, cols.clamp(max=table.shape[1] - 1))
    k, v = _gathered(s, "k", pages), _gathered(s, "v", pages)
    wat, win = rows_of(qo[:-1], qo[1:] - qo[:-1], T)
    seen = (torch.arange(wide * n, device=dev) < (s["seq_lens"].long() - skip * n)[:, None])[:, None].expand(B, T, wide * n)
    if c["mask"] != "none":
        t = torch.arange(T, device=dev)
        if c["mask"] == "tree":
            par = torch.where(win, s["parents"].long()[wat], torch.full_like(wat, -1))
            step = (par[:, :, None] == t).float() + torch.eye(T, device=dev)
            sees = torch.linalg.matrix_power(step, T) > 0            # itself and its ancestors
        else:
            sees = (t[:, None] >= t).expand(B, T, T)
        seen = torch.cat([seen, sees & win[:, None, :]], -1)
        k = torch.cat([k, s["k_new"].float()[wat].transpose(1, 2)], 2)
        v = torch.cat([v, s["v_new"].float()[wat].transpose(1, 2)], 2)
    o, m, l = _part(q[:, wat].permute(1, 0, 2, 3, 4).flatten(2, 3), k, v, seen.repeat_interleave(G, 1))
    o, m, l = packed(o, win), packed(m, win), packed(l, win)
    if most:
        o0, m0, l0 = packed(o0, inside), packed(m0, inside), packed(l0, inside)
        to = torch.maximum(m, m0)
        a, b = torch.exp(m - to), torch.exp(m0 - to)
        o, l, m = o * a + o0 * b, l * a + l0 * b, to
    out = (o / l).permute(1, 0, 2, 3).reshape(-1, c["Hq"], D)
    lse = (m + torch.log(l)).permute(1, 0, 2, 3).reshape(-1, c["Hq"])
    return {"out": out.to(s["q"].dtype), "lse": lse.contiguous()}


def _entries(s, lens):
    """Which table entries hold tokens, and which of them name a page."""
    t = s["page_table"]
    used = torch.arange(t.shape[1], device=t.device) < ((lens + s["case"]["page"] - 1) // s["case"]["page"])[:, None]
    return used, used & (t >= 0) & (t < s["refcount"].numel())


def _counted(s, pages, by):
    return s["refcount"].clone().index_add_(0, pages, torch.full_like(pages, by, dtype=torch.int32))


def _plain_fork(s):
    src = s["sources"].long()
    used, named = _entries(s, s["seq_lens"])
    t = torch.where(used, s["page_table"], -1)[src]
    return {"page_table": t, "seq_lens": s["seq_lens"][src], "refcount": _counted(s, t[named[src]].long(), 1)}


def _plain_free(s):
    _, named = _entries(s, s["seq_lens"])
    return {"refcount": _counted(s, s["page_table"][named & (s["release"] != 0)[:, None]].long(), -1)}


def _plain_reserve(s):
    c = s["case"]
    n, N = c["page"], s["refcount"].numel()
    t, count = s["page_table"].long(), s["refcount"].long()
    dev = t.device
    B, P = t.shape
    b = torch.arange(B, device=dev)
    at = torch.arange(P, device=dev)
    lens = s["seq_lens"].long()
    want = torch.maximum(lens, s["new_lens"].long().clamp(max=P * n))
    have, need = (lens + n - 1) // n, (want + n - 1) // n
    part = (want > lens) & (lens % n > 0)                          # writes to its last page
    last = t[b, (lens // n).clamp(max=P - 1)]
    part = part & (count[last.clamp(0, N - 1)] > 1) & (last >= 0) & (last < N)
    last = torch.where(part, last, torch.zeros_like(last))
    held = torch.zeros(N, dtype=torch.long, device=dev).index_add_(0, last, part.long())
    end = torch.full((N,), -1, dtype=torch.long, device=dev).scatter_reduce_(0, last, torch.where(part, b, -1), "amax")
    keeps = part & (held[last] >= count[last]) & (end[last] == b)
    copies = part & ~keeps
    ask = copies.long() + need - have
    upto = torch.cumsum(ask, 0)
    free = torch.nonzero(count <= 0).squeeze(1)
    served = (upto <= free.numel()) | ((ask == 0) & ~keeps)
    first = upto - ask                                             # number of the first page given
    copies = copies & served
    # the table: its entries, the copy in the place of the last, fresh pages behind
    number = (first + copies.long())[:, None] + at - have[:, None]
    fresh = served[:, None] & (at >= have[:, None]) & (at < need[:, None])
    pad = torch.cat([free, free.new_zeros(1)])
    out = torch.where(at < have[:, None], t, torch.full_like(t, -1))
    out = torch.where(fresh, pad[number.clamp(0, free.numel())], out)
    rows = torch.nonzero(copies).squeeze(1)
    to, come = pad[first[rows]], last[rows]
    out[rows, lens[rows] // n] = to
    now = count.clone().index_add_(0, come, torch.full_like(come, -1))
    now[out[fresh]] = 1
    now[to] = 1
    inside = torch.arange(n, device=dev) < (lens[rows] % n)[:, None]                       # [copies, n]
    res = {"page_table": out.to(torch.int32), "refcount": now.to(torch.int32),
           "reserved": torch.where(served, want, lens).to(torch.int32)}
    for name in ("k", "v"):
        x = s[name + "_cache"].view(torch.uint8)
        x[to] = torch.where(inside[:, None, :, None], x[come], x[to])
        s[name + "_scale"][to] = s[name + "_scale"][come]
        res[name + "_cache"], res[name + "_scale"] = s[name + "_cache"], s[name + "_scale"]
    return res


def _plain_compact(s):
    count = s["refcount"]
    N = count.numel()
    live = count > 0
    n = live.sum()
    at = torch.arange(N, device=count.device)
    come, to = torch.nonzero(live & (at >= n)).squeeze(1), torch.nonzero(~live & (at < n)).squeeze(1)
    place = torch.where(live, at, torch.full_like(at, -1))
    place[come] = to
    _, named = _entries(s, s["seq_lens"])
    t = torch.where(named, place[s["page_table"].long().clamp(0, N - 1)], -1)
    now = count.clone()
    now[to] = count[come]
    now[come] = 0
    res = {"page_table": t.to(torch.int32), "refcount": now, "live": n.to(torch.int32).view(1)}
    for name in ("k", "v"):
        x, sc = s[name + "_cache"].view(torch.uint8), s[name + "_scale"]
        x[to] = x[come]
        sc[to] = sc[come]
        res[name + "_cache"], res[name + "_scale"] = s[name + "_cache"], sc
    return res


def run(state):
    if own:
        return _run_own(state)
    return {"attn": _plain_attn, "fork": _plain_fork, "free": _plain_free, "reserve": _plain_reserve,
            "compact": _plain_compact}[state["case"]["kind"]](state)


# ---- in 64 bits, request by request -----------------------------------------------------

def _exact_attn(s):
    c = s["case"]
    G, n = c["Hq"] // c["Hkv"], c["page"]
    outs, lses, row = [], [], 0
    for b, (length, t) in enumerate(zip(_lens(c), _windows(c))):
        pages = s["page_table"][b, : _ceil(length, n)].long()
        kv = []
        for name in ("k", "v"):
            x = s[name + "_cache"].view(torch.uint8)[pages].view(_F8).double() * s[name + "_scale"][pages].double()[:, :, None, None]
            x = x.transpose(0, 1).flatten(1, 2)[:, :length]
            if c["mask"] != "none":
                x = torch.cat([x, s[name + "_new"][row:row + t].double().transpose(0, 1)], 1)
            kv.append(x)
        k, v = kv
        seen = np.ones((t, k.shape[1]), bool)
        if c["mask"] != "none":
            seen[:, length:] = np.tril(np.ones((t, t), bool))
            if c["mask"] == "tree":
                par = s["parents"][row:row + t].tolist()
                for i in range(t):
                    seen[i, length:] = seen[par[i], length:] if i else False
                    seen[i, length + i] = True
        seen = torch.from_numpy(seen).to(k.device)
        q = s["q"][row:row + t].double().view(t, c["Hkv"], G, c["D"]).permute(1, 2, 0, 3).flatten(1, 2)
        x = torch.matmul(q, k.transpose(1, 2)) / math.sqrt(c["D"])
        x.masked_fill_(~seen.repeat(G, 1), -math.inf)
        z = torch.logsumexp(x, -1, keepdim=True)
        o = torch.matmul(torch.exp(x - z), v).view(c["Hkv"], G, t, c["D"])
        outs.append(o.permute(2, 0, 1, 3).reshape(t, c["Hq"], c["D"]))
        lses.append(z.view(c["Hq"], t).T)
        row += t
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def _exact_pages(s):
    """Fork, free, reserve and compact with lists."""
    c = s["case"]
    n = c["page"]
    table, lens, count = s["page_table"].tolist(), s["seq_lens"].tolist(), s["refcount"].tolist()
    rows = [t[: _ceil(x, n)] for t, x in zip(table, lens)]
    wide = s["page_table"].shape[1]

    def whole(rows):
        return torch.tensor([r + [-1] * (wide - len(r)) for r in rows], dtype=torch.int32)

    if c["kind"] == "fork":
        src = s["sources"].tolist()
        times = np.bincount(src, minlength=len(rows))
        for r, k in zip(rows, times.tolist()):
            for p in r if k else ():
                count[p] += k
        return {"page_table": whole([rows[i] for i in src]), "seq_lens": torch.tensor([lens[i] for i in src]),
                "refcount": torch.tensor(count)}
    if c["kind"] == "free":
        for r, gone in zip(rows, s["release"].tolist()):
            for p in r if gone else ():
                count[p] -= 1
        return {"refcount": torch.tensor(count)}
    caches = {k: s[k].clone() for k in ("k_cache", "v_cache", "k_scale", "v_scale")}
    codes = [caches[k].view(torch.uint8) for k in ("k_cache", "v_cache")]
    scales = [caches[k] for k in ("k_scale", "v_scale")]
    if c["kind"] == "compact":
        live = [p for p, k in enumerate(count) if k > 0]
        holes = [p for p in range(len(live)) if count[p] <= 0]
        come = [p for p in live if p >= len(live)]
        place = {p: p for p in live}
        for a, b in zip(come, holes):
            place[a] = b
            count[b], count[a] = count[a], 0
        for x in codes + scales:
            x[holes] = x[come]
        return {"page_table": whole([[place.get(p, -1) for p in r] for r in rows]), "refcount": torch.tensor(count),
                "live": torch.tensor([len(live)]), **caches}
    free = [p for p, k in enumerate(count) if k <= 0]
    want = [max(a, min(b, wide * n)) for a, b in zip(lens, s["new_lens"].tolist())]
    writers = {}
    for b, (a, w) in enumerate(zip(lens, want)):
        if w > a and a % n and count[rows[b][-1]] > 1:
            writers.setdefault(rows[b][-1], []).append(b)
    keepers = {w[-1] for p, w in writers.items() if len(w) >= count[p]}
    copying = {b for w in writers.values() for b in w} - keepers
    reserved, asked, at = [], 0, 0
    for b, (a, w) in enumerate(zip(lens, want)):
        ask = (b in copying) + _ceil(w, n) - _ceil(a, n)
        asked += ask
        if asked > len(free) and (ask or b in keepers):
            reserved.append(a)
            continue
        reserved.append(w)
        given, at = free[at:at + ask], at + ask
        for p in given:
            count[p] = 1
        if b in copying:
            p, q = rows[b][-1], given.pop(0)
            count[p] -= 1
            for x in codes:
                x[q, :, : a % n] = x[p, :, : a % n]
            for x in scales:
                x[q] = x[p]
            rows[b] = rows[b][:-1] + [q]
        rows[b] = rows[b] + given
    return {"page_table": whole(rows), "refcount": torch.tensor(count), "reserved": torch.tensor(reserved), **caches}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_attn(s) if case["kind"] == "attn" else _exact_pages(s)


# ---- what a pass cannot do without ------------------------------------------------------

def work(case):
    c = case
    n = c["page"]
    lens = _lens(c)
    if c["kind"] == "attn":
        Hkv, D = c["Hkv"], c["D"]
        w, own_kv = _windows(c), 0 if c["mask"] == "none" else 1
        held, _, _ = _pool(c)
        of = [s // n * n for s, k in zip(_shared(c), _groups(c)) for _ in range(k)]
        tokens = sum(s // n * n for s in _shared(c)) + sum(x - s for x, s in zip(lens, of))
        pairs = sum(t * x + own_kv * t * (t + 1) // 2 for t, x in zip(w, lens))
        return {"bytes": float(tokens * Hkv * D * 2 + held * (Hkv * 8 + 4) + sum(w) * (c["Hq"] * (4 * D + 4) + own_kv * Hkv * D * 4)),
                "flops": 4.0 * pairs * c["Hq"] * D}
    held, pages, wide = _pool(c)
    entries = sum(_ceil(x, n) for x in lens)
    if c["kind"] == "fork":  # entries read once a source, rows written whole, counts read and written
        rows = min(c["n"], c["B"])
        return {"bytes": float(rows * (entries // len(lens)) * 4 + c["n"] * (wide + 2) * 4 + pages * 8), "flops": float(entries)}
    if c["kind"] == "free":
        return {"bytes": float(entries * 2 + len(lens) * 8 + pages * 8), "flops": float(entries)}
    block = c["Hkv"] * (n * c["D"] * 2 + 8)  # a page's codes and scales
    if c["kind"] == "compact":
        moved = held * (pages - held) / pages
        return {"bytes": float(2 * moved * block + (entries + len(lens) * wide) * 4 + pages * 8), "flops": float(entries)}
    # of each context the requests that grow copy, but for one where all holders grow
    grow = [w > x and x % n > 0 for w, x in zip(_new_lens(c), lens)]
    copied = 0
    for b in range(0, len(lens), c["share"]):
        k = grow[b:b + c["share"]]
        copied += (sum(k) - (1 if all(k) else 0) if len(k) > 1 else 0) * (lens[b] % n) / n
    return {"bytes": float(2 * copied * block + (entries + len(lens) * (wide + 3)) * 4 + pages * 8), "flops": float(entries)}
