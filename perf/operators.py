"""The operators around the verify step, as they are measured: window attention over a paged
8-bit KV cache, quantising accepted tokens into that cache and reading it back, and the
verification of a drafted tree.

A case is a dict of plain values; `prepare` makes its inputs on the GPU from a seed, `run` is
one pass: with `own` false in elementary torch operations, with `own` true through
`speculative_decoding_verify_temp_gb300.tsverify`. `exact` gives the same results in 64 bits.

Definitions (G = Hq / Hkv; a block is one page of one head):
  cache     value = e4m3 code * scale[page, head]; K and V each [pages, Hkv, page, D]
  attention row t of a request sees all seq_len cached tokens and, of the window's own K and
            V, the tokens 0..t (chain) or itself and its ancestors (tree)
  append    new token j of a request goes to position seq_len + j. The scale of a block is
            the power of two 2^e, e the least integer in [-60, 60] with max|x| <= 448 * 2^e
            over the new tokens in it; in a block that holds earlier tokens it is never
            lowered, and when it grows the earlier codes are rounded again to the new scale
  tree      a node's children are tried in index order: child x with coin u is accepted iff
            u * (1 - mass of the siblings rejected before) < p(x); when none is, the last
            token is drawn from p without the rejected children (coin: the root's)
"""
import math

import numpy as np
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_F8 = torch.float8_e4m3fn


def listed():
    return [
        # latency: one request, one token, a context that ends inside its third page
        dict(name="attn one short", kind="attn", B=1, T=1, ragged=False, Hq=8, Hkv=2, D=64, L=37,
             page=16, dtype="bf16", mask="chain"),
        # plain decoding of a full batch, contexts of different lengths
        dict(name="attn decode", kind="attn", B=64, T=1, ragged=False, Hq=32, Hkv=8, D=128,
             L=4096, page=16, dtype="bf16", mask="chain"),
        # verification of drafted chains (up to 4 drafts), packed windows of different lengths
        dict(name="attn chain ragged", kind="attn", B=128, T=5, ragged=True, Hq=32, Hkv=8, D=128,
             L=2003, page=32, dtype="fp16", mask="chain"),
        # verification of drafted trees: the largest number of rows a cached token meets
        dict(name="attn tree", kind="attn", B=16, T=32, ragged=False, Hq=64, Hkv=8, D=128,
             L=8191, page=64, dtype="bf16", mask="tree"),
        # two very long contexts: the work has to be split over the tokens
        dict(name="attn long", kind="attn", B=2, T=8, ragged=False, Hq=64, Hkv=8, D=128,
             L=131071, page=128, dtype="bf16", mask="chain"),
        # after a verify step: the accepted rows of each window go into the cache
        dict(name="append accepted", kind="append", B=128, T=5, Hkv=8, D=128, L=1000, page=16,
             dtype="bf16", accepted=True),
        # after a prompt: thousands of rows a request
        dict(name="append prompt", kind="append", B=3, T=8009, Hkv=8, D=128, L=21, page=64,
             dtype="fp16", accepted=False),
        # a few short prefixes back in 32 bits
        dict(name="read short", kind="read", B=8, Hkv=2, D=64, L=45, page=16, dtype="fp32"),
        # long prefixes back in 16 bits, for a prompt that continues them
        dict(name="read prefix", kind="read", B=4, Hkv=8, D=128, L=20011, page=32, dtype="bf16"),
        # a tree of 8 nodes over a small vocabulary: latency
        dict(name="tree small", kind="tree", B=4, T=8, V=1024, width=2),
        # trees of 32 nodes
        dict(name="tree", kind="tree", B=64, T=32, V=128256, width=3),
        # a large batch of small trees
        dict(name="tree batch", kind="tree", B=256, T=8, V=151936, width=2),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))

    kind = rng.choice(("attn", "attn", "append", "read", "tree"))
    if kind == "tree":
        c = dict(kind=kind, B=log(1, 256), T=log(1, 64), V=log(100, 200019), width=rng.randint(1, 4))
        while c["B"] * c["T"] * c["V"] > 256 * 8 * 151936:
            c["B"] = max(1, c["B"] // 2)
            c["T"] = max(1, c["T"] - 3) if c["B"] == 1 else c["T"]
        return c
    c = dict(kind=kind, B=log(1, 128), Hkv=rng.choice((1, 2, 4, 8)), D=rng.choice((64, 128)),
             L=log(1, 100000), page=rng.choice((16, 32, 64, 128)),
             dtype=rng.choice(("bf16", "fp16")))
    if kind == "attn":
        c.update(T=log(1, 64), ragged=rng.random() < 0.4, mask=rng.choice(("none", "chain", "tree")))
        c["Hq"] = c["Hkv"] * rng.choice((1, 2, 4, 5, 7, 8))
        while c["B"] * c["Hkv"] * c["L"] * c["D"] > 2 ** 28 or \
                c["B"] * c["Hq"] * c["T"] * c["L"] * c["D"] > 2 ** 35:
            c["L" if c["L"] > 500 else "B"] = max(1, c["L" if c["L"] > 500 else "B"] // 2)
    elif kind == "append":
        c.update(accepted=rng.random() < 0.5, L=log(1, 2000))
        c["T"] = log(1, 64) if c["accepted"] else log(1, 8000)
        while c["B"] * c["T"] * c["Hkv"] * c["D"] > 3 * 2 ** 23:
            c["B"] = max(1, c["B"] // 2)
            c["T"] = max(1, c["T"] // 2) if c["B"] == 1 else c["T"]
        c["dtype"] = rng.choice(("bf16", "fp16", "fp32"))
    else:
        while c["B"] * c["L"] * c["Hkv"] * c["D"] > 2 ** 26:
            c["B" if c["B"] > 1 else "L"] //= 2
        c["dtype"] = rng.choice(("bf16", "fp16", "fp32"))
    return c


# ---- sizes that follow from a case alone ------------------------------------------------

def _lens(c):
    """Cached tokens of each request: between half of L and L."""
    return [c["L"] - (b * 7919) % (c["L"] // 2 + 1) for b in range(c["B"])]


def _windows(c):
    """Rows of each request's window."""
    if c["kind"] == "append":  # rows offered: all of a prompt, or the window verified
        return [c["T"] - (0 if c["accepted"] else (b * 31) % (c["T"] // 2 + 1)) for b in range(c["B"])]
    return [c["T"] - ((b * 13) % c["T"] if c["ragged"] else 0) for b in range(c["B"])]


def _taken(c):
    """Rows of each request that an append stores."""
    return [1 + (b * 5) % t if c["accepted"] else t for b, t in enumerate(_windows(c))]


def _extent(c):
    """Tokens a request's page table has room for."""
    if c["kind"] == "append":
        return max(x + t for x, t in zip(_lens(c), _taken(c)))
    return c["L"]


# ---- inputs -----------------------------------------------------------------------------

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _indptr(v):
    return _ints([0] + list(np.cumsum(v)))


def _cache(c, g):
    """Pages with e4m3 codes and power-of-two scales, and a page table in random order."""
    per = -(-_extent(c) // c["page"])
    n = c["B"] * per + 3
    s = {"page_table": torch.randperm(n, generator=g, device="cuda")[: c["B"] * per].to(torch.int32).view(c["B"], per)}
    for name in ("k", "v"):
        x = torch.randn((n, c["Hkv"], c["page"], c["D"]), generator=g, device="cuda", dtype=torch.float16)
        s[name + "_cache"] = (x * 64).clamp_(-448, 448).to(_F8)
        s[name + "_scale"] = torch.exp2(torch.randint(-8, -4, (n, c["Hkv"]), generator=g, device="cuda").float())
    s["seq_lens"] = _ints(_lens(c))
    return s


def _parents(c, seed):
    """Trees in index order: node i hangs on a node before it that has fewer than `width` children."""
    r = np.random.default_rng(seed)
    width = c.get("width", 3)
    out = np.full((c["B"], c["T"]), -1, np.int64)
    left = np.zeros((c["B"], c["T"]), np.int64)
    left[:, 0] = width
    rows = np.arange(c["B"])
    for i in range(1, c["T"]):
        # a recent open node more often than an early one, so that trees are deep
        score = r.random((c["B"], i)) ** (1.0 / (1.0 + np.arange(i)))
        p = np.where(left[:, :i] > 0, score, -1.0).argmax(1)
        out[:, i] = p
        left[rows, p] -= 1
        left[:, i] = width
    return torch.from_numpy(out).to("cuda", torch.int32)


def prepare(case, seed):
    c = case
    g = torch.Generator("cuda").manual_seed(seed)
    s = {"case": c}
    if c["kind"] == "tree":
        B, T, V = c["B"], c["T"], c["V"]
        x = torch.randn((B * T, V), generator=g, device="cuda") * 3
        x -= 1.1 * torch.log(torch.arange(1, V + 1, device="cuda", dtype=torch.float32))
        p = torch.softmax(x, -1)
        del x
        s["probs"] = p
        parents = _parents(c, seed)
        par = parents.long()
        before = torch.ones(T, T, dtype=torch.bool, device="cuda").tril(-1)
        rank = ((par[:, :, None] == par[:, None, :]) & before).sum(-1)
        top = torch.topk(p, min(8, V), dim=-1).indices.view(B, T, -1)
        likely = top[torch.arange(B, device="cuda")[:, None], par.clamp(min=0), rank.clamp(max=top.shape[-1] - 1)]
        other = torch.randint(0, V, (B, T), generator=g, device="cuda")
        pick = torch.rand((B, T), generator=g, device="cuda") < 0.8
        s["tokens"] = torch.where(pick, likely, other).to(torch.int32)
        s["parents"] = parents
        k = torch.randint(0, 1 << 23, (B, T), generator=g, device="cuda")
        s["uniforms"] = ((2 * k + 1).double() * 2.0 ** -24).float()
        return s
    s.update(_cache(c, g))
    B, Hkv, D = c["B"], c["Hkv"], c["D"]
    if c["kind"] == "attn":
        dt = _DTYPES[c["dtype"]]
        w = _windows(c)
        n = sum(w)
        s["q"] = (torch.randn((n, c["Hq"], D), generator=g, device="cuda") * 1.5).to(dt)
        s["k_new"] = torch.randn((n, Hkv, D), generator=g, device="cuda").to(dt)
        s["v_new"] = torch.randn((n, Hkv, D), generator=g, device="cuda").to(dt)
        s["qo_indptr"] = _indptr(w)
        if c["mask"] == "tree":
            full = _parents(c, seed)
            s["parents"] = torch.cat([full[b, :t] for b, t in enumerate(w)]).contiguous()
    elif c["kind"] == "append":
        dt = _DTYPES[c["dtype"]]
        w, taken = _windows(c), _taken(c)
        # some tokens much larger than the rest, as keys and values have them: the scales grow
        big = torch.exp2(torch.randint(-2, 3, (sum(w), Hkv, 1), generator=g, device="cuda").float())
        s["k"] = (torch.randn((sum(w), Hkv, D), generator=g, device="cuda") * big).to(dt)
        s["v"] = (torch.randn((sum(w), Hkv, D), generator=g, device="cuda") * big).to(dt)
        if c["accepted"]:
            # the accepted path of each window: increasing rows, the window's first among them
            r = np.random.default_rng(seed)
            idx = np.full((B, c["T"]), -1, np.int32)
            for b, (t, a) in enumerate(zip(w, taken)):
                idx[b, :a] = b * c["T"] + np.concatenate([[0], 1 + np.sort(r.permutation(t - 1)[: a - 1])])
            s["src_index"] = torch.from_numpy(idx).cuda()
            s["src_len"] = _ints(taken)
        else:
            s["qo_indptr"] = _indptr(w)
    else:
        s["out_indptr"] = _indptr(_lens(c))
        s["total"] = sum(_lens(c))
    return s


# ---- the framework's calls --------------------------------------------------------------

def _run_own(s):
    from speculative_decoding_verify_temp_gb300 import tsverify as tv

    c = s["case"]
    if c["kind"] == "tree":
        return tv.tree_spec_sampling(s["probs"], c["T"] - 1, s["tokens"], s["parents"], s["uniforms"])
    cache = (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["page_table"], s["seq_lens"])
    if c["kind"] == "attn":
        new = {} if c["mask"] == "none" else dict(k_new=s["k_new"], v_new=s["v_new"])
        return tv.window_attention(s["q"], *cache, qo_indptr=s["qo_indptr"], parents=s.get("parents"),
                                   lse=True, **new)
    if c["kind"] == "append":
        tv.kv_append(s["k"], s["v"], *cache, qo_indptr=s.get("qo_indptr"), src_index=s.get("src_index"),
                     src_len=s.get("src_len"))
        return {n: s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")}
    return tv.kv_read(*cache, out_indptr=s["out_indptr"], total_rows=s["total"], dtype=_DTYPES[c["dtype"]])


# ---- the plain forms --------------------------------------------------------------------

def _take8(x, pages):
    return x.view(torch.uint8)[pages].view(_F8).float()


def _gathered(s, name):
    """A cache in page-table order, 32 bits: [B, Hkv, tokens, D]."""
    pages = s["page_table"].long()
    x = _take8(s[name + "_cache"], pages) * s[name + "_scale"][pages][..., None, None]
    B, P, H, n, D = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(B, H, P * n, D)


def _plain_attn(s):
    c = s["case"]
    B, Hkv, D, G = c["B"], c["Hkv"], c["D"], c["Hq"] // c["Hkv"]
    dev = s["q"].device
    k, v = _gathered(s, "k"), _gathered(s, "v")
    qo = s["qo_indptr"].long()
    w = qo[1:] - qo[:-1]
    T = c["T"]
    t = torch.arange(T, device=dev)
    inside = t < w[:, None]                                      # [B, T]
    rows = (qo[:-1, None] + t).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float()[rows].view(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D)
    scale = 1.0 / math.sqrt(D)
    cached = torch.arange(k.shape[2], device=dev) < s["seq_lens"][:, None]   # [B, tokens]
    x = (torch.matmul(q, k.transpose(2, 3)) * scale).masked_fill(~cached[:, None, None], -math.inf)
    if c["mask"] != "none":
        kn = s["k_new"].float()[rows].transpose(1, 2)            # [B, Hkv, T, D]
        vn = s["v_new"].float()[rows].transpose(1, 2)
        if c["mask"] == "tree":
            par = torch.full((B, T), -1, dtype=torch.long, device=dev)
            par = torch.where(inside, s["parents"].long()[rows], par)
            step = (par[:, :, None] == t).float() + torch.eye(T, device=dev)
            sees = torch.linalg.matrix_power(step, T) > 0        # itself and its ancestors
        else:
            sees = (t[:, None] >= t).expand(B, T, T)
        sees = sees & inside[:, None, :]
        y = (torch.matmul(q, kn.transpose(2, 3)) * scale).view(B, Hkv, T, G, T)
        y = y.masked_fill(~sees[:, None, :, None, :], -math.inf).view(B, Hkv, T * G, T)
        x, v = torch.cat([x, y], -1), torch.cat([v, vn], 2)
    m = x.amax(-1, keepdim=True).clamp(min=-1e38)
    e = torch.exp(x - m)
    z = e.sum(-1, keepdim=True)
    o = torch.matmul(e, v) / z
    lse = (m + torch.log(z)).squeeze(-1)

    def packed(a):
        a = a.reshape(B, Hkv, T, G, -1).permute(0, 2, 1, 3, 4).reshape(B * T, c["Hq"], -1)
        return a[inside.reshape(-1)]

    return {"out": packed(o).to(s["q"].dtype), "lse": packed(lse[..., None]).squeeze(-1)}


def _plain_append(s):
    c = s["case"]
    dev = s["k"].device
    B, n = c["B"], c["page"]
    lens = s["seq_lens"].long()
    if c["accepted"]:
        count, j = s["src_len"].long(), torch.arange(c["T"], device=dev)
        rows = s["src_index"].long()
    else:
        qo = s["qo_indptr"].long()
        count, j = qo[1:] - qo[:-1], torch.arange(c["T"], device=dev)
        rows = qo[:-1, None] + j
    new = j < count[:, None]
    b = torch.arange(B, device=dev)[:, None].expand_as(new)[new]
    rows = rows.expand_as(new)[new]
    pos = (lens[:, None] + j)[new]
    page, slot = s["page_table"].long()[b, pos // n], pos % n
    out = {}
    for name in ("k", "v"):
        cache, sc = s[name + "_cache"], s[name + "_scale"]
        x = s[name].float()[rows]                               # [tokens, Hkv, D]
        top = torch.zeros(sc.shape, device=dev)
        top.index_reduce_(0, page, x.abs().amax(-1), "amax")
        frac, e = torch.frexp(top)
        e = torch.where(frac > 0.875, e - 8, e - 9).clamp(-60, 60)
        e = torch.where(top > 0, e, torch.full_like(e, -60))
        need = torch.exp2(e.float())
        # blocks written now: those with tokens from before keep at least their scale
        slots = torch.arange(n, device=dev)
        touched = torch.zeros(sc.shape[0], dtype=torch.bool, device=dev)
        touched[page] = True
        at = torch.arange(s["page_table"].shape[1], device=dev)
        fill = torch.zeros(sc.shape[0], dtype=torch.long, device=dev)
        fill[s["page_table"].long()] = (lens[:, None] - at * n).clamp(0, n)
        held = touched & (fill > 0)
        scale = torch.where(held[:, None], torch.maximum(sc, need), need)
        scale = torch.where(touched[:, None], scale, sc)
        # only the pages whose scale grew are rounded again, only their earlier tokens
        p = torch.nonzero((held[:, None] & (scale > sc)).any(1)).squeeze(1)
        old = _take8(cache, p)
        again = (old * (sc[p] / scale[p])[..., None, None]).to(_F8).float()
        earlier = (slots < fill[p][:, None])[:, None, :, None]
        cache.view(torch.uint8)[p] = torch.where(earlier, again, old).to(_F8).view(torch.uint8)
        y = (x / scale[page][..., None]).clamp(-448, 448).to(_F8)
        h = torch.arange(c["Hkv"], device=dev)
        cache.view(torch.uint8)[page[:, None], h, slot[:, None]] = y.view(torch.uint8)
        sc.copy_(scale)
        out[name + "_cache"], out[name + "_scale"] = cache, sc
    return out


def _plain_read(s):
    c = s["case"]
    ptr = s["out_indptr"].long()
    i = torch.arange(s["total"], device=ptr.device)
    b = torch.searchsorted(ptr, i, right=True) - 1
    pos = i - ptr[b]
    page, slot = s["page_table"].long()[b, pos // c["page"]], pos % c["page"]
    out = {}
    for name in ("k", "v"):
        x = s[name + "_cache"].view(torch.uint8)[page, :, slot].view(_F8).float()
        out[name] = (x * s[name + "_scale"][page][..., None]).to(_DTYPES[c["dtype"]])
    return out


def _plain_tree(s):
    c = s["case"]
    B, T, V = c["B"], c["T"], c["V"]
    p, tok, u = s["probs"].view(B, T, V), s["tokens"].long(), s["uniforms"].double()
    par = s["parents"].long()
    dev = p.device
    b = torch.arange(B, device=dev)
    i = torch.arange(T, device=dev)
    sib = (par[:, :, None] == par[:, None, :]) & (i[:, None] > i) & (par >= 0)[:, :, None]
    px = p[b[:, None], par.clamp(min=0), tok].double()
    px = torch.where((sib & (tok[:, :, None] == tok[:, None, :])).any(-1), torch.zeros_like(px), px)
    gone = (sib * px[:, None, :]).sum(-1)                        # mass of the siblings before
    test = (u * (1 - gone) < px) & (par >= 0)
    taken = test & ~(sib & test[:, None, :]).any(-1)             # the first sibling that passes
    up = (par[:, :, None] == i).float() + torch.eye(T, device=dev)
    above = torch.linalg.matrix_power(up, T) > 0                 # [B, node, ancestor or itself]
    root = i == 0
    path = (~above | (taken | root)[:, None, :]).all(-1) & above[:, :, 0]
    depth = above.sum(-1) - 1
    length = path.sum(-1)                                        # nodes kept, the root among them
    at = torch.where(path, depth, torch.full_like(depth, T))     # position of each kept node
    node = torch.zeros((B, T + 1), dtype=torch.long, device=dev).scatter(1, at, i.expand(B, T))[:, :T]
    end = node.gather(1, (length - 1)[:, None]).squeeze(1)
    w = p[b, end].double()
    full = w.clone()
    child = (par == end[:, None]) & (i > 0)
    w[b[:, None].expand(B, T)[child], tok[child]] = 0
    w = torch.where(w.sum(-1, keepdim=True) > 0, w, full)
    mass = torch.cumsum(w, -1)
    last = (mass <= u[:, :1] * mass[:, -1:]).sum(-1).clamp(max=V - 1)
    pos = i.expand(B, T)
    inner = pos < (length - 1)[:, None]
    nxt = tok.gather(1, torch.cat([node[:, 1:], node[:, :1]], 1))
    emitted = torch.where(inner, nxt, torch.where(pos == (length - 1)[:, None], last[:, None], torch.full_like(nxt, -1)))
    kept = pos < length[:, None]
    logp = torch.log(p[b[:, None], node, emitted.clamp(min=0)].double())
    return {"accepted_tokens": emitted.to(torch.int32), "accept_length": length.to(torch.int32),
            "accept_index": torch.where(kept, b[:, None] * T + node, -1).to(torch.int32),
            "logprobs": torch.where(kept, logp, torch.zeros_like(logp)).float()}


def run(state):
    if own:
        return _run_own(state)
    return {"attn": _plain_attn, "append": _plain_append, "read": _plain_read,
            "tree": _plain_tree}[state["case"]["kind"]](state)


# ---- in 64 bits, request by request -----------------------------------------------------

def _cached64(s, name, b, n):
    """The first n tokens of request b in 64 bits: [Hkv, n, D]."""
    size = s["case"]["page"]
    pages = s["page_table"][b, : -(-n // size)].long()
    x = s[name + "_cache"].view(torch.uint8)[pages].view(_F8).double()
    x = x * s[name + "_scale"][pages].double()[:, :, None, None]
    return x.transpose(0, 1).flatten(1, 2)[:, :n]


def _exact_attn(s):
    c = s["case"]
    G = c["Hq"] // c["Hkv"]
    outs, lses = [], []
    first = 0
    for b, (n, t) in enumerate(zip(_lens(c), _windows(c))):
        k, v = _cached64(s, "k", b, n), _cached64(s, "v", b, n)
        seen = torch.ones(t, n, dtype=torch.bool, device=k.device)
        if c["mask"] != "none":
            k = torch.cat([k, s["k_new"][first:first + t].double().transpose(0, 1)], 1)
            v = torch.cat([v, s["v_new"][first:first + t].double().transpose(0, 1)], 1)
            m = np.tril(np.ones((t, t), bool))
            if c["mask"] == "tree":
                par = s["parents"][first:first + t].tolist()
                m = np.zeros((t, t), bool)
                for i in range(t):
                    m[i] = m[par[i]] if i else False
                    m[i, i] = True
            seen = torch.cat([seen, torch.from_numpy(m).to(k.device)], 1)
        q = s["q"][first:first + t].double().view(t, c["Hkv"], G, c["D"]).permute(1, 2, 0, 3)
        x = torch.einsum("hgtd,hnd->hgtn", q, k) / math.sqrt(c["D"])
        x = torch.where(seen, x, torch.full_like(x, -math.inf))
        top = x.max(-1, keepdim=True).values
        e = torch.exp(x - top)
        z = e.sum(-1, keepdim=True)
        o = torch.einsum("hgtn,hnd->hgtd", e / z, v)
        outs.append(o.permute(2, 0, 1, 3).reshape(t, c["Hq"], c["D"]))
        lses.append((top + torch.log(z)).squeeze(-1).permute(2, 0, 1).reshape(t, c["Hq"]))
        first += t
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def _e4m3(x):
    """x rounded to the nearest e4m3 value, ties to even, saturating; in 64 bits."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 4).clamp(min=-9).double())
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_append(s):
    c = s["case"]
    n = c["page"]
    out = {}
    starts = np.concatenate([[0], np.cumsum(_windows(c))])
    for name in ("k", "v"):
        codes = s[name + "_cache"].double()
        scales = s[name + "_scale"].double()
        for b, (length, count) in enumerate(zip(_lens(c), _taken(c))):
            if c["accepted"]:
                x = s[name][s["src_index"][b, :count].long()].double()
            else:
                x = s[name][int(starts[b]):int(starts[b]) + count].double()
            table = s["page_table"][b].tolist()
            lo = length
            while lo < length + count:
                page, a = table[lo // n], lo % n
                z = min(n, a + length + count - lo)
                part = x[lo - length:lo - length + z - a].transpose(0, 1)      # [Hkv, tokens, D]
                top = part.abs().amax((1, 2)).clamp(min=2.0 ** -200)
                e = torch.ceil(torch.log2(top / 448) - 1e-12).clamp(-60, 60)
                e = torch.where(top > 448 * torch.exp2(e), e + 1, e)
                scale = torch.exp2(e.clamp(-60, 60))
                if a:
                    scale = torch.maximum(scale, scales[page])
                    codes[page, :, :a] = _e4m3(codes[page, :, :a] * (scales[page] / scale)[:, None, None])
                codes[page, :, a:z] = _e4m3(part / scale[:, None, None])
                scales[page] = scale
                lo += z - a
        out[name + "_cache"], out[name + "_scale"] = codes, scales
    return out


def _exact_read(s):
    c = s["case"]
    return {name: torch.cat([_cached64(s, name, b, n).transpose(0, 1) for b, n in enumerate(_lens(c))])
            for name in ("k", "v")}


def _exact_tree(s):
    c = s["case"]
    B, T, V = c["B"], c["T"], c["V"]
    p = s["probs"].view(B, T, V)
    tok, par, u = s["tokens"].cpu().numpy(), s["parents"].cpu().numpy(), s["uniforms"].cpu().double().numpy()
    px = p[torch.arange(B, device=p.device)[:, None], s["parents"].long().clamp(min=0), s["tokens"].long()]
    px = px.cpu().double().numpy()
    res = {"accepted_tokens": np.full((B, T), -1, np.int32), "accept_length": np.zeros(B, np.int32),
           "accept_index": np.full((B, T), -1, np.int32), "logprobs": np.zeros((B, T))}
    for b in range(B):
        cur, j = 0, 0
        while True:
            res["accept_index"][b, j] = b * T + cur
            gone, seen, chosen = 0.0, [], None
            for ch in np.nonzero(par[b] == cur)[0]:
                x = int(tok[b, ch])
                q = 0.0 if x in seen else px[b, ch]
                if u[b, ch] * (1.0 - gone) < q:
                    chosen = int(ch)
                    break
                gone += q
                seen.append(x)
            if chosen is None:
                break
            res["accepted_tokens"][b, j] = tok[b, chosen]
            res["logprobs"][b, j] = math.log(px[b, chosen])
            cur, j = chosen, j + 1
        row = p[b, cur].cpu().double().numpy()
        w = row.copy()
        w[seen] = 0.0
        if not w.sum() > 0:
            w = row
        mass = np.cumsum(w)
        x = min(int(np.searchsorted(mass, u[b, 0] * mass[-1], side="right")), V - 1)
        res["accepted_tokens"][b, j] = x
        res["logprobs"][b, j] = math.log(row[x])
        res["accept_length"][b] = j + 1
    return res


def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _exact_attn, "append": _exact_append, "read": _exact_read,
            "tree": _exact_tree}[case["kind"]](s)


# ---- what a pass cannot do without ------------------------------------------------------

def work(case):
    c = case
    if c["kind"] == "tree":
        # the coins, tokens, parents and one probability of each node; one row for the draw
        n = c["B"] * c["T"]
        return {"bytes": c["B"] * c["V"] * 4.0 + n * (16 + 12) + c["B"] * 4, "flops": c["B"] * c["V"] * 1.0}
    Hkv, D = c["Hkv"], c["D"]
    lens = _lens(c)
    if c["kind"] == "attn":
        w = _windows(c)
        rows, own_kv = sum(w), 0 if c["mask"] == "none" else 1
        cache = sum(n * Hkv * D * 2 + -(-n // c["page"]) * (Hkv * 8 + 4) for n in lens)
        pairs = sum(t * n + own_kv * t * (t + 1) // 2 for t, n in zip(w, lens))
        return {"bytes": float(cache + rows * (c["Hq"] * (4 * D + 4) + own_kv * Hkv * D * 4)),
                "flops": 4.0 * pairs * c["Hq"] * D}
    size = {"bf16": 2, "fp16": 2, "fp32": 4}[c["dtype"]]
    if c["kind"] == "append":
        n = sum(_taken(c))
        blocks = sum((x + t - 1) // c["page"] - x // c["page"] + 1 for x, t in zip(lens, _taken(c)))
        return {"bytes": float(n * Hkv * D * 2 * (size + 1) + blocks * (Hkv * 8 + 4)), "flops": 4.0 * n * Hkv * D}
    n = sum(lens)
    return {"bytes": float(n * Hkv * D * 2 * (size + 1) + sum(-(-x // c["page"]) for x in lens) * (Hkv * 8 + 4)),
            "flops": 2.0 * n * Hkv * D}
