"""Plain 64-bit implementations of the operators around the verify step (attention of a window
over the 8-bit cache, appending to the cache, tree verification), for the tests: loops over
requests and heads, written from the definitions."""
import math

import numpy as np
import torch

F8 = torch.float8_e4m3fn


def codes64(cache):
    """The e4m3 values of a cache as float64 (CPU)."""
    return cache.cpu().view(torch.uint8).view(F8).to(torch.float32).double()


def cached(cache, scale, table, b, n):
    """K or V of request b's first n tokens, [n, H, D] float64, and which of them exist."""
    codes, scale = codes64(cache), scale.cpu().double()
    pages, H, size, D = codes.shape
    out = torch.zeros((n, H, D), dtype=torch.float64)
    there = torch.zeros(n, dtype=torch.bool)
    for i in range(n):
        page = int(table[b, i // size])
        if 0 <= page < pages:
            out[i] = codes[page, :, i % size] * scale[page][:, None]
            there[i] = True
    return out, there


def sees(t, parents=None):
    """[t, t] truth values: which rows of its window a row sees."""
    m = np.tril(np.ones((t, t), bool))
    if parents is not None:
        m = np.zeros((t, t), bool)
        for i in range(t):
            up = int(parents[i])
            if 0 <= up < i:
                m[i] = m[up]
            m[i, i] = True
    return torch.from_numpy(m)


def attention(q, k_cache, v_cache, k_scale, v_scale, table, lens, windows, k_new=None, v_new=None,
              parents=None, sm_scale=None):
    """out, lse and, per output element, what its error bound is made of: the weighted mean of
    |v| and, per row, the largest sum of |q k|, the number of tokens, and the largest |q| of the
    request's rows of a KV head times the largest sum of |k|. windows: (first row, rows) of
    each request."""
    rows, Hq, D = q.shape
    H = k_cache.shape[1]
    G = Hq // H
    scale = D ** -0.5 if sm_scale is None else sm_scale
    q = q.cpu().double()
    out = torch.zeros((rows, Hq, D), dtype=torch.float64)
    absv = torch.zeros_like(out)
    lse = torch.full((rows, Hq), -math.inf, dtype=torch.float64)
    big = torch.zeros_like(lse)
    count = torch.zeros_like(lse)
    floor = torch.zeros_like(lse)
    table = table.cpu()
    for b, (r0, t) in enumerate(windows):
        n = min(max(int(lens[b]), 0), table.shape[1] * k_cache.shape[2])
        k, there = cached(k_cache, k_scale, table, b, n)
        v, _ = cached(v_cache, v_scale, table, b, n)
        seen = there[None].expand(t, n)
        if k_new is not None:
            k = torch.cat([k, k_new[r0:r0 + t].cpu().double()])
            v = torch.cat([v, v_new[r0:r0 + t].cpu().double()])
            seen = torch.cat([seen, sees(t, None if parents is None else parents[r0:r0 + t].tolist())], 1)
        for h in range(Hq):
            for i in range(t):
                idx = torch.nonzero(seen[i]).squeeze(1)
                if len(idx) == 0:
                    continue
                kk, vv = k[idx, h // G], v[idx, h // G]
                x = (kk @ q[r0 + i, h]) * scale
                m = x.max()
                e = torch.exp(x - m)
                z = e.sum()
                out[r0 + i, h] = (e / z) @ vv
                absv[r0 + i, h] = (e / z) @ vv.abs()
                lse[r0 + i, h] = m + torch.log(z)
                big[r0 + i, h] = (kk.abs() @ q[r0 + i, h].abs()).max() * abs(scale)
                count[r0 + i, h] = len(idx)
                heads = q[r0:r0 + t, h // G * G:(h // G + 1) * G].abs()
                floor[r0 + i, h] = heads.max() * kk.abs().sum(1).max() * abs(scale)
    return out, lse, absv, big, count, floor


def attention_bounds(out, lse, absv, big, count, floor, dtype, D, two_parts=False):
    """How far the kernel may be off, from its roundings.
    Scores: D + 8 fp32 roundings or truncations of partial sums no larger than sum |q k|
    (2^-23 each), and an error of each q of 2^-17 of the largest of its row block (e4m3 parts: the
    largest lies in [2^7, 2^8), the last part is rounded to a multiple of 2^-9 or better):
    d = (D + 8) 2^-23 sum |q k| + 2^-17 max |q| sum |k|; the exponent's
    argument is rounded in log2 units, at most as large (2^-23 of it) and the hardware 2^x is
    good to 2^-22. Probabilities: 2^-11 (fp16); two_parts (bf16, head_dim 128, more than 32 rows
    of a KV head a window): an e4m3 part and an e5m2 part of its rest, half a step of either,
    2^-4 2^-3 = 2^-7. Sums over n tokens: n 2^-23. The quotient of two
    such sums doubles what they share. The output is rounded by eps / 2 of its value."""
    d = (D + 8) * 2.0 ** -23 * big + 2.0 ** -17 * floor + 2.0 ** -21
    prob = 2.0 ** -7 if two_parts else 2.0 ** -11
    share = prob + 2 * d + 2 * count * 2.0 ** -23
    half = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).tiny
    b = half * out.abs() + (1 + half) * absv * share[..., None] + tiny
    fine = torch.isfinite(lse)
    z = torch.where(fine, lse.abs(), torch.zeros_like(lse))
    return b, d + count * 2.0 ** -23 + 2.0 ** -22 * (z + 1)


def e4m3(x):
    """Nearest e4m3 value, ties to even, saturating; NaN stays. x: float64."""
    step = torch.exp2((torch.frexp(x)[1] - 4).clamp(min=-9).double())
    return (torch.round(x / step) * step).clamp(-448, 448)


def block_exponent(top):
    for e in range(-60, 61):
        if top <= 448.0 * 2.0 ** e:
            return e
    return 60


def append(cache, scales, x, table, lens, rows_of):
    """Codes (as values) and scales after an append; rows_of[b]: row numbers of x (or None where
    the number is out of range)."""
    codes, scales = codes64(cache), scales.cpu().double().clone()
    pages, H, size, D = codes.shape
    x = x.cpu().double()
    for b, rows in enumerate(rows_of):
        cap = table.shape[1] * size
        n = min(max(int(lens[b]), 0), cap)
        blocks = {}
        for j, r in enumerate(rows):
            if n + j < cap and r is not None:
                blocks.setdefault((n + j) // size, []).append(((n + j) % size, r))
        for i, items in blocks.items():
            page = int(table[b, i])
            if not 0 <= page < pages:
                continue
            held = max(0, n - i * size)
            for h in range(H):
                new = torch.stack([x[r, h] for _, r in items])
                finite = new[torch.isfinite(new)].abs()
                s = 2.0 ** block_exponent(float(finite.max()) if len(finite) else 0.0)
                old = float(scales[page, h])
                if held:
                    s = max(old, s)
                    if s != old:
                        codes[page, h, :held] = e4m3(codes[page, h, :held] * (old / s))
                for slot, r in items:
                    y = x[r, h] / s
                    y = torch.where(torch.isinf(y), torch.sign(y) * 448, y)
                    codes[page, h, slot] = e4m3(y)
                scales[page, h] = s
    return codes, scales


def tree(probs, tokens, parents, uniforms, windows, D):
    """Tree verification: dict of numpy arrays as the call returns them."""
    p = probs.cpu().double().numpy()
    tok, par = tokens.cpu().numpy().reshape(-1), parents.cpu().numpy().reshape(-1)
    u = uniforms.cpu().double().numpy().reshape(-1)
    B, V = len(windows), p.shape[1]
    res = dict(accepted_tokens=np.full((B, D + 1), -1, np.int32), accept_length=np.zeros(B, np.int32),
               accept_index=np.full((B, D + 1), -1, np.int32), logprobs=np.zeros((B, D + 1)))
    for b, (r0, n) in enumerate(windows):
        cur, j = 0, 0
        while True:
            res["accept_index"][b, j] = r0 + cur
            gone, removed, chosen = 0.0, [], None
            if j < D:
                for ch in range(cur + 1, n):
                    if par[r0 + ch] != cur:
                        continue
                    x = int(tok[r0 + ch])
                    q = p[r0 + cur, x] if 0 <= x < V and x not in removed else 0.0
                    if u[r0 + ch] * (1.0 - gone) < q:
                        chosen = ch
                        break
                    gone += q
                    if 0 <= x < V:
                        removed.append(x)
            if chosen is None:
                break
            res["accepted_tokens"][b, j] = tok[r0 + chosen]
            res["logprobs"][b, j] = math.log(p[r0 + cur, tok[r0 + chosen]])
            cur, j = chosen, j + 1
        w = p[r0 + cur].copy()
        w[removed] = 0.0
        if not w.sum() > 0:
            w = p[r0 + cur]
        mass = np.cumsum(w)
        x = min(int(np.searchsorted(mass, u[r0] * mass[-1], side="right")), V - 1)
        res["accepted_tokens"][b, j] = x
        with np.errstate(divide="ignore"):
            res["logprobs"][b, j] = np.log(p[r0 + cur, x])
        res["accept_length"][b] = j + 1
    return res
