"""Attention that reads a group's shared prefix once, against plain attention in 64 bits over each
request's whole table."""
import math

import numpy as np
import pytest
import torch

from tests import window_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    from speculative_decoding_verify_temp_gb300 import tsverify

    yield tsverify
    assert tsverify.device_error() == 0


def ints(v):
    return torch.tensor(np.asarray(v, np.int64).astype(np.int32), device="cuda")


def case(seed, groups, Hq, Hkv, D, page, dtype=torch.bfloat16, mask="chain", outside=0, strided=False):
    """groups: a list of (shared tokens, [(own tokens, window rows) of each request]); `outside`
    requests behind them belong to no group."""
    r = np.random.default_rng(seed)
    g = torch.Generator("cuda").manual_seed(seed)
    lens, windows, tables, ptr, shared, used = [], [], [], [0], [], 0
    for s, members in groups:
        common = list(range(used, used + s // page))
        used += s // page
        for own, w in members:
            n = -(-(s + own) // page) - s // page
            tables.append(common + list(range(used, used + n)))
            used += n
            lens.append(s + own)
            windows.append(w)
        ptr.append(len(lens))
        shared.append(s)
    for i in range(outside):
        tables.append(list(range(used, used + 3)))
        used += 3
        lens.append(3 * page - 5)
        windows.append(2)
    pages = used + 2
    ids = r.permutation(pages)
    P = max(max(len(t) for t in tables), 1)
    table = np.full((len(lens), P), -1, np.int64)
    for b, t in enumerate(tables):
        table[b, :len(t)] = ids[t]
    rows = sum(windows)

    def codes():
        x = (torch.randn((pages, Hkv, page, D), generator=g, device="cuda") * 60).clamp(-448, 448).to(window_ref.F8)
        if strided:  # heads behind tokens
            return x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
        return x

    def scales():
        return torch.exp2(torch.rand((pages, Hkv), generator=g, device="cuda") * 4 - 8)

    def new(h):
        x = torch.randn((rows, h, D), generator=g, device="cuda").to(dtype)
        return torch.cat([x, x], -1)[..., :D] if strided else x

    c = dict(q=new(Hq) * 2, k_cache=codes(), v_cache=codes(), k_scale=scales(), v_scale=scales(),
             page_table=ints(table), seq_lens=ints(lens), qo_indptr=ints([0] + list(np.cumsum(windows))),
             group_indptr=ints(ptr), shared_lens=ints(shared))
    if mask != "none":
        c.update(k_new=new(Hkv), v_new=new(Hkv))
    if mask == "tree":
        c["parents"] = ints([int(r.integers(max(0, i - 3), i)) if i else -1 for w in windows for i in range(w)])
    return c


def reference(c, sm_scale=None):
    """window_ref.attention's results, request by request and KV head by KV head, on the GPU."""
    q, page = c["q"].double(), c["k_cache"].shape[2]
    rows, Hq, D = q.shape
    pages, H = c["k_scale"].shape
    G = Hq // H
    scale = D ** -0.5 if sm_scale is None else sm_scale
    out = torch.zeros_like(q)
    absv = torch.zeros_like(q)
    lse = torch.full((rows, Hq), -math.inf, dtype=torch.float64, device="cuda")
    big, count, floor = (torch.zeros_like(lse) for _ in range(3))
    qo = c["qo_indptr"].tolist()
    table, lens = c["page_table"].long(), c["seq_lens"].tolist()
    for b in range(len(lens)):
        r0, t = qo[b], qo[b + 1] - qo[b]
        n = min(max(lens[b], 0), table.shape[1] * page)
        if t <= 0 or t > 128:
            continue
        ids = table[b, : -(-n // page)]
        ok = (ids >= 0) & (ids < pages)
        there = ok.repeat_interleave(page)[:n]
        kv = []
        for name in ("k", "v"):
            x = c[name + "_cache"].view(torch.uint8)[ids.clamp(0, pages - 1)].view(window_ref.F8).double()
            x = x * c[name + "_scale"][ids.clamp(0, pages - 1)].double()[..., None, None]
            kv.append(x.permute(0, 2, 1, 3).reshape(-1, H, D)[:n])
        k, v = kv
        seen = there.expand(t, n)
        if "k_new" in c:
            k, v = (torch.cat([x, c[name][r0:r0 + t].double()]) for x, name in ((k, "k_new"), (v, "v_new")))
            par = c["parents"][r0:r0 + t].tolist() if "parents" in c else None
            seen = torch.cat([seen, window_ref.sees(t, par).cuda()], 1)
        # tokens that nobody sees must not matter
        v = torch.where(seen.any(0)[:, None, None], v, torch.zeros_like(v))
        k = torch.where(seen.any(0)[:, None, None], k, torch.zeros_like(k))
        for h in range(H):
            qq = q[r0:r0 + t, h * G:(h + 1) * G]                       # [t, G, D]
            x = torch.einsum("tgd,nd->tgn", qq, k[:, h]) * scale
            x = torch.where(seen[:, None], x, torch.full_like(x, -math.inf))
            at = (slice(r0, r0 + t), slice(h * G, (h + 1) * G))
            z = torch.logsumexp(x, -1)
            e = torch.exp(x - torch.where(z == -math.inf, torch.zeros_like(z), z)[..., None])
            lse[at] = z
            out[at] = torch.einsum("tgn,nd->tgd", e, v[:, h])
            absv[at] = torch.einsum("tgn,nd->tgd", e, v[:, h].abs())
            qk = torch.einsum("tgd,nd->tgn", qq.abs(), k[:, h].abs()) * seen[:, None]
            big[at] = (qk.amax(-1) if qk.shape[-1] else 0) * abs(scale)
            count[at] = seen.sum(-1).double()[:, None].expand(t, G)
            ks = (k[:, h].abs().sum(-1) * seen.any(0)).max() if k.shape[0] else 0
            floor[at] = qq.abs().max() * ks * abs(scale)
    return out, lse, absv, big, count, floor


def check(c, got, ref=None, sm_scale=None):
    """Within window attention's bounds. Joining parts (slots, pieces, the prefix with the rest)
    multiplies outputs and sums by hardware powers of two, good to 2^-22 with arguments rounded at
    2^-24 of at most 2^5 where their result matters to 2^-24: 2^-18 for each of four joinings.
    Probabilities of shared tokens are multiples of 2^-24, the largest at least 2^4: half a step
    each is 2^-29 of the row's sum, times the largest value of V (largest code, largest scale)."""
    ref = ref or reference(c, sm_scale)
    rows = torch.isfinite(ref[1]) | (ref[1] == -math.inf)
    b, z = window_ref.attention_bounds(*ref, c["q"].dtype, c["q"].shape[-1])
    named = c["page_table"][(c["page_table"] >= 0) & (c["page_table"] < c["v_scale"].shape[0])].long()
    vmax = c["v_cache"].view(torch.uint8)[named].view(window_ref.F8).float().abs().nan_to_num(0).max() * c["v_scale"][named].max() \
        if named.numel() else 0
    b = b + 4 * 2.0 ** -18 * ref[2] + ref[4][..., None] * 2.0 ** -29 * vmax
    z = z + 4 * 2.0 ** -18
    err = (got["out"].double() - ref[0]).abs()
    assert (err <= b)[rows].all(), (err / b)[rows].max().item()
    if got["lse"] is not None:
        both = (got["lse"] == -math.inf) & (ref[1] == -math.inf)
        err = torch.where(both, torch.zeros_like(z), (got["lse"].double() - ref[1]).abs())
        assert (err <= z)[rows].all(), (err / z)[rows].max().item()
    return ref


CASES = {
    "one tile": dict(groups=[(128, [(1, 1)] * 2)], Hq=8, Hkv=2, page=16),
    "part of a tile": dict(groups=[(48, [(3, 1), (40, 2)])], Hq=4, Hkv=1, page=16),
    "several tiles, both slots on one block": dict(groups=[(700, [(9, 1)] * 5)], Hq=16, Hkv=2, page=32),
    "rows just over a slot": dict(groups=[(500, [(9, 3)] * 11)], Hq=8, Hkv=2, page=64),
    "rows of a whole block": dict(groups=[(640, [(30, 4)] * 16)], Hq=8, Hkv=2, page=128),
    "several blocks, a small last one": dict(groups=[(1500, [(5, 8)] * 21)], Hq=8, Hkv=2, page=16),
    "groups of many sizes": dict(groups=[(0, [(5, 1)] * 2), (16, [(1, 2)]), (15, [(9, 3)] * 3), (1000, [(100, 1)] * 40),
                                         (300, [(0, 2), (1, 1), (77, 5)]), (4000, [(10, 7)])], Hq=8, Hkv=4, page=16, outside=3),
    "a group of five heads": dict(groups=[(333, [(50, 3)] * 7), (900, [(1, 1)] * 3)], Hq=15, Hkv=3, page=32, outside=1),
    "long": dict(groups=[(20000, [(100, 2)] * 9)], Hq=8, Hkv=1, page=64),
    "blocks for eight CTAs side by side": dict(groups=[(1000, [(3, 16)] * 32)], Hq=16, Hkv=4, page=64),
    "blocks for two": dict(groups=[(700, [(1, 20)] * 32), (300, [(2, 9)] * 30)], Hq=4, Hkv=1, page=16),
    "many units a CTA": dict(groups=[(200 + 16 * i, [(20, 1)] * (1 + i % 4)) for i in range(60)], Hq=16, Hkv=8, page=16),
}


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("dtype,mask", [(torch.bfloat16, "chain"), (torch.float16, "tree"), (torch.bfloat16, "none")])
def test_against_plain_attention(tv, name, D, dtype, mask):
    c = case(1, D=D, dtype=dtype, mask=mask, strided=mask == "tree", **CASES[name])
    ref = check(c, tv.shared_attention(**c, lse=True))
    # the same where nothing is shared: all of each request's tokens are its own
    c["shared_lens"] = torch.zeros_like(c["shared_lens"])
    check(c, tv.shared_attention(**c, lse=True), ref)


@pytest.mark.parametrize("D", [64, 128])
def test_how_many_tokens_are_shared(tv, D):
    c = case(2, [(500, [(3, 2), (60, 2), (0, 1)]), (64, [(0, 1)] * 2)], 8, 2, D, 16)
    ref = reference(c)
    # more than the shortest request has, not whole pages, fewer than there are, none, less than none
    for lens in ([10 ** 9, 2 ** 31 - 1], [499, 63], [17, 16], [15, 0], [-5, -2 ** 31]):
        c["shared_lens"] = ints(lens)
        check(c, tv.shared_attention(**c, lse=True), ref)


@pytest.mark.parametrize("D", [64, 128])
def test_a_request_without_a_window_does_not_limit_its_group(tv, D):
    # a padded batch: the group's first and last requests are empty, of length 0 and with tables of
    # their own; one window is too long and is skipped
    c = case(3, [(300, [(5, 0), (7, 2), (9, 129), (11, 3), (0, 0)])], 4, 2, D, 16)
    c["page_table"][0] = -1
    c["page_table"][4] = 10 ** 6
    c["seq_lens"][0] = c["seq_lens"][4] = 0
    out = torch.full_like(c["q"], 7.0)
    ref = reference(c)
    tv.shared_attention(**c, out=out)
    err = (out.double() - ref[0]).abs()
    b, _ = window_ref.attention_bounds(*ref, c["q"].dtype, D)
    b = b + 4 * 2.0 ** -18 * ref[2]
    keep = torch.tensor([True] * 2 + [False] * 129 + [True] * 3, device="cuda")
    assert (err <= b)[keep].all()
    assert (out[~keep] == 7.0).all()


@pytest.mark.parametrize("D", [64, 128])
def test_groups_that_do_not_fit_share_nothing(tv, D):
    c = case(4, [(300, [(5, 1)] * 3), (200, [(9, 2)] * 2)], 4, 2, D, 16, outside=2)
    ref = reference(c)
    for ptr in ([9, 9, 9], [-3, -1, 0], [3, 99, 99]):
        c["group_indptr"] = ints(ptr)
        check(c, tv.shared_attention(**c, lse=True), ref)
    # equal windows without qo_indptr
    c = case(5, [(300, [(5, 2)] * 3)], 4, 2, D, 16)
    check(c, tv.shared_attention(**{k: v for k, v in c.items() if k != "qo_indptr"}, lse=True))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows", [1, 40])
def test_pages_that_are_not_there(tv, D, rows):
    c = case(6, [(16 * 30, [(5, 2)] * rows), (64, [(4, 1)] * 3)], 8, 2, D, 16, mask="none")
    c["page_table"][:rows, 3] = -1
    c["page_table"][:rows, 8:20] = 10 ** 6     # a whole tile and more
    c["page_table"][rows:, :] = -7             # rows that see nothing at all
    got = tv.shared_attention(**c, lse=True)
    ref = check(c, got)
    assert (ref[1][2 * rows:] == -math.inf).all() and (got["out"][2 * rows:] == 0).all()
    # nor does what lies in pages that nobody names matter
    used = torch.unique(c["page_table"][:rows])
    for t in range(c["k_cache"].shape[0]):
        if t not in used.tolist():
            c["k_cache"].view(torch.uint8)[t] = 0x7F
            c["v_cache"].view(torch.uint8)[t] = 0x7F
            c["k_scale"][t] = c["v_scale"][t] = math.nan
    again = tv.shared_attention(**c, lse=True)
    assert torch.equal(got["out"], again["out"]) and torch.equal(got["lse"], again["lse"])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_values_that_are_not_finite(tv, D, dtype):
    c = case(7, [(400, [(20, 3)] * 30)], 8, 2, D, 16, dtype=dtype)
    base = tv.shared_attention(**c, lse=True)
    # a query: its row and head alone
    q = c["q"].clone()
    q[5, 3, 7] = math.nan
    q[40, 0, 0] = math.inf
    got = tv.shared_attention(**dict(c, q=q), lse=True)
    bad = torch.zeros(90, 8, dtype=torch.bool, device="cuda")
    bad[5, 3] = bad[40, 0] = True
    assert torch.isnan(got["out"][bad]).all() and torch.isnan(got["lse"][bad]).all()
    assert torch.equal(got["out"][~bad], base["out"][~bad])
    # a shared key: every row of its heads; a shared value: one dim of them
    page = int(c["page_table"][0, 2])
    k = c["k_cache"].clone()
    k.view(torch.uint8)[page, 1, 4, 9] = 0x7F
    got = tv.shared_attention(**dict(c, k_cache=k), lse=True)
    assert torch.isnan(got["out"][:, 4:]).all() and torch.equal(got["out"][:, :4], base["out"][:, :4])
    v = c["v_cache"].clone()
    v.view(torch.uint8)[page, 0, 4, 9] = 0xFF
    got = tv.shared_attention(**dict(c, v_cache=v), lse=True)
    dims = torch.arange(D, device="cuda") == 9
    assert torch.isnan(got["out"][:, :4, dims]).all() and torch.equal(got["out"][:, 4:], base["out"][:, 4:])
    assert torch.equal(got["out"][:, :4, ~dims], base["out"][:, :4, ~dims])
    assert torch.equal(got["lse"], base["lse"])
    # a scale
    for name in ("k_scale", "v_scale"):
        s = c[name].clone()
        s[page, 0] = math.nan
        got = tv.shared_attention(**dict(c, **{name: s}), lse=True)
        assert torch.isnan(got["out"][:, :4]).all() and torch.equal(got["out"][:, 4:], base["out"][:, 4:])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype,sizes", [(torch.bfloat16, [2.0 ** 120, 2.0 ** -120, 1.0]), (torch.float16, [2.0 ** 12, 2.0 ** -20, 1.0])])
def test_queries_of_any_size(tv, D, dtype, sizes):
    # each row with a size of its own, scales of K that bring the scores back
    c = case(8, [(500, [(20, 3)] * 20)], 8, 2, D, 32, dtype=dtype, mask="none")
    for size in sizes:
        cc = dict(c, q=(c["q"].float() * size).to(dtype))
        for k_by, sm in ((1.0, D ** -0.5 / size), (2.0 ** -60, D ** -0.5 / size * 2.0 ** 60)):
            if not 2.0 ** -126 < abs(sm) < 2.0 ** 126:
                continue
            x = dict(cc, k_scale=c["k_scale"] * k_by)
            check(x, tv.shared_attention(**x, sm_scale=sm, lse=True), sm_scale=sm)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows", [3, 60])
@pytest.mark.parametrize("order", ["rising", "falling", "one", "last"])
def test_references_that_move(tv, D, rows, order):
    # scores over hundreds of powers of two: K's scales make the tiles' largest scores rise or fall
    c = case(9, [(128 * 24, [(20, 1)] * rows)], 8, 2, D, 128)
    n = 24
    e = {"rising": torch.arange(n) / 3 - 4, "falling": 4 - torch.arange(n) / 3,
         "one": torch.where(torch.arange(n) == 11, 5.0, -3.0), "last": torch.where(torch.arange(n) == n - 1, 5.0, -3.0)}[order]
    c["k_scale"][c["page_table"][0, :n].long()] = torch.exp2(e - 4).cuda()[:, None].float()
    check(c, tv.shared_attention(**c, lse=True))
    # scores that are all very negative are scores too
    c["k_scale"][c["page_table"][0, :n].long()] = 2.0 ** 100
    c["k_cache"].view(torch.uint8)[:] = 0x38          # ones
    c["q"] = -c["q"].abs()
    got = tv.shared_attention(**c, lse=True)
    assert torch.isfinite(got["out"]).all()
    assert torch.allclose(got["lse"].double(), reference(c)[1], rtol=1e-5)


@pytest.mark.parametrize("D", [64, 128])
def test_scales_of_v(tv, D):
    # of very different sizes from block to block
    c = case(10, [(16 * 40, [(20, 2)] * 40)], 8, 2, D, 16)
    pages = c["page_table"][0, :40].long()
    c["v_scale"][pages] = torch.exp2(torch.randint(-20, 20, (40, 2), device="cuda").float())
    check(c, tv.shared_attention(**c, lse=True))
    # zero and tiny ones count as 2^-80: no output, all of the sum
    c["v_scale"][pages] = 0
    c["v_scale"][pages[:20]] = 2.0 ** -140
    got = tv.shared_attention(**c, lse=True)
    _, z = window_ref.attention_bounds(*reference(c), c["q"].dtype, D)
    assert torch.isfinite(got["out"]).all()
    assert ((got["lse"].double() - reference(c)[1]).abs() <= z + 2.0 ** -16).all()


@pytest.mark.parametrize("D", [64, 128])
def test_one_large_probability_and_many_small_ones(tv, D):
    # the small ones' share must not get lost behind the large one's reference
    n = 128 * 100
    c = case(11, [(n, [(1, 1)] * 3)], 4, 1, D, 128, mask="none")
    c["q"][:] = 0
    c["q"][..., 0] = 1
    c["k_cache"].view(torch.uint8)[:] = 0
    c["k_scale"][:] = 1
    c["v_scale"][:] = 1
    c["v_cache"].view(torch.uint8)[:] = 0x38          # ones
    first = int(c["page_table"][0, 0])
    c["k_cache"].view(torch.uint8)[first, 0, 5, 0] = 0x50   # a score of 16 at sm_scale 1: e^16 against 12800 of 1
    c["v_cache"].view(torch.uint8)[first, 0, 5, :] = 0
    ref = reference(c, 1.0)
    check(c, tv.shared_attention(**c, sm_scale=1.0, lse=True), ref)


def test_offsets_past_32_bits(tv):
    # a pool of 36000 pages of 131072 bytes: 4.7 GB
    pages, D, H = 36000, 128, 8
    c = case(12, [(128 * 6, [(20, 2)] * 20)], 16, H, D, 128)
    n = c["k_cache"].shape[0]
    big = {}
    for name in ("k", "v"):
        x = torch.zeros((pages, H, 128, D), dtype=torch.uint8, device="cuda")
        x[pages - n:] = c[name + "_cache"].view(torch.uint8)
        s = torch.ones((pages, H), device="cuda")
        s[pages - n:] = c[name + "_scale"]
        big.update({name + "_cache": x.view(window_ref.F8), name + "_scale": s})
    want = tv.shared_attention(**c, lse=True)
    c.update(big, page_table=torch.where(c["page_table"] >= 0, c["page_table"] + pages - n, c["page_table"]))
    got = tv.shared_attention(**c, lse=True)
    assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])


@pytest.mark.parametrize("D", [64, 128])
def test_captured_on_another_stream_with_its_own_workspace(tv, D):
    c = case(13, [(900, [(40, 2)] * 12), (100, [(40, 1)] * 4)], 8, 2, D, 16)
    ws = tv.make_shared_attention_workspace(16, 2, 28, 8, 2, D)
    out = torch.empty_like(c["q"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        tv.shared_attention(**c, out=out, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tv.shared_attention(**c, out=out, workspace=ws)
    for seed in (14, 15):
        o = case(seed, [(900, [(40, 2)] * 12), (100, [(40, 1)] * 4)], 8, 2, D, 16)
        for k in c:
            c[k].copy_(o[k]) if k not in ("k_cache", "v_cache") else c[k].view(torch.uint8).copy_(o[k].view(torch.uint8))
        c["seq_lens"] -= seed - 10
        c["shared_lens"] -= 100 * (seed - 14)
        out.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        check(c, dict(out=out, lse=None))
        ws.fill_(0xFF)  # the workspace needs nothing from the call before
        again = tv.shared_attention(**c, workspace=ws, stream=side)
        side.synchronize()
        assert torch.equal(again["out"], out)


def test_runs_agree_bit_for_bit(tv):
    c = case(16, [(5000, [(40, 2)] * 30), (1000, [(300, 1)] * 9)], 32, 8, 128, 16)
    a = tv.shared_attention(**c, lse=True)
    for _ in range(5):
        b = tv.shared_attention(**c, lse=True)
        assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows,page", [((20,), 128), ((5, 19, 36, 8, 23), 16), ((37,), 64)])
def test_units_that_follow_each_other(tv, D, rows, page):
    # several short units a CTA, of 7 x rows rows: warps without rows in the second slot, whole slots, one slot;
    # a warp that is done with a unit early must not disturb its neighbours, which still write their outputs
    groups = [(128 + 128 * (i % 5) + page * (i % 3), [(5, rows[i % len(rows)])]) for i in range(120)]
    c = case(21, groups, 28, 4, D, page)
    a = tv.shared_attention(**c, lse=True)
    check(c, a)
    cold = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")  # more than L2
    for i in range(100):
        if i % 4 == 0:
            cold.fill_(i)
        b = tv.shared_attention(**c, lse=True)
        assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])


@pytest.mark.parametrize("D", [64, 128])
def test_long_units_with_pages_of_a_tile(tv, D):
    # one copy a tile of K or V: these land in any order, and none may be taken for the one before it
    c = case(22, [(9163, [(5, 10)] * 2), (5826, [(4, 10)] * 2), (30000, [(1, 10)] * 2), (8316, [(5, 3)] * 2)], 28, 4, D, 128)
    a = tv.shared_attention(**c, lse=True)
    check(c, a)
    for _ in range(100):
        b = tv.shared_attention(**c, lse=True)
        assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])


@pytest.mark.parametrize("D", [64, 128])
def test_answers_to_one_prompt(tv, D):
    """The calls together: a prompt is appended, forked into answers that grow by windows of drafted
    rows of which some are kept; each step's attention is that of window attention."""
    H, Hq, size, pages = 2, 8, 16, 200
    g = torch.Generator("cuda").manual_seed(0)
    z = torch.zeros((2, pages, H, size, D), dtype=torch.uint8, device="cuda").view(window_ref.F8)
    sc = torch.ones((2, pages, H), device="cuda")
    kv = dict(k_cache=z[0], v_cache=z[1], k_scale=sc[0], v_scale=sc[1])
    count = torch.zeros(pages, dtype=torch.int32, device="cuda")
    cache = dict(kv, page_table=torch.full((2, 40), -1, dtype=torch.int32, device="cuda"), seq_lens=ints([0, 0]))
    prompt = ints([300, 77])
    assert torch.equal(tv.kv_reserve(**cache, new_lens=prompt, refcount=count)["reserved"], prompt)
    x = torch.randn((2, 377, H, D), generator=g, device="cuda").bfloat16()
    tv.kv_append(x[0], x[1], **cache, qo_indptr=ints([0, 300, 377]))
    cache["seq_lens"] += prompt
    f = tv.kv_fork(**cache, sources=ints([0] * 5 + [1] * 3), refcount=count)
    tv.kv_free(**cache, refcount=count)
    cache = dict(kv, page_table=f["page_table"], seq_lens=f["seq_lens"])
    groups = dict(group_indptr=ints([0, 5, 8]), shared_lens=prompt)
    T = 4
    for step in range(4):
        q, k, v = (torch.randn((8 * T, h, D), generator=g, device="cuda").bfloat16() for h in (Hq, H, H))
        qo = ints(np.arange(0, 8 * T + 1, T))
        c = dict(cache, q=q, k_new=k, v_new=v, qo_indptr=qo)
        check(c, tv.shared_attention(**c, **groups, lse=True))
        length = ints([1 + (b + step) % T for b in range(8)])
        index = ints([[b * T + j for j in range(T)] for b in range(8)])
        r = tv.kv_reserve(**cache, new_lens=cache["seq_lens"] + length, refcount=count)
        assert torch.equal(r["reserved"], cache["seq_lens"] + length)
        tv.kv_append(k, v, **cache, src_index=index, src_len=length)
        cache["seq_lens"] += length
        if step == 1:
            tv.kv_compact(**cache, refcount=count)
            assert torch.equal(count > 0, torch.arange(pages, device="cuda") < (count > 0).sum())
    tv.kv_free(**cache, refcount=count)
    assert (count == 0).all()


@pytest.mark.parametrize("D", [64, 128])
def test_many_requests_and_groups(tv, D):
    # more groups and requests than the planning CTAs have threads; group sizes from none to nine
    r = np.random.default_rng(17)
    groups = [(int(r.integers(0, 90)), [(int(r.integers(0, 40)), int(r.integers(0, 3))) for _ in range(i % 10)]) for i in range(1500)]
    c = case(17, groups, 2, 1, D, 16)
    check(c, tv.shared_attention(**c, lse=True))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_what_is_left_may_be_long(tv, D, dtype):
    # more tiles of its own than a round of page numbers, split over CTAs; short windows and long ones
    for members in ([(5000, 1), (3, 2)], [(4100, 9)] * 3, [(2100, 40), (64, 5)]):
        c = case(18, [(200, members)], 8, 2, D, 32, dtype=dtype, mask="tree")
        check(c, tv.shared_attention(**c, lse=True))


@pytest.mark.parametrize("D", [64, 128])
def test_a_wait_that_runs_out(tv, D):
    """With a budget of one cycle waits give up before their copies land: nothing faults or hangs, the
    call's outputs are unspecified, ts_device_error reports it (bit 28), and the next call is not affected.
    A wait's first tries take some time of their own: with head_dim 64 every wait may end within it."""
    c = case(19, [(3000, [(20, 4)] * 50), (1700, [(20, 9)] * 30)], 64, 8, D, 16)
    want = tv.shared_attention(**c, lse=True)
    assert tv.device_error() == 0
    guard = torch.full((c["q"].shape[0] + 2, 64, D), 7.0, dtype=torch.bfloat16, device="cuda")
    word = 0
    for _ in range(10):
        tv.set_wait_cycles(1)
        try:
            tv.shared_attention(**c, out=guard[1:-1])
            torch.cuda.synchronize()
        finally:
            tv.set_wait_cycles(0)
        word |= tv.device_error(clear=True)
    assert word == 1 << 28 or (D == 64 and word == 0), hex(word)
    assert (guard[0] == 7.0).all() and (guard[-1] == 7.0).all()
    got = tv.shared_attention(**c, lse=True)
    assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])
    assert tv.device_error() == 0


def test_rows_that_no_window_owns_and_strided_rows(tv):
    c = case(20, [(300, [(5, 2), (7, 3)]), (100, [(9, 4)])], 8, 2, 128, 16)
    ref = reference(c)
    big = {k: torch.full((12, 2 * c[k].shape[1], 256), 3.0, dtype=torch.bfloat16, device="cuda") for k in ("q", "k_new", "v_new")}
    x = dict(c)
    for k in big:
        big[k][1:10, ::2, 64:192] = c[k]
        x[k] = big[k][1:11, ::2, 64:192]            # a row behind the last window
    out = torch.full((10, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    tv.shared_attention(**x, out=out)
    check(c, dict(out=out[:9], lse=None), ref)
    assert (out[9] == 7.0).all()
    # one row of q for all (stride 0)
    one = dict(c, q=c["q"][:1].expand(9, -1, -1))
    check(dict(c, q=one["q"].contiguous()), tv.shared_attention(**one, lse=True))


def test_two_streams_at_once(tv):
    a = case(21, [(3000, [(40, 2)] * 20)], 16, 4, 128, 16)
    b = case(22, [(900, [(10, 5)] * 50)], 8, 2, 64, 32, dtype=torch.float16)
    want = [tv.shared_attention(**x, lse=True) for x in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[tv.shared_attention(**x, lse=True, stream=s) for x, s in zip((a, b), streams)] for _ in range(10)]
    torch.cuda.synchronize()
    for pair in got:
        for x, y in zip(pair, want):
            assert torch.equal(x["out"], y["out"]) and torch.equal(x["lse"], y["lse"])
