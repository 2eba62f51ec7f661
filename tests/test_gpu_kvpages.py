"""The calls on the cache's pages against plain lists: every result is a whole number or a copied
byte, so all of them have to be equal."""
import numpy as np
import pytest
import torch

from tests import pages_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    from speculative_decoding_verify_temp_gb300 import tsverify

    return tsverify


def ints(v):
    return torch.tensor(np.asarray(v, np.int64).astype(np.int32), device="cuda")


def pool(seed, lens, size, P, pages, share=1, H=2, D=64, strided=False):
    """Requests next to each other, `share` at a time, continue one context."""
    r = np.random.default_rng(seed)
    ids = list(r.permutation(pages))
    table = np.full((len(lens), P), -1, np.int64)
    for b in range(0, len(lens), share):
        n = ref.entries(min(max(lens[b], 0), P * size), size)
        table[b:b + share, :n] = [ids.pop() for _ in range(n)]
    lens = [lens[b // share * share] for b in range(len(lens))]
    count = np.bincount(table[table >= 0], minlength=pages)
    codes = torch.from_numpy(r.integers(0, 256, (2, pages, H, size, D), dtype=np.uint8)).cuda()
    if strided:  # K and V side by side, heads behind tokens
        codes = torch.from_numpy(r.integers(0, 256, (pages, size, H, 2 * D), dtype=np.uint8)).cuda()
        codes = (codes[..., :D].permute(0, 2, 1, 3), codes[..., D:].permute(0, 2, 1, 3))
    scales = torch.from_numpy(r.random((2, pages, H), dtype=np.float32)).cuda()
    return dict(k_cache=codes[0], v_cache=codes[1], k_scale=scales[0].clone(), v_scale=scales[1].clone(),
                page_table=ints(table), seq_lens=ints(lens)), ints(count)


def numbers(cache, count):
    return cache["page_table"].tolist(), cache["seq_lens"].tolist(), count.tolist(), cache["k_cache"].shape[2]


def data(cache):
    return [cache[k].clone() for k in ("k_cache", "v_cache", "k_scale", "v_scale")]


def copied(before, moves):
    """The cache's arrays after pages were copied: (from, to, tokens or None for all)."""
    k, v, ks, vs = [x.clone() for x in before]
    for m in moves:
        a, b, t = m if len(m) == 3 else (*m, None)
        for x, y in ((k, before[0]), (v, before[1])):
            x[b, :, :t] = y[a, :, :t]
        for x, y in ((ks, before[2]), (vs, before[3])):
            x[b] = y[a]
    return [k, v, ks, vs]


def same(got, want):
    for x, y in zip(got, want):
        assert torch.equal(x, y)


SHAPES = [  # lens, page size, entries, pages, share
    ([1], 16, 1, 1, 1),
    ([0, 5], 16, 2, 9, 1),
    ([16, 17, 31, 32, 33], 16, 4, 20, 1),
    ([40] * 6, 16, 5, 30, 3),
    ([300, 2, 999, 64] * 5, 64, 20, 400, 2),
    ([130] * 16, 128, 4, 60, 8),
    ([9000, 1, 4097], 32, 300, 5000, 1),
    ([-3, 10 ** 6, 20], 16, 6, 40, 1),      # clamped to [0, 96]
]


@pytest.mark.parametrize("lens,size,P,pages,share", SHAPES)
@pytest.mark.parametrize("in_place", [False, True])
def test_fork(tv, lens, size, P, pages, share, in_place):
    cache, count = pool(1, lens, size, P, pages, share)
    B = len(lens)
    for sources in ([0], list(range(B)), [B - 1] * 7 + [-1, B, 0]):
        want = ref.fork(*numbers(cache, count)[:2], sources, count.tolist(), size)
        c = count.clone()
        kw = {} if in_place else dict(refcount_out=torch.full_like(c, 77))
        got = tv.kv_fork(**cache, sources=ints(sources), refcount=c, **kw)
        assert got["page_table"].tolist() == want[0]
        assert got["seq_lens"].tolist() == want[1]
        assert got["refcount"].tolist() == want[2]
        assert got["refcount"] is (c if in_place else kw["refcount_out"])
        if not in_place:
            assert torch.equal(c, count)


@pytest.mark.parametrize("lens,size,P,pages,share", SHAPES)
@pytest.mark.parametrize("in_place", [False, True])
def test_free(tv, lens, size, P, pages, share, in_place):
    cache, count = pool(2, lens, size, P, pages, share)
    for release in (None, [b % 2 for b in range(len(lens))], [0] * len(lens)):
        want = ref.free(*numbers(cache, count)[:2], release or [1] * len(lens), count.tolist(), size)
        c = count.clone()
        kw = {} if in_place else dict(refcount_out=torch.full_like(c, 77))
        got = tv.kv_free(**cache, refcount=c, release=None if release is None else ints(release), **kw)
        if release is None:
            want = ref.free(*numbers(cache, count)[:2], [1] * len(lens), count.tolist(), size)
        assert got.tolist() == want


@pytest.mark.parametrize("lens,size,P,pages,share", SHAPES)
@pytest.mark.parametrize("grow", ["one", "mixed", "far"])
@pytest.mark.parametrize("in_place", [False, True])
def test_reserve(tv, lens, size, P, pages, share, grow, in_place):
    cache, count = pool(3, lens, size, P, pages, share, strided=share == 2, D=128 if share == 8 else 64)
    table, now, cnt, _ = numbers(cache, count)
    r = np.random.default_rng(4)
    new = {"one": [x + 1 for x in now], "mixed": [x + int(r.integers(-2, 2 * size)) for x in now],
           "far": [x + 10 ** 7 for x in now]}[grow]
    new = [min(x, 2 ** 31 - 1) for x in new]
    want = ref.reserve(table, now, new, cnt, size)
    before, c = data(cache), count.clone()
    kw = {} if in_place else dict(refcount_out=torch.full_like(c, 77), page_table_out=torch.full_like(cache["page_table"], 55))
    got = tv.kv_reserve(**cache, new_lens=ints(new), refcount=c, **kw)
    assert got["reserved"].tolist() == want[2]
    assert got["page_table"].tolist() == want[0]
    assert got["refcount"].tolist() == want[1]
    same(data(cache), copied(before, want[3]))
    if in_place:
        assert got["page_table"] is cache["page_table"] and got["refcount"] is c
    else:
        assert cache["page_table"].tolist() == table and torch.equal(c, count)


@pytest.mark.parametrize("missing", [0, 1, 2, 5, 1000])
def test_reserve_from_a_pool_that_runs_out(tv, missing):
    lens = [40] * 4 + [17] * 4 + [64] * 4 + [5] * 4
    cache, count = pool(5, lens, 16, 8, 40, share=4)
    # the last context has a holder outside the batch; free pages are taken until few are left
    count[cache["page_table"][12, 0]] += 1
    table, now, cnt, _ = numbers(cache, count)
    new = [x + 20 if b % 3 else x for b, x in enumerate(now)]
    for p in [p for p in range(40) if cnt[p] == 0][: missing * 3]:
        count[p] = -1 if p % 2 else 1
    cnt = count.tolist()
    want = ref.reserve(table, now, new, cnt, 16)
    before = data(cache)
    got = tv.kv_reserve(**cache, new_lens=ints(new), refcount=count)
    assert got["reserved"].tolist() == want[2]
    assert got["page_table"].tolist() == want[0] and count.tolist() == want[1]
    same(data(cache), copied(before, want[3]))


def test_the_last_holder_keeps_its_page_only_when_the_others_are_served(tv):
    # three holders of page 2, all growing: two copies and one that keeps it; a free page less and
    # the second copy and the keeper both wait
    for spare, reserved in ((2, [6, 6, 6]), (1, [6, 5, 5]), (0, [5, 5, 5])):
        cache, count = pool(6, [5], 16, 2, 3 + spare, H=1)
        cache["page_table"] = ints([[2, -1]] * 3)
        cache["seq_lens"] = ints([5] * 3)
        count = ints([1, 1, 3] + [0] * spare)
        got = tv.kv_reserve(**cache, new_lens=ints([6] * 3), refcount=count)
        assert got["reserved"].tolist() == reserved
        assert got["page_table"][:, 0].tolist() == [3, 4, 2][:spare] + [2] * (3 - spare)
        assert count.tolist() == [1, 1, 3 - spare] + [1] * spare


@pytest.mark.parametrize("lens,size,P,pages,share", SHAPES)
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(tv, lens, size, P, pages, share, in_place):
    cache, count = pool(7, lens, size, P, pages, share, strided=share == 2, D=128 if share == 8 else 64)
    r = np.random.default_rng(8)
    used = torch.nonzero(count).squeeze(1).tolist()
    for p in used[::3]:  # an entry whose page is free or whose count is wrong
        count[p] = int(r.integers(-1, 1))
    table, now, cnt, _ = numbers(cache, count)
    want = ref.compact(table, now, cnt, size)
    before, c = data(cache), count.clone()
    kw = {} if in_place else dict(refcount_out=torch.full_like(c, 77), page_table_out=torch.full_like(cache["page_table"], 55))
    got = tv.kv_compact(**cache, refcount=c, **kw)
    assert got["live"].tolist() == [want[2]]
    assert got["page_table"].tolist() == want[0]
    assert got["refcount"].tolist() == want[1]
    same(data(cache), copied(before, want[3]))


@pytest.mark.parametrize("fill", [0, 1])
def test_compact_of_an_empty_and_of_a_full_pool(tv, fill):
    cache, count = pool(9, [16, 16], 16, 1, 2, H=1)
    count = ints([fill] * 2)
    before = data(cache)
    got = tv.kv_compact(**cache, refcount=count)
    assert got["live"].tolist() == [2 * fill] and count.tolist() == [fill] * 2
    assert (got["page_table"] == -1).all().item() == (not fill)
    same(data(cache), before)


def test_large_pools_and_batches(tv):
    # more pages than the chunks of 2048 that are looked at side by side; more requests than a CTA
    # has threads; a request that asks for thousands of pages
    pages, size, B = 2_300_001, 16, 700
    r = np.random.default_rng(10)
    count = (r.random(pages) < 0.97).astype(np.int64)
    P = 9000
    table = np.full((B, P), -1, np.int64)
    lens = r.integers(0, 40, B)
    lens[13] = 16 * 100 + 3
    held = np.nonzero(count)[0]
    at = 0
    for b in range(0, B, 2):
        lens[b + 1] = lens[b]
        n = ref.entries(int(lens[b]), size)
        table[b:b + 2, :n] = held[at:at + n]
        count[held[at:at + n]] = 2
        at += n
    cache = dict(k_cache=torch.zeros((pages, 1, size, 64), dtype=torch.uint8, device="cuda"))
    cache["v_cache"] = cache["k_cache"].clone()
    cache["k_cache"][:, 0, 0, 0] = torch.arange(pages, device="cuda").to(torch.uint8)
    cache["k_scale"] = torch.arange(pages, device="cuda").float().view(-1, 1)
    cache["v_scale"] = -cache["k_scale"]
    cache["page_table"], cache["seq_lens"] = ints(table), ints(lens)
    new = lens + r.integers(0, 3, B)
    new[77] = 16 * 8000
    want = ref.reserve(table.tolist(), lens.tolist(), new.tolist(), count.tolist(), size)
    before = data(cache)
    cnt = ints(count)
    out = torch.empty_like(cache["page_table"])
    got = tv.kv_reserve(**cache, new_lens=ints(new), refcount=cnt, page_table_out=out)
    assert got["reserved"].tolist() == want[2]
    assert torch.equal(out, ints(want[0])) and torch.equal(cnt, ints(want[1]))
    same(data(cache), copied(before, want[3]))
    cache["page_table"], cache["seq_lens"] = out, got["reserved"]
    t, c, n, moves = ref.compact(out.tolist(), got["reserved"].tolist(), cnt.tolist(), size)
    before = data(cache)
    got = tv.kv_compact(**cache, refcount=cnt)
    assert got["live"].item() == n and torch.equal(cnt, ints(c)) and torch.equal(out, ints(t))
    a, b = (torch.tensor(x, device="cuda") for x in zip(*moves))
    for x, y in zip(data(cache), before):
        y[b] = y[a]
        assert torch.equal(x, y)


def test_offsets_past_32_bits(tv):
    # pages of 2 x 8 heads x 128 x 128 bytes, the last of them 4.5 GB behind the first
    pages = 36000
    cache, _ = pool(11, [5, 5], 16, 3, 4, H=1)
    k = torch.zeros((pages, 8, 128, 128), dtype=torch.uint8, device="cuda")
    cache = dict(k_cache=k, v_cache=k.view(pages, 8, 128, 128), k_scale=torch.zeros((pages, 8), device="cuda"),
                 v_scale=torch.zeros((pages, 8), device="cuda"), page_table=ints([[pages - 1, -1]] * 2),
                 seq_lens=ints([100, 100]))
    k[pages - 1] = 7
    cache["k_scale"][pages - 1] = 3
    count = torch.zeros(pages, dtype=torch.int32, device="cuda")
    count[pages - 1] = 2
    count[:pages - 2] = 1
    got = tv.kv_reserve(**cache, new_lens=ints([101, 100]), refcount=count)
    assert got["page_table"][:, 0].tolist() == [pages - 2, pages - 1]
    assert (k[pages - 2, :, :100] == 7).all() and (k[pages - 2, :, 100:] == 0).all() and (cache["k_scale"][pages - 2] == 3).all()
    count[:pages - 2] = 0
    got = tv.kv_compact(**cache, refcount=count)
    assert got["page_table"][:, 0].tolist() == [0, 1] and got["live"].item() == 2
    assert (k[0, :, :100] == 7).all() and (k[1] == 7).all()


def test_a_step_of_branching_requests(tv):
    """A prompt, four answers, tokens appended to each: what the answers read back is what was
    appended, and in the end every page is free."""
    H, D, size, pages = 2, 64, 16, 40
    g = torch.Generator().manual_seed(0)
    z = torch.zeros((2, pages, H, size, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    sc = torch.ones((2, pages, H), device="cuda")
    kv = dict(k_cache=z[0], v_cache=z[1], k_scale=sc[0], v_scale=sc[1])
    count = torch.zeros(pages, dtype=torch.int32, device="cuda")
    cache = dict(kv, page_table=torch.full((1, 6), -1, dtype=torch.int32, device="cuda"), seq_lens=ints([0]))
    tv.kv_reserve(**cache, new_lens=ints([37]), refcount=count)
    x = torch.randn((2, 37, H, D), generator=g).cuda().half()
    tv.kv_append(x[0], x[1], **cache)
    cache["seq_lens"] += 37
    f = tv.kv_fork(**cache, sources=ints([0] * 4), refcount=count)
    tv.kv_free(**cache, refcount=count)
    assert count.sum().item() == 12 and count.max().item() == 4
    cache = dict(kv, page_table=f["page_table"], seq_lens=f["seq_lens"])
    y = torch.randn((2, 4 * 9, H, D), generator=g).cuda().half()
    r = tv.kv_reserve(**cache, new_lens=cache["seq_lens"] + 9, refcount=count)
    assert r["reserved"].tolist() == [46] * 4 and (count > 0).sum().item() == 6
    tv.kv_append(y[0], y[1], **cache)
    cache["seq_lens"] += 9
    tv.kv_compact(**cache, refcount=count)
    assert torch.equal(count > 0, torch.arange(pages, device="cuda") < 6)
    got = tv.kv_read(**cache, out_indptr=ints([0, 46, 92, 138, 184]), total_rows=184, dtype=torch.float32)
    for name, i in (("k", 0), ("v", 1)):
        for b in range(4):
            rows = torch.cat([x[i], y[i, 9 * b:9 * b + 9]])
            # the last prompt page's scale may have grown: its codes are rounded twice
            want = rows.float()
            err = (got[name][46 * b:46 * b + 46] - want).abs()
            assert (err <= want.abs() * (2.0 ** -4 + 2.0 ** -4 * 1.0625) + 2.0 ** -9).all()
    tv.kv_free(**cache, refcount=count)
    assert (count == 0).all()


def test_captured_with_other_lengths_and_on_another_stream(tv):
    cache, count = pool(12, [40] * 6, 16, 8, 60, share=3)
    new, sources = ints([0] * 6), ints([0] * 4)
    out = dict(refcount_out=torch.empty_like(count), page_table_out=torch.empty_like(cache["page_table"]))
    ws = tv.make_pages_workspace(6, 60)
    side = torch.cuda.Stream()
    before = data(cache)

    def step():
        f = tv.kv_fork(**cache, sources=sources, refcount=count, refcount_out=torch.empty_like(count))
        return f, tv.kv_reserve(**cache, new_lens=new, refcount=count, workspace=ws, **out)

    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f, r = step()
    for k in (0, 1, 30):
        new.copy_(cache["seq_lens"] + k)
        sources.copy_(ints([k % 6, 5, 0, -1]))
        for x, y in zip([cache[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")], before):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        table, now, cnt, size = numbers(cache, count)
        want = ref.reserve(table, now, new.tolist(), cnt, size)
        assert r["reserved"].tolist() == want[2] and r["page_table"].tolist() == want[0] and r["refcount"].tolist() == want[1]
        same(data(cache), copied(before, want[3]))
        assert f["refcount"].tolist() == ref.fork(table, now, sources.tolist(), cnt, size)[2]
    # by the stream argument
    c2 = count.clone()
    torch.cuda.synchronize()
    got = tv.kv_free(**cache, refcount=c2, stream=side)
    side.synchronize()
    assert got.tolist() == ref.free(table, now, [1] * 6, cnt, size)
