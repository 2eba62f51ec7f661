"""The calls on the cache's pages where requests have room for more tokens than they hold: every result is
a whole number or a copied byte, so all of them have to be equal."""
import numpy as np
import pytest
import torch

from tests import pages_ref as ref
from tests.test_gpu_kvpages import copied, data, ints, numbers, pool, same, tv  # noqa: F401 (tv: a fixture)

pytestmark = pytest.mark.gpu


def reserve(table, lens, held, new_lens, count, size):
    """pages_ref.reserve where request b has the pages of held[b] tokens: table, count, reserved, copies."""
    P, N = len(table[0]), len(count)
    cap = P * size
    lens = [min(max(x, 0), cap) for x in lens]
    held = [max(x, min(h, cap)) for x, h in zip(lens, held)]
    want = [max(x, min(w, cap)) for x, w in zip(lens, new_lens)]
    rows = [list(t[: ref.entries(h, size)]) for t, h in zip(table, held)]
    before, count = list(count), list(count)
    free = [p for p in range(N) if before[p] <= 0]
    last = []
    for b, row in enumerate(rows):
        p = row[lens[b] // size] if want[b] > lens[b] and lens[b] % size else -1
        last.append(p if 0 <= p < N and before[p] > 1 else None)
    keepers = {max(b for b, q in enumerate(last) if q == p) for p in set(last) - {None} if last.count(p) >= before[p]}
    reserved, copies, asked = [], [], 0
    for b, row in enumerate(rows):
        copy = last[b] is not None and b not in keepers
        n = max(ref.entries(want[b], size) - len(row), 0) + copy
        given = free[asked:asked + n]
        asked += n
        if asked > len(free) and (n > 0 or b in keepers):
            reserved.append(lens[b])
            continue
        reserved.append(want[b])
        for p in given:
            count[p] = 1
        if copy:
            copies.append((last[b], given[0], lens[b] % size))
            count[last[b]] -= 1
            row[lens[b] // size] = given[0]
        row.extend(given[copy:])
    return [r + [-1] * (P - len(r)) for r in rows], count, reserved, copies


def holding(seed, B, size, P, pages, share):
    """A pool whose requests have pages behind those of their tokens; share: requests of a context."""
    cache, count = pool(seed, [size * (1 + b % (P // 2)) - (7 * b) % size for b in range(B)], size, P, pages, share)
    r = np.random.default_rng(seed + 1)
    table, lens, cnt, _ = numbers(cache, count)
    free = [p for p in range(pages) if cnt[p] == 0]
    held = []
    for b in range(B):
        n = ref.entries(lens[b], size)
        more = min(int(r.integers(0, 3)), P - n)
        for j in range(n, n + more):
            table[b][j] = free.pop(0)
            cnt[table[b][j]] = 1
        held.append([lens[b] - 9, (n + more) * size - int(r.integers(0, size))][more > 0])  # less than it has: none more
    cache["page_table"] = ints(table)
    return cache, ints(cnt), held


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,size,P,pages,share", [(1, 16, 2, 4, 1), (12, 16, 8, 90, 3), (24, 64, 6, 70, 4), (300, 32, 10, 2600, 2)])
@pytest.mark.parametrize("grow", ["within", "one", "mixed", "far"])
def test_reserve(tv, grow, B, size, P, pages, share, in_place):  # noqa: F811
    cache, count, held = holding(41, B, size, P, pages, share)
    table, lens, cnt, _ = numbers(cache, count)
    r = np.random.default_rng(43)
    new = {"within": [max(h, n) for h, n in zip(held, lens)], "one": [n + 1 for n in lens],
           "mixed": [n + int(r.integers(-3, 3 * size)) for n in lens], "far": [2 ** 31 - 1] * B}[grow]
    want = reserve(table, lens, held, new, cnt, size)
    before, c = data(cache), count.clone()
    kw = {} if in_place else dict(refcount_out=torch.full_like(c, 77), page_table_out=torch.full_like(cache["page_table"], 55))
    got = tv.kv_reserve(**cache, new_lens=ints(new), held_lens=ints(held), refcount=c, **kw)
    assert got["reserved"].tolist() == want[2]
    assert got["page_table"].tolist() == want[0] and got["refcount"].tolist() == want[1]
    same(data(cache), copied(before, want[3]))


@pytest.mark.parametrize("B,size,P,pages,share", [(1, 16, 2, 4, 1), (12, 16, 8, 90, 3), (24, 64, 6, 70, 4)])
def test_free_and_compact(tv, B, size, P, pages, share):  # noqa: F811
    cache, count, held = holding(44, B, size, P, pages, share)
    table, lens, cnt, _ = numbers(cache, count)
    most = [max(a, b) for a, b in zip(lens, held)]
    for release in (None, [b % 2 for b in range(B)]):
        got = tv.kv_free(**cache, refcount=count, held_lens=ints(held), refcount_out=torch.empty_like(count),
                         release=None if release is None else ints(release))
        assert got.tolist() == ref.free(table, most, release or [1] * B, cnt, size)
    want = ref.compact(table, most, cnt, size)
    before = data(cache)
    got = tv.kv_compact(**cache, refcount=count, held_lens=ints(held))
    assert got["live"].tolist() == [want[2]] and got["page_table"].tolist() == want[0] and count.tolist() == want[1]
    same(data(cache), copied(before, want[3]))


def test_lengths_out_of_range(tv):  # noqa: F811
    # held lengths below seq_len and below nothing count as seq_len, those past the table as all of it
    cache, count, _ = holding(45, 6, 16, 4, 40, 1)
    table, lens, cnt, _ = numbers(cache, count)
    for held in ([-2 ** 31] * 6, [0] * 6, [2 ** 31 - 1] * 6):
        want = reserve(table, lens, held, [x + 20 for x in lens], cnt, 16)
        got = tv.kv_reserve(**cache, new_lens=ints([x + 20 for x in lens]), held_lens=ints(held), refcount=count,
                            refcount_out=torch.empty_like(count), page_table_out=torch.empty_like(cache["page_table"]))
        assert got["reserved"].tolist() == want[2] and got["page_table"].tolist() == want[0]
        assert got["refcount"].tolist() == want[1]


@pytest.mark.parametrize("pages", [200, 26, 14])
def test_drafts_that_are_not_accepted(tv, pages):  # noqa: F811
    """Each step reserves room for all it drafts and appends what is accepted, with a fork, compacting and
    requests that end on the way, in a pool that is large and one that runs out: what is read back is
    what was appended, and in the end no page is held."""
    H, D, size, P, B, T = 2, 64, 16, 20, 6, 40
    g = torch.Generator("cuda").manual_seed(0)
    r = np.random.default_rng(0)
    z = torch.zeros((2, pages, H, size, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    sc = torch.ones((2, pages, H), device="cuda")
    kv = dict(k_cache=z[0], v_cache=z[1], k_scale=sc[0], v_scale=sc[1])
    count = torch.zeros(pages, dtype=torch.int32, device="cuda")
    cache = dict(kv, page_table=torch.full((1, P), -1, dtype=torch.int32, device="cuda"), seq_lens=ints([0]))
    assert tv.kv_reserve(**cache, new_lens=ints([45]), refcount=count)["reserved"].tolist() == [45]
    x = torch.randint(-7, 8, (2, 45, H, D), generator=g, device="cuda").half() * 64  # one scale for all: codes are exact
    x[..., 0] = 448
    tv.kv_append(x[0], x[1], **cache)
    cache["seq_lens"] += 45
    f = tv.kv_fork(**cache, sources=ints([0] * B), refcount=count)
    tv.kv_free(**cache, refcount=count, held_lens=ints([45]))
    cache = dict(kv, page_table=f["page_table"], seq_lens=f["seq_lens"])
    held = cache["seq_lens"].clone()
    rows = [x for _ in range(B)]
    short = 0
    for step in range(6):
        y = torch.randint(-7, 8, (2, B * T, H, D), generator=g, device="cuda").half() * 64
        y[..., 0] = 448
        accepted = ints(r.integers(0, T if pages > 100 else 9, B))
        got = tv.kv_reserve(**cache, new_lens=cache["seq_lens"] + (T if pages > 100 else 20), refcount=count, held_lens=held)
        held = torch.maximum(held, got["reserved"])
        if step in (1, 3):
            tv.kv_compact(**cache, refcount=count, held_lens=held)
            assert torch.equal(count > 0, torch.arange(pages, device="cuda") < (count > 0).sum())
        index = torch.arange(B * T, dtype=torch.int32, device="cuda").view(B, T)
        take = torch.minimum(accepted, got["reserved"] - cache["seq_lens"])
        short += int((take < accepted).sum())
        tv.kv_append(y[0], y[1], **cache, src_index=index, src_len=take)
        cache["seq_lens"] += take
        for b, n in enumerate(take.tolist()):
            rows[b] = torch.cat([rows[b], y[:, b * T:b * T + n]], 1)
        if step == 3:  # a request ends and another takes its place, from one that goes on
            gone = ints([1] + [0] * (B - 1))
            tv.kv_free(**cache, refcount=count, release=gone, held_lens=held)
            f = tv.kv_fork(**cache, sources=ints([1]), refcount=count)
            cache["page_table"][0], cache["seq_lens"][0] = f["page_table"][0], f["seq_lens"][0]
            held[0] = cache["seq_lens"][0]
            rows[0] = rows[1]
        lens = cache["seq_lens"].tolist()
        ptr = [0] + list(np.cumsum(lens))
        back = tv.kv_read(**cache, out_indptr=ints(ptr), total_rows=ptr[-1], dtype=torch.float32)
        for b in range(B):
            for i, name in enumerate("kv"):
                assert torch.equal(back[name][ptr[b]:ptr[b + 1]], rows[b][i].float()), (step, b)
    assert short == 0 if pages == 200 else short > 0 or pages == 26
    tv.kv_free(**cache, refcount=count, held_lens=held)
    assert (count == 0).all()


def test_captured(tv):  # noqa: F811
    cache, count, held = holding(46, 12, 16, 8, 90, 3)
    table, lens, cnt, _ = numbers(cache, count)
    new, h = ints(lens), ints(held)
    out = dict(refcount_out=torch.empty_like(count), page_table_out=torch.empty_like(cache["page_table"]))
    ws = tv.make_pages_workspace(12, 90)
    before = data(cache)
    tv.kv_reserve(**cache, new_lens=new, held_lens=h, refcount=count, workspace=ws, **out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = tv.kv_reserve(**cache, new_lens=new, held_lens=h, refcount=count, workspace=ws, **out)
    for k in (1, 17, 60):
        for a, b in zip((cache[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")), before):
            a.copy_(b)
        new.copy_(ints([x + k for x in lens]))
        h.copy_(ints([x - k // 3 for x in held]))
        graph.replay()
        torch.cuda.synchronize()
        want = reserve(table, lens, [x - k // 3 for x in held], [x + k for x in lens], cnt, 16)
        assert got["reserved"].tolist() == want[2] and got["page_table"].tolist() == want[0]
        assert got["refcount"].tolist() == want[1]
        same(data(cache), copied(before, want[3]))
