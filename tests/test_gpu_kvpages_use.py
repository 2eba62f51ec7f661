"""The calls on the cache's pages as a server makes them, step by step."""
import numpy as np
import pytest
import torch

from tests.test_gpu_kvpages import data, same
from tests.test_gpu_shared import check, ints, tv  # noqa: F401 (tv: a fixture)
from tests.window_ref import F8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("pages", [300, 16])
def test_answers_that_grow_until_the_pool_ends(tv, pages, D):  # noqa: F811
    """The README's example, in a pool that is large and one that runs out: what an answer reads back is what
    it was given, whoever got no page, and attention is that of its own tokens."""
    H, Hq, size, T, n = 2, 8, 16, 12, 5
    g = torch.Generator("cuda").manual_seed(1)
    r = np.random.default_rng(1)
    z = torch.zeros((2, pages, H, size, D), dtype=torch.uint8, device="cuda").view(F8)
    sc = torch.ones((2, pages, H), device="cuda")
    kv = dict(k_cache=z[0], v_cache=z[1], k_scale=sc[0], v_scale=sc[1])
    count = torch.zeros(pages, dtype=torch.int32, device="cuda")
    cache = dict(kv, page_table=torch.full((1, 30), -1, dtype=torch.int32, device="cuda"), seq_lens=ints([0]))
    prompt = ints([70])

    def rows(h):  # one scale for all, so that codes are exact
        x = torch.randint(-7, 8, (h, H, D), generator=g, device="cuda").bfloat16() / 4
        x[..., 0] = 1.75
        return x

    first = rows(70), rows(70)
    tv.kv_reserve(**cache, new_lens=prompt, refcount=count)
    tv.kv_append(*first, **cache)
    cache["seq_lens"] += prompt
    f = tv.kv_fork(**cache, sources=ints([0] * n), refcount=count)
    tv.kv_free(**cache, refcount=count)
    cache = dict(kv, page_table=f["page_table"], seq_lens=f["seq_lens"])
    held = cache["seq_lens"].clone()
    want = [list(first) for _ in range(n)]
    ptr, index = ints(np.arange(n + 1) * T), ints(np.arange(n * T).reshape(n, T))
    refused = 0
    for _ in range(5):
        q = torch.randn((n * T, Hq, D), generator=g, device="cuda").bfloat16()
        k, v = rows(n * T), rows(n * T)
        accepted = ints(1 + r.integers(0, T, n))
        c = dict(cache, q=q, k_new=k, v_new=v, qo_indptr=ptr, group_indptr=ints([0, n]), shared_lens=prompt)
        check(c, tv.shared_attention(**c, lse=True))
        room = tv.kv_reserve(**cache, new_lens=cache["seq_lens"] + T, held_lens=held, refcount=count)["reserved"]
        held = torch.maximum(held, room)
        kept = torch.minimum(accepted, room - cache["seq_lens"])
        refused += int((kept < accepted).sum())
        tv.kv_append(k, v, **cache, src_index=index, src_len=kept)
        cache["seq_lens"] += kept
        for b, m in enumerate(kept.tolist()):
            want[b] = [torch.cat([w, x[b * T:b * T + m]]) for w, x in zip(want[b], (k, v))]
        at = [0] + list(np.cumsum(cache["seq_lens"].tolist()))
        back = tv.kv_read(**cache, out_indptr=ints(at), total_rows=at[-1], dtype=torch.bfloat16)
        for b in range(n):
            for w, name in zip(want[b], "kv"):
                assert torch.equal(back[name][at[b]:at[b + 1]], w)
    assert (refused > 0) == (pages == 16)
    tv.kv_free(**cache, held_lens=held, refcount=count)
    assert (count == 0).all()


@pytest.mark.parametrize("split", [False, True])
def test_layers_under_one_table(tv, split):  # noqa: F811
    """Three layers, a pool each: a step's calls once a layer, from the same tables and counts into the same others
    (or, split, the last one in place). Every layer reads back what it was given."""
    H, D, size, pages, layers, n = 2, 64, 16, 60, 3, 4
    g = torch.Generator("cuda").manual_seed(2)
    z = torch.zeros((layers, 2, pages, H, size, D), dtype=torch.uint8, device="cuda").view(F8)
    sc = torch.ones((layers, 2, pages, H), device="cuda")
    pools = [dict(k_cache=z[i, 0], v_cache=z[i, 1], k_scale=sc[i, 0], v_scale=sc[i, 1]) for i in range(layers)]
    count, count2 = torch.zeros((2, pages), dtype=torch.int32, device="cuda")
    table, table2 = torch.full((2, n, 10), -1, dtype=torch.int32, device="cuda")
    lens = ints([0] * n)
    want = [[[torch.zeros((0, H, D), device="cuda")] * 2 for _ in range(n)] for _ in range(layers)]

    def each(call, **kw):
        """The call a layer; the tables and counts are the new ones then."""
        nonlocal table, table2, count, count2
        got = []
        for i, kv in enumerate(pools):
            out = {} if split and i == layers - 1 else dict(page_table_out=table2, refcount_out=count2)
            got.append(call(**kv, page_table=table, seq_lens=lens, refcount=count, **kw, **out))
        assert all(torch.equal(a[k], got[0][k]) for a in got for k in a)
        if not split:
            table, table2, count, count2 = table2, table, count2, count

    for step in range(4):
        grown = ints([37, 0, 0, 0] if step == 0 else [5 + (b + step) % 9 for b in range(n)])
        each(tv.kv_reserve, new_lens=lens + grown)
        if step == 2:
            each(tv.kv_compact, held_lens=lens + grown)
        ptr = [0] + list(np.cumsum(grown.tolist()))
        for i, kv in enumerate(pools):
            x = torch.randint(-7, 8, (2, ptr[-1], H, D), generator=g, device="cuda").half() * 64
            x[..., 0] = 448  # one scale for all: codes are exact
            tv.kv_append(x[0], x[1], **kv, page_table=table, seq_lens=lens, qo_indptr=ints(ptr))
            for b in range(n):
                want[i][b] = [torch.cat([w, y[ptr[b]:ptr[b + 1]].float()]) for w, y in zip(want[i][b], x)]
        lens += grown
        if step == 0:  # all continue the first: the tables and counts once
            f = tv.kv_fork(**pools[0], page_table=table, seq_lens=lens, sources=ints([0] * n), refcount=count)
            tv.kv_free(**pools[0], page_table=table, seq_lens=lens, refcount=count)
            table.copy_(f["page_table"])
            lens.copy_(f["seq_lens"])
            want = [[w[0]] * n for w in want]
        at = [0] + list(np.cumsum(lens.tolist()))
        for i, kv in enumerate(pools):
            back = tv.kv_read(**kv, page_table=table, seq_lens=lens, out_indptr=ints(at), total_rows=at[-1], dtype=torch.float32)
            for b in range(n):
                for w, name in zip(want[i][b], "kv"):
                    assert torch.equal(back[name][at[b]:at[b + 1]], w), (step, i, b, name)
    tv.kv_free(**pools[0], page_table=table, seq_lens=lens, refcount=count)
    assert (count == 0).all()


def test_pools_of_their_own_past_32_bits(tv):  # noqa: F811
    # K and V of 36000 pages of 8 heads x 128 x 128 bytes each, apart, with what differs in every page, head and
    # of K and V: a copy and a move between pages 4.7 GB apart
    pages, H, size, D = 36000, 8, 128, 128
    kv = {}
    for i, name in enumerate("kv"):
        x = torch.zeros((pages, H, size, D), dtype=torch.uint8, device="cuda")
        for p in (pages - 1, pages - 2, 0, 1):
            x[p] = torch.arange(size * D, device="cuda").view(size, D) % 100 + torch.arange(H, device="cuda")[:, None, None] + 10 * i + p % 5
        kv[name + "_cache"] = x
        kv[name + "_scale"] = torch.arange(pages, device="cuda").float()[:, None] + torch.arange(H, device="cuda") / 16 + 0.5 * i
    cache = dict(kv, page_table=ints([[pages - 1, -1]] * 2), seq_lens=ints([100, 100]))
    count = torch.ones(pages, dtype=torch.int32, device="cuda")
    count[pages - 1], count[1] = 2, 0
    k, v, ks, vs = data(cache)
    got = tv.kv_reserve(**cache, new_lens=ints([101, 100]), refcount=count)
    assert got["page_table"][:, 0].tolist() == [1, pages - 1]
    for x in (k, v):
        x[1, :, :100] = x[pages - 1, :, :100]
    for x in (ks, vs):
        x[1] = x[pages - 1]
    same(data(cache), [k, v, ks, vs])
    count[2:pages - 2] = 0
    got = tv.kv_compact(**cache, refcount=count)  # 0 and 1 stay, the last two come to 2 and 3
    assert got["live"].item() == 4 and got["page_table"][:, 0].tolist() == [1, 3]
    for x in (k, v, ks, vs):
        x[2], x[3] = x[pages - 2], x[pages - 1]
    same(data(cache), [k, v, ks, vs])
