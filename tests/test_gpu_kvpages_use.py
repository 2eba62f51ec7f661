"""The calls on the cache's pages as a server makes them, step by step."""
import numpy as np
import pytest
import torch

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
