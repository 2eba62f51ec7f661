"""GPU: window attention with head_dim 128 (its own kernel) where it can go wrong, and a decoding
step that runs the operators together. Bounds as in tests/window_ref.py."""
import math

import numpy as np
import pytest
import torch

from speculative_decoding_verify_temp_gb300 import tsverify as tv
from tests import window_ref as ref
from tests.test_gpu_window import _built, check, make, two_parts, wanted  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


def run(s, windows, lens, sm_scale=None, **kw):
    got = tv.window_attention(**s, sm_scale=sm_scale, lse=True, **kw)
    check(got, wanted(s, windows, lens, sm_scale), s["q"].dtype, 128, two_parts(s))
    return got


CASES = [
    # windows, lens, Hq, H, page, dtype, mask, layout
    ([33, 16], [130, 255], 4, 2, 16, F16, "tree", "pages"),            # blocks of 64 rows, three parts
    ([33, 16], [130, 255], 4, 2, 16, BF16, "tree", "pages"),           # two parts
    ([16], [1000], 8, 2, 128, BF16, "chain", "tokens"),                # 64 rows exactly
    ([65], [513], 8, 2, 32, BF16, "tree", "pool"),                     # several blocks of rows
    ([65], [513], 8, 2, 32, F16, "chain", "pages"),
    ([1, 2, 3, 1, 5], [0, 127, 128, 129, 384], 32, 4, 64, BF16, "chain", "pages"),
    ([1] * 3, [0, 0, 0], 8, 2, 16, BF16, "none", "pages"),             # nothing anywhere
    ([2] * 400, [(i * 61) % 300 for i in range(400)], 8, 1, 64, BF16, "chain", "pages"),
    ([8] * 160, [(i * 29) % 130 for i in range(160)], 8, 1, 16, F16, "tree", "pages"),
    ([1] * 90, [0 if i % 3 else 17 * i for i in range(90)], 4, 4, 16, BF16, "none", "tokens"),
    ([1] * 512, [40] * 512, 2, 2, 128, F16, "chain", "pages"),         # units of one tile
    ([2], [60011], 4, 1, 16, BF16, "chain", "pages"),                  # a line over all multiprocessors
    ([20], [30003], 4, 1, 128, BF16, "tree", "pages"),
]


@pytest.mark.parametrize("case", CASES,
                         ids=lambda c: f"{len(c[0])}x{max(c[0])}_{max(c[1])}_{c[2]}x{c[3]}_{c[4]}_{c[6]}")
def test_attention(case):
    windows, lens, Hq, H, size, dtype, mask, layout = case
    s = make(21, windows, lens, Hq, H, 128, size, dtype, mask, layout)
    got = run(s, windows, lens)
    again = tv.window_attention(**s, lse=True)
    assert torch.equal(got["out"], again["out"]) and torch.equal(got["lse"], again["lse"])


@pytest.mark.parametrize("rows", [3, 40])
def test_scales_far_apart(rows):
    s = make(22, [rows], [290], 2, 1, 128, 16, BF16, vscale=(-59, 9), garbage=False)
    s["k_scale"].fill_(2.0 ** -7)
    run(s, [rows], [290])


@pytest.mark.parametrize("rows", [2, 20])
@pytest.mark.parametrize("scale", [1.0, 0.0, -0.3])
def test_scale_and_large_scores(rows, scale):
    windows, lens = [rows, 2], [400, 77]
    run(make(23, windows, lens, 4, 2, 128, 16, BF16, vscale=(-3, 3)), windows, lens, scale)


def test_scores_that_rise_along_the_line():
    # every block's largest score is above the block's before: the references follow each time
    windows, lens = [2, 40], [1500, 1400]
    for dtype in (BF16, F16):
        s = make(24, windows, lens, 2, 1, 128, 16, dtype, garbage=False)
        s["q"].fill_(0.25)
        s["k_cache"] = (torch.ones(s["k_cache"].shape) * 8).to(ref.F8).cuda()
        for b in range(2):
            for i, page in enumerate(s["page_table"][b].tolist()):
                s["k_scale"][page] = 0.015625 * (i + 1)
        run(s, windows, lens)


def test_pages_out_of_range_count_as_absent():
    windows, lens = [3, 2], [300, 40]
    s = make(25, windows, lens, 4, 2, 128, 16, BF16)
    s["page_table"][0, 1] = -1
    s["page_table"][0, 9:] = s["k_cache"].shape[0]
    s["page_table"][1, :] = 2 ** 31 - 1
    run(s, windows, lens)
    s.pop("k_new"), s.pop("v_new")
    got = run(s, windows, lens)
    assert (got["out"][3:] == 0).all() and torch.isneginf(got["lse"][3:]).all()


def test_lengths_are_clamped():
    s = make(26, [2, 2], [304, 304], 2, 1, 128, 16, BF16, garbage=False)
    s["seq_lens"] = torch.tensor([-5, 2 ** 31 - 1], dtype=torch.int32).cuda()
    check(tv.window_attention(**s, lse=True), wanted(s, [2, 2], [0, 304]), BF16, 128)


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("Hq", [8, 32])  # blocks of 32 rows, of 64
def test_masked_values_that_are_not_finite_do_not_matter(value, Hq):
    windows, lens = [6, 3], [140, 10]
    for dtype in (BF16, F16):
        s = make(27, windows, lens, Hq, 2, 128, 16, dtype, "tree")
        s["parents"] = torch.tensor([-1, 0, 1, 0, 3, 3, -1, 0, 1], dtype=torch.int32).cuda()
        clean = tv.window_attention(**s, lse=True)
        for n in ("k_new", "v_new"):
            s[n] = s[n].clone()
            s[n][3:6] = value
        got = tv.window_attention(**s, lse=True)
        for r in (0, 1, 2, 6, 7, 8):
            assert torch.equal(got["out"][r], clean["out"][r]) and torch.equal(got["lse"][r], clean["lse"][r])
        s["k_new"][3:6] = 0.5  # V alone: the rows that see it get it
        got = tv.window_attention(**s)["out"]
        for r in (3, 4, 5):
            bad = got[r].float()
            assert (torch.isnan(bad) if math.isnan(value) else bad == value).all()
        assert torch.isfinite(got[[0, 1, 2, 6, 7, 8]].float()).all()


def test_queries_of_zeros_and_extremes():
    windows, lens = [3, 1], [200, 33]
    for dtype in (BF16, F16):
        s = make(28, windows, lens, 4, 2, 128, 32, dtype)
        s["q"][1] = 0
        run(s, windows, lens)
        s["q"].zero_()
        run(s, windows, lens)
        # one row large, the others small: what a row may lose is 2^-17 of its block's largest
        s["q"].copy_(torch.randn(s["q"].shape, generator=torch.Generator().manual_seed(1)))
        s["q"][2] *= 200
        run(s, windows, lens, 0.001)


def test_parents_that_are_no_ancestors():
    for Hq in (4, 32):
        s = make(29, [5], [20], Hq, 2, 128, 16, BF16, "tree")
        s["parents"] = torch.tensor([3, 1, 7, -9, 2], dtype=torch.int32).cuda()
        run(s, [5], [20])


def test_windows_that_do_not_fit_are_left_alone():
    s = make(30, [4, 4, 4], [20, 300, 40], 4, 2, 128, 16, BF16)
    full = tv.window_attention(**s, lse=True)
    for indptr in ([0, 4, 2, 6], [4, 8, 8, 13], [-1, 4, 8, 12], [0, 0, 4, 8]):
        s["qo_indptr"] = torch.tensor(indptr, dtype=torch.int32).cuda()
        out = torch.full_like(full["out"], 7.0)
        tv.window_attention(**s, out=out)
        owned = torch.zeros(12, dtype=torch.bool)
        for a, b in zip(indptr[:-1], indptr[1:]):
            if 0 <= a < b <= 12:
                owned[a:b] = True
        assert (out.cpu()[~owned] == 7.0).all() and (out.cpu()[owned] != 7.0).any(-1).all()
    assert tv.device_error() == 0


def test_one_page_and_one_token():
    s = make(31, [1, 1], [1, 1], 1, 1, 128, 16, BF16)
    run(s, [1, 1], [1, 1])
    s = make(32, [1], [3], 1, 1, 128, 128, F16, garbage=False)
    for n in ("k_cache", "v_cache", "k_scale", "v_scale"):
        s[n] = s[n][:1].clone()
    s["page_table"].zero_()
    run(s, [1], [3])


def test_cache_of_more_than_4_gb():
    # the pages used lie behind 2^32 bytes, of K and of V
    pages, H, size = 2 ** 32 // (2 * 128 * 128) + 40, 2, 128
    s = make(33, [2, 1], [300, 17], 4, H, 128, size, BF16)
    small = {n: s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")}
    n = small["k_cache"].shape[0]
    for name in ("k", "v"):
        s[name + "_cache"] = torch.empty((pages, H, size, 128), dtype=torch.uint8, device="cuda")
        s[name + "_cache"][-n:] = small[name + "_cache"].view(torch.uint8)
        s[name + "_cache"] = s[name + "_cache"].view(ref.F8)
        s[name + "_scale"] = torch.full((pages, H), math.nan, device="cuda")
        s[name + "_scale"][-n:] = small[name + "_scale"]
    near = dict(s, **small)
    want = tv.window_attention(**near, lse=True)
    s["page_table"] = s["page_table"] + (pages - n)
    got = tv.window_attention(**s, lse=True)
    assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])
    cache = {k: s[k] for k in ("k_cache", "v_cache", "k_scale", "v_scale", "page_table", "seq_lens")}
    base = {k: near[k] for k in cache}
    ptr = torch.tensor([0, 300, 317], dtype=torch.int32).cuda()
    far, here = (tv.kv_read(**c, out_indptr=ptr, total_rows=317) for c in (cache, base))
    assert torch.equal(far["k"], here["k"]) and torch.equal(far["v"], here["v"])
    tv.kv_append(s["k_new"], s["v_new"], **cache, qo_indptr=s["qo_indptr"])
    tv.kv_append(s["k_new"], s["v_new"], **base, qo_indptr=s["qo_indptr"])
    for name in ("k", "v"):
        assert torch.equal(cache[name + "_cache"][-n:].view(torch.uint8), base[name + "_cache"].view(torch.uint8))


@pytest.mark.parametrize("D", [64, 128])
def test_another_stream_and_a_graph_with_everything(D):
    # a step captured once and replayed: attention, sampling of the tree and the append
    w = [4, 6]
    s = make(34, w, [40, 130], 4, 2, D, 16, BF16, "tree", garbage=False)
    s["page_table"] = torch.arange(40, dtype=torch.int32).view(2, 20).cuda()
    for n in ("k_cache", "v_cache"):
        s[n] = torch.zeros((40, 2, 16, D), dtype=torch.uint8, device="cuda").view(ref.F8)
    for n in ("k_scale", "v_scale"):
        s[n] = torch.ones((40, 2), device="cuda")
    g = torch.Generator().manual_seed(3)
    probs = torch.softmax(torch.randn((10, 1000), generator=g) * 2, -1).cuda()
    tokens = torch.randint(0, 1000, (10,), generator=g, dtype=torch.int32).cuda()
    coins = torch.rand(10, generator=g).cuda()
    cache = {k: s[k] for k in ("k_cache", "v_cache", "k_scale", "v_scale", "page_table", "seq_lens")}
    ws = tv.make_attention_workspace(2, 10, 4, 2, D)
    out = torch.empty_like(s["q"].contiguous())

    def step():
        tv.window_attention(**s, out=out, workspace=ws)
        r = tv.tree_spec_sampling(probs, 3, tokens, s["parents"], coins, qo_indptr=s["qo_indptr"], outputs=res)
        tv.kv_append(s["k_new"], s["v_new"], **cache, src_index=r["accept_index"], src_len=r["accept_length"])
        s["seq_lens"] += r["accept_length"]

    res = (torch.empty((2, 4), dtype=torch.int32).cuda(), torch.empty(2, dtype=torch.int32).cuda(),
           torch.empty((2, 4), dtype=torch.int32).cuda(), torch.empty((2, 4)).cuda())
    start = {k: v.clone() for k, v in cache.items()}

    def back():
        for k, v in start.items():
            cache[k].view(torch.uint8 if v.dtype == ref.F8 else v.dtype).copy_(
                v.view(torch.uint8) if v.dtype == ref.F8 else v)

    step(), step()
    torch.cuda.synchronize()
    want = [out.clone(), *(t.clone() for t in res), *(v.clone() for v in cache.values())]
    back()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    back()
    graph.replay(), graph.replay()
    torch.cuda.synchronize()
    for a, b in zip([out, *res, *cache.values()], want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("D,dtype", [(64, F16), (128, BF16)])
@pytest.mark.parametrize("kind", ["tree", "chain"])
def test_decoding_steps(D, dtype, kind):
    """Verify steps over the cache, as a server runs them: a prompt is appended; then, a few times,
    the window attends, its outputs make the distributions, a path is accepted, its K and V are
    appended. Each call is compared with the plain 64-bit form on the state that it got."""
    B, Dd, Hq, H, size, V = 3, 3, 4, 2, 16, 400
    T = 7 if kind == "tree" else Dd + 1
    prompt = [37, 0, 80]
    g = torch.Generator().manual_seed(41)
    rng = np.random.default_rng(41)
    pages, per = 40, 12
    table = torch.randperm(pages, generator=g)[: B * per].to(torch.int32).view(B, per)
    cache = dict(k_cache=torch.zeros((pages, H, size, D), dtype=torch.uint8).cuda().view(ref.F8),
                 v_cache=torch.zeros((pages, H, size, D), dtype=torch.uint8).cuda().view(ref.F8),
                 k_scale=torch.ones((pages, H)).cuda(), v_scale=torch.ones((pages, H)).cuda(),
                 page_table=table.cuda(), seq_lens=torch.zeros(B, dtype=torch.int32).cuda())
    lens = [0] * B
    head = torch.randn((Hq * D, V), generator=g).cuda() * 0.3

    def append_check(k, v, rows_of, **how):
        before = {n: t.clone() for n, t in cache.items()}
        tv.kv_append(k, v, **cache, **how)
        for name, x in (("k", k), ("v", v)):
            codes, scales = ref.append(before[name + "_cache"], before[name + "_scale"], x, table, lens, rows_of)
            assert torch.equal(cache[name + "_scale"].cpu().double(), scales)
            assert torch.equal(ref.codes64(cache[name + "_cache"]), codes)

    def draw(n):
        return torch.randn((n, Hq + 2 * H, D), generator=g).to(dtype).cuda()

    x = draw(sum(prompt))
    ptr = np.concatenate([[0], np.cumsum(prompt)]).astype(np.int32)
    append_check(x[:, Hq:Hq + H], x[:, Hq + H:], [range(a, b) for a, b in zip(ptr[:-1], ptr[1:])],
                 qo_indptr=torch.from_numpy(ptr).cuda())
    lens = list(prompt)
    cache["seq_lens"].copy_(torch.tensor(lens, dtype=torch.int32))
    moved = 0
    for step in range(4):
        x = draw(B * T)
        s = dict(cache, q=x[:, :Hq], k_new=x[:, Hq:Hq + H], v_new=x[:, Hq + H:])
        par = [[-1] + [int(rng.integers(0, i)) for i in range(1, T)] for _ in range(B)]
        if kind == "tree":
            s["parents"] = torch.tensor(par, dtype=torch.int32).flatten().cuda()
        got = tv.window_attention(**s, lse=True)
        check(got, wanted(s, [T] * B, lens), dtype, D)
        probs = torch.softmax(got["out"].flatten(1).float() @ head, -1)
        coins = torch.rand(B * T, generator=g).cuda()
        if kind == "tree":
            tokens = torch.zeros(B * T, dtype=torch.int32)
            for b in range(B):
                for i in range(1, T):  # likely tokens of the parent's distribution
                    tokens[b * T + i] = int(probs[b * T + par[b][i]].topk(4).indices[i % 4])
            r = tv.tree_spec_sampling(probs, Dd, tokens.view(B, T).cuda(), s["parents"].view(B, T), coins)
            windows = [(b * T, T) for b in range(B)]
            want = ref.tree(probs, tokens, s["parents"].cpu(), coins, windows, Dd)
            for name in ("accepted_tokens", "accept_length", "accept_index"):
                assert torch.equal(r[name].cpu(), torch.as_tensor(want[name]).to(torch.int32)), name
        else:
            drafts = probs.view(B, T, V)[:, :Dd].argmax(-1).to(torch.int32).contiguous()
            r = tv.chain_spec_sampling(probs, False, Dd, drafts,
                                       uniforms=torch.rand((B, 2 * Dd + 1), generator=g).cuda())
        n, idx = r["accept_length"].tolist(), r["accept_index"].tolist()
        assert all(1 <= a <= Dd + 1 for a in n)
        append_check(s["k_new"], s["v_new"], [i[:a] for i, a in zip(idx, n)], src_index=r["accept_index"],
                     src_len=r["accept_length"])
        cache["seq_lens"] += r["accept_length"]
        lens = [a + b for a, b in zip(lens, n)]
        moved += sum(n)
        assert cache["seq_lens"].tolist() == lens
    ptr = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    read = tv.kv_read(**cache, out_indptr=torch.from_numpy(ptr).cuda(), total_rows=int(ptr[-1]), dtype=torch.float32)
    for name, got in read.items():
        for b in range(B):
            want, _ = ref.cached(cache[name + "_cache"], cache[name + "_scale"], table, b, lens[b])
            assert torch.equal(got[ptr[b]:ptr[b + 1]].cpu().double(), want)
    assert moved >= 4 * B and tv.device_error() == 0
