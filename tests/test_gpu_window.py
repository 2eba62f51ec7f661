"""GPU: attention of windows over the 8-bit cache against the plain 64-bit implementation, with
bounds formed from the kernel's roundings (tests/window_ref.py)."""
import math

import numpy as np
import pytest
import torch

from speculative_decoding_verify_temp_gb300 import tsverify as tv
from tests import window_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()


def make(seed, windows, lens, Hq, H, D, size, dtype, mask="chain", layout="pages", vscale=(-8, -4),
         garbage=True):
    """Tensors of a call on the GPU; unseen slots hold NaN codes, unseen pages NaN scales."""
    g = torch.Generator().manual_seed(seed)
    B, rows = len(windows), sum(windows)
    per = max(1, max((n + size - 1) // size for n in lens))
    pages = B * per + 2
    table = torch.randperm(pages, generator=g)[: B * per].to(torch.int32).view(B, per)
    s = {}
    used = torch.zeros((pages, size), dtype=torch.bool)
    for b, n in enumerate(lens):
        for i in range(n):
            used[table[b, i // size], i % size] = True
    both = torch.zeros((pages, 2, H, size, D), dtype=torch.uint8)
    for w, name in enumerate(("k", "v")):
        x = (torch.randn((pages, H, size, D), generator=g) * 70).clamp(-448, 448).to(ref.F8).view(torch.uint8)
        if garbage:
            x[~used[:, None, :, None].expand_as(x)] = 0x7F
        sc = torch.exp2(torch.randint(*vscale, (pages, H), generator=g).float())
        if garbage:
            sc[~used.any(1)] = math.nan
        s[name + "_scale"] = sc.cuda()
        if layout == "tokens":  # [pages, size, H, D] in memory
            s[name + "_cache"] = x.transpose(1, 2).contiguous().cuda().transpose(1, 2)
        elif layout == "pool":  # K and V of a page side by side
            both[:, w] = x
        else:
            s[name + "_cache"] = x.cuda().view(ref.F8)
    if layout == "pool":
        both = both.cuda()
        s["k_cache"], s["v_cache"] = both[:, 0], both[:, 1]
    s["page_table"] = table.cuda()
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32).cuda()
    qkv = torch.randn((rows, Hq + 2 * H, D), generator=g)
    qkv[:, :Hq] *= 1.7
    qkv = qkv.to(dtype).cuda()
    s["q"] = qkv[:, :Hq] if layout != "pages" else qkv[:, :Hq].contiguous()
    if mask != "none":
        s["k_new"], s["v_new"] = qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
    if mask == "tree":
        r = np.random.default_rng(seed)
        s["parents"] = torch.tensor([-1 if i == 0 else int(r.integers(0, i)) for t in windows for i in range(t)],
                                    dtype=torch.int32).cuda()
    s["qo_indptr"] = torch.tensor(np.concatenate([[0], np.cumsum(windows)]), dtype=torch.int32).cuda()
    return s


def wanted(s, windows, lens, sm_scale=None):
    first = np.concatenate([[0], np.cumsum(windows)])[:-1]
    return ref.attention(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["page_table"], lens,
                         list(zip(first.tolist(), windows)), s.get("k_new"), s.get("v_new"), s.get("parents"),
                         sm_scale)


def two_parts(s):
    """Whether a call's probabilities go into the product in two parts (see attention_bounds)."""
    rows, Hq, D = s["q"].shape
    mean = -(-rows * (Hq // s["k_cache"].shape[1]) // s["page_table"].shape[0])
    return s["q"].dtype == torch.bfloat16 and D == 128 and mean > 32


def check(got, want, dtype, D, two=False):
    out, lse = want[0], want[1]
    b, z = ref.attention_bounds(*want, dtype, D, two)
    o, l = got["out"].cpu().double(), got["lse"].cpu().double()
    assert torch.equal(torch.isneginf(l), torch.isneginf(lse))
    fine = torch.isfinite(lse)
    assert (l - lse)[fine].abs().le(z[fine]).all(), (l - lse)[fine].abs().max()
    far = (o - out).abs() - b
    assert far.max() <= 0, (far.max(), (o - out).abs().max())


CASES = [
    # windows, lens, Hq, H, D, page, dtype, mask, layout
    ([1], [37], 8, 2, 64, 16, torch.bfloat16, "chain", "pages"),
    ([1], [0], 4, 4, 128, 16, torch.bfloat16, "chain", "pages"),
    ([1, 1, 1], [1, 16, 17], 2, 1, 128, 16, torch.float16, "chain", "pages"),
    ([5, 3, 1, 4], [63, 64, 65, 127], 8, 2, 128, 32, torch.bfloat16, "chain", "pages"),
    ([4, 4], [200, 31], 10, 2, 64, 64, torch.float16, "chain", "tokens"),
    ([8, 8], [300, 129], 8, 1, 128, 128, torch.bfloat16, "tree", "pool"),
    ([65, 64, 2], [100, 5, 0], 4, 2, 64, 16, torch.bfloat16, "chain", "pages"),
    ([65, 33], [40, 257], 2, 2, 128, 16, torch.float16, "tree", "tokens"),
    ([7, 2], [90, 15], 3, 3, 128, 32, torch.bfloat16, "none", "pages"),
    ([3, 5], [0, 20], 8, 1, 64, 16, torch.float16, "none", "pool"),
    ([13], [700], 14, 2, 128, 16, torch.bfloat16, "tree", "pages"),
    ([2] * 40, [(i * 37) % 150 for i in range(40)], 16, 1, 64, 16, torch.bfloat16, "chain", "pages"),
    ([6], [20011], 4, 1, 64, 32, torch.bfloat16, "chain", "pages"),      # many pieces of a unit
    ([3, 1], [9001, 30], 16, 1, 128, 64, torch.float16, "chain", "pages"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[2]}x{c[3]}x{c[4]}_{max(c[0])}_{max(c[1])}_{c[7]}")
def test_attention(case):
    windows, lens, Hq, H, D, size, dtype, mask, layout = case
    s = make(11, windows, lens, Hq, H, D, size, dtype, mask, layout)
    got = tv.window_attention(**s, lse=True)
    check(got, wanted(s, windows, lens), dtype, D, two_parts(s))
    again = tv.window_attention(**s, lse=True)
    assert torch.equal(got["out"], again["out"]) and torch.equal(got["lse"], again["lse"])


@pytest.mark.parametrize("windows,lens,Hq,H,size,dtype,mask,layout", [
    ([12, 9, 20], [300, 64, 0], 8, 2, 16, torch.bfloat16, "chain", "pages"),
    ([65, 20], [200, 5000], 4, 2, 64, torch.float16, "tree", "tokens"),
    ([17, 33, 40], [63, 65, 129], 2, 1, 128, torch.bfloat16, "none", "pool"),
])
def test_blocks_of_64_rows(windows, lens, Hq, H, size, dtype, mask, layout):
    # many rows a KV head and room in the page tables for more than 2^19 tokens: wider blocks
    s = make(31, windows, lens, Hq, H, 64, size, dtype, mask, layout)
    room = 2 ** 19 // (size * H * len(windows)) + 1
    s["page_table"] = torch.cat([s["page_table"], torch.full((len(windows), room), -1, dtype=torch.int32).cuda()], 1)
    got = tv.window_attention(**s, lse=True)
    check(got, wanted(s, windows, lens), dtype, 64)


def test_equal_windows_need_no_indptr():
    s = make(3, [4, 4, 4], [50, 0, 333], 8, 2, 128, 16, torch.bfloat16)
    a = tv.window_attention(**s)["out"]
    s.pop("qo_indptr")
    assert torch.equal(a, tv.window_attention(**s)["out"])


def test_scale_and_large_scores():
    # scores of several hundred: the softmax is nearly one-hot
    windows, lens = [4, 2], [200, 77]
    s = make(5, windows, lens, 4, 2, 64, 16, torch.bfloat16, vscale=(-3, 3))
    for scale in (1.0, 0.0, -0.3):
        check(tv.window_attention(**s, sm_scale=scale, lse=True), wanted(s, windows, lens, scale), torch.bfloat16, 64)


def test_scales_far_apart():
    # block scales between 2^-59 and 2^8, for K small where V is large: no product may lose the
    # small ones to the large
    windows, lens = [3], [150]
    s = make(6, windows, lens, 2, 1, 64, 16, torch.bfloat16, vscale=(-59, 9), garbage=False)
    s["k_scale"].fill_(2.0 ** -7)
    check(tv.window_attention(**s, lse=True), wanted(s, windows, lens), torch.bfloat16, 64)


def test_arbitrary_scales():
    windows, lens = [4], [120]
    s = make(8, windows, lens, 4, 2, 128, 32, torch.float16, garbage=False)
    for n in ("k_scale", "v_scale"):
        s[n] = torch.rand(s[n].shape, generator=torch.Generator().manual_seed(1)).cuda() * 0.02 + 0.001
    # log2 of the scale and its reciprocal: 2^-21 of the probability more, inside the bounds
    check(tv.window_attention(**s, lse=True), wanted(s, windows, lens), torch.float16, 128)


def test_pages_out_of_range_count_as_absent():
    windows, lens = [3, 2], [100, 40]
    s = make(9, windows, lens, 4, 2, 64, 16, torch.bfloat16)
    s["page_table"][0, 1] = -1
    s["page_table"][0, 3] = s["k_cache"].shape[0]
    s["page_table"][1, :] = 2 ** 31 - 1
    check(tv.window_attention(**s, lse=True), wanted(s, windows, lens), torch.bfloat16, 64)
    s.pop("k_new"), s.pop("v_new")
    got = tv.window_attention(**s, lse=True)
    check(got, wanted(s, windows, lens), torch.bfloat16, 64)
    assert (got["out"][3:] == 0).all() and torch.isneginf(got["lse"][3:]).all()


def test_lengths_are_clamped():
    windows = [2, 2]
    s = make(10, windows, [48, 48], 2, 1, 64, 16, torch.bfloat16, garbage=False)
    s["seq_lens"] = torch.tensor([-5, 2 ** 31 - 1], dtype=torch.int32).cuda()
    check(tv.window_attention(**s, lse=True), wanted(s, windows, [0, 48]), torch.bfloat16, 64)


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_masked_values_that_are_not_finite_do_not_matter(value, dtype):
    # a tree of two branches; the tokens of the second hold the value in K and V
    windows, lens = [6, 3], [30, 10]
    s = make(12, windows, lens, 8, 2, 64, 16, dtype, "tree")
    s["parents"] = torch.tensor([-1, 0, 1, 0, 3, 3, -1, 0, 1], dtype=torch.int32).cuda()
    clean = tv.window_attention(**s, lse=True)
    for n in ("k_new", "v_new"):
        s[n] = s[n].clone()
        s[n][3:6] = value
    got = tv.window_attention(**s, lse=True)
    for r in (0, 1, 2, 6, 7, 8):
        assert torch.equal(got["out"][r], clean["out"][r]) and torch.equal(got["lse"][r], clean["lse"][r])
    # V alone: the rows that see it get it
    s["k_new"][3:6] = 0.5
    got = tv.window_attention(**s)["out"]
    for r in (3, 4, 5):
        bad = got[r].float()
        assert (torch.isnan(bad) if math.isnan(value) else bad == value).all()
    assert torch.isfinite(got[[0, 1, 2, 6, 7, 8]].float()).all()


def test_parents_that_are_no_ancestors():
    windows, lens = [5], [20]
    s = make(13, windows, lens, 4, 2, 64, 16, torch.bfloat16, "tree")
    s["parents"] = torch.tensor([3, 1, 7, -9, 2], dtype=torch.int32).cuda()
    check(tv.window_attention(**s, lse=True), wanted(s, windows, lens), torch.bfloat16, 64)


def test_windows_that_do_not_fit_are_left_alone():
    s = make(14, [4, 4, 4], [20, 30, 40], 4, 2, 64, 16, torch.bfloat16)
    full = tv.window_attention(**s, lse=True)
    for indptr, live in (([0, 4, 2, 6], [(0, 4)]), ([4, 8, 8, 13], [(4, 8)]), ([-1, 4, 8, 12], None),
                         ([0, 0, 4, 8], None)):
        s["qo_indptr"] = torch.tensor(indptr, dtype=torch.int32).cuda()
        out = torch.full_like(full["out"], 7.0)
        tv.window_attention(**s, out=out)
        owned = torch.zeros(12, dtype=torch.bool)
        for a, b in zip(indptr[:-1], indptr[1:]):
            if 0 <= a < b <= 12:
                owned[a:b] = True
        assert (out.cpu()[~owned] == 7.0).all() and (out.cpu()[owned] != 7.0).any(-1).all()
    # a window of 66 rows
    s = make(15, [65, 2], [20, 30], 2, 1, 64, 16, torch.bfloat16)
    s["qo_indptr"] = torch.tensor([0, 66, 67], dtype=torch.int32).cuda()
    out = torch.full_like(s["q"].contiguous(), 7.0)
    tv.window_attention(**s, out=out)
    assert (out[:66] == 7.0).all() and (out[66] != 7.0).any()


def test_graph_streams_and_two_calls_at_once():
    a = make(16, [5, 2], [700, 90], 8, 2, 128, 16, torch.bfloat16)
    b = make(17, [3, 9], [11, 1500], 8, 2, 128, 32, torch.bfloat16)
    want = [tv.window_attention(**x, lse=True) for x in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    ws = [tv.make_attention_workspace(2, n, 8, 2, 128) for n in (7, 12)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, x in enumerate((a, b)):
            got[i].append(tv.window_attention(**x, lse=True, workspace=ws[i], stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert torch.equal(r["out"], want[i]["out"]) and torch.equal(r["lse"], want[i]["lse"])
    # captured; replayed after the inputs changed in place
    out = torch.empty_like(want[0]["out"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tv.window_attention(**a, out=out, workspace=ws[0])
    a["seq_lens"][0] = 123
    a["q"].mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, tv.window_attention(**a)["out"])
