"""GPU: appending to the 8-bit cache and reading it back, exactly as defined."""
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


def make(seed, lens, room, H, D, size, layout="pages"):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    per = -(-max(n + r for n, r in zip(lens, room)) // size)
    pages = B * per + 2
    c = {"page_table": torch.randperm(pages, generator=g)[: B * per].to(torch.int32).view(B, per).cuda()}
    for n in ("k", "v"):
        x = (torch.randn((pages, H, size, D), generator=g) * 70).clamp(-448, 448).to(ref.F8).view(torch.uint8)
        x = x.transpose(1, 2).contiguous().cuda().transpose(1, 2) if layout == "tokens" else x.cuda()
        c[n + "_cache"] = x if layout == "tokens" else x.view(ref.F8)
        c[n + "_scale"] = torch.exp2(torch.randint(-8, -3, (pages, H), generator=g).float()).cuda()
    c["seq_lens"] = torch.tensor(lens, dtype=torch.int32).cuda()
    return c


def rows(seed, n, H, D, dtype, spread=6):
    g = torch.Generator().manual_seed(seed + 1000)
    x = torch.randn((n, 2 * H, D), generator=g) * torch.exp2(torch.randint(-spread, spread, (n, 2 * H, 1), generator=g).float())
    x = x.to(dtype).cuda()
    return x[:, :H], x[:, H:]


def compare(c, before, k, v, lens, rows_of):
    for name, x in (("k", k), ("v", v)):
        codes, scales = ref.append(before[name + "_cache"], before[name + "_scale"], x, before["page_table"].cpu(),
                                   lens, rows_of)
        torch.testing.assert_close(c[name + "_scale"].cpu().double(), scales, rtol=0, atol=0)
        torch.testing.assert_close(ref.codes64(c[name + "_cache"]), codes, rtol=0, atol=0, equal_nan=True)


def copy(c):
    return {n: t.clone() for n, t in c.items()}


CASES = [
    # lens, rows of each request, H, D, page, dtype, layout
    ([0], [1], 1, 64, 16, torch.bfloat16, "pages"),
    ([5, 16, 31, 32], [3, 1, 2, 5], 2, 128, 16, torch.bfloat16, "pages"),
    ([0, 7, 100], [65, 1, 30], 3, 64, 32, torch.float16, "tokens"),
    ([13, 0], [200, 131], 2, 128, 64, torch.float32, "pages"),
    ([127, 128, 1], [2, 1, 300], 1, 128, 128, torch.bfloat16, "tokens"),
    ([9], [700], 2, 64, 16, torch.float16, "pages"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{max(c[0])}_{max(c[1])}_{c[4]}_{c[6]}")
def test_append_packed(case):
    lens, n, H, D, size, dtype, layout = case
    c = make(1, lens, n, H, D, size, layout)
    before = copy(c)
    k, v = rows(1, sum(n), H, D, dtype)
    ptr = np.concatenate([[0], np.cumsum(n)])
    tv.kv_append(k, v, **c, qo_indptr=torch.tensor(ptr, dtype=torch.int32).cuda())
    compare(c, before, k, v, lens, [list(range(a, b)) for a, b in zip(ptr[:-1], ptr[1:])])
    assert torch.equal(c["seq_lens"], before["seq_lens"])


@pytest.mark.parametrize("size", [16, 64])
def test_append_accepted_rows(size):
    lens, R = [15, 40, 0, 3, 63], 6
    c = make(2, lens, [R] * 5, 2, 64, size)
    before = copy(c)
    k, v = rows(2, 30, 2, 64, torch.bfloat16)
    idx = torch.full((5, R), -1, dtype=torch.int32)
    n = [6, 1, 3, 0, 4]
    r = np.random.default_rng(3)
    for b in range(5):
        idx[b, :n[b]] = torch.tensor(b * R + np.sort(r.permutation(R)[: n[b]]), dtype=torch.int32)
    tv.kv_append(k, v, **c, src_index=idx.cuda(), src_len=torch.tensor(n, dtype=torch.int32).cuda())
    compare(c, before, k, v, lens, [idx[b, :n[b]].tolist() for b in range(5)])


def test_append_equal_windows_and_the_same_row_twice():
    c = make(4, [3, 20], [4, 4], 2, 64, 16)
    before = copy(c)
    k, v = rows(4, 8, 2, 64, torch.bfloat16)
    tv.kv_append(k, v, **c)
    compare(c, before, k, v, [3, 20], [range(4), range(4, 8)])
    c = copy(before)
    idx = torch.tensor([[2, 2, 2, 5], [2, 0, 0, 2]], dtype=torch.int32).cuda()
    tv.kv_append(k, v, **c, src_index=idx, src_len=torch.tensor([4, 4], dtype=torch.int32).cuda())
    compare(c, before, k, v, [3, 20], idx.tolist())


def test_append_leaves_what_does_not_fit():
    c = make(5, [30, 10, 40, 5], [4] * 4, 2, 64, 16)
    c["page_table"] = c["page_table"][:, :3].contiguous()  # room for 48 tokens
    c["page_table"][1, 0] = -1
    c["page_table"][3, 0] = c["k_cache"].shape[0]
    c["seq_lens"] = torch.tensor([47, 10, -3, 5], dtype=torch.int32).cuda()
    before = copy(c)
    k, v = rows(5, 16, 2, 64, torch.bfloat16)
    idx = torch.tensor([[0, 1, 2, 3], [4, 5, 6, 7], [8, -1, 16, 9], [10, 11, 12, 13]], dtype=torch.int32).cuda()
    tv.kv_append(k, v, **c, src_index=idx, src_len=torch.tensor([9, 4, 4, 4], dtype=torch.int32).cuda())
    compare(c, before, k, v, [47, 10, 0, 5], [[0, 1, 2, 3], [4, 5, 6, 7], [8, None, None, 9], [10, 11, 12, 13]])
    # no row to store: the block keeps its scale
    c = copy(before)
    idx = torch.full((4, 4), 99, dtype=torch.int32).cuda()
    tv.kv_append(k, v, **c, src_index=idx, src_len=torch.tensor([4, 0, -2, 4], dtype=torch.int32).cuda())
    for n in c:
        assert torch.equal(c[n].view(torch.uint8), before[n].view(torch.uint8))
    # pairs of an indptr that do not fit
    ptr = torch.tensor([0, 4, 2, 20, 16], dtype=torch.int32).cuda()
    tv.kv_append(k, v, **c, qo_indptr=ptr)
    compare(c, before, k, v, [47, 10, 0, 5], [range(4), [], [], []])


def test_append_values_at_the_borders():
    # the largest magnitude exactly 448 2^e, one step above, zero, subnormal, huge; not finite
    H, D, size = 1, 64, 16
    tops = [448.0, 449.0, 447.0, 896.0, 0.0, 2.0 ** -130, 3e38, 2.0 ** 68, 448 * 2.0 ** -60, 1.0]
    c = make(6, [0] * len(tops), [2] * len(tops), H, D, size)
    before = copy(c)
    g = torch.Generator().manual_seed(1)
    x = (torch.rand((2 * len(tops), H, D), generator=g) * 2 - 1)
    for i, t in enumerate(tops):
        x[2 * i:2 * i + 2] *= t
        x[2 * i, 0, 5] = t
    x[18, 0, 7], x[18, 0, 9], x[19, 0, 3] = math.inf, -math.inf, math.nan
    x = x.cuda()
    tv.kv_append(x, -x, **c)
    compare(c, before, x, -x, [0] * len(tops), [range(2 * i, 2 * i + 2) for i in range(len(tops))])
    assert c["k_scale"][c["page_table"][0, 0], 0] == 1.0 and c["k_scale"][c["page_table"][1, 0], 0] == 2.0


def test_append_token_by_token_grows_the_scale():
    # one token a call with growing magnitudes: every call rounds the block's codes again
    c = make(7, [0, 3], [40, 40], 2, 64, 16)
    lens = [0, 3]
    for t in range(20):
        before = copy(c)
        k, v = rows(100 + t, 2, 2, 64, torch.bfloat16, spread=1)
        k, v = k * 2.0 ** (t - 10), v * 2.0 ** (5 - t)
        tv.kv_append(k, v, **c)
        compare(c, before, k, v, lens, [[0], [1]])
        lens = [n + 1 for n in lens]
        c["seq_lens"] += 1


def test_append_keeps_a_callers_scale():
    # a scale that is no power of two, large enough to stay, and one that has to grow
    c = make(8, [4, 4], [3, 3], 1, 64, 16)
    c["k_scale"].fill_(0.3)
    c["v_scale"].fill_(1e-5)
    before = copy(c)
    k, v = rows(8, 6, 1, 64, torch.float32, spread=1)
    tv.kv_append(k, v, **c)
    held = before["page_table"][:, 0].long()
    assert (c["k_scale"][held] == 0.3).all() and (c["v_scale"][held] > 2e-5).all()
    for name, x in (("k", k), ("v", v)):
        # the fp32 quotient is rounded before the code is: one e4m3 step where that crosses a tie
        codes, scales = ref.append(before[name + "_cache"], before[name + "_scale"], x, before["page_table"].cpu(),
                                   [4, 4], [range(3), range(3, 6)])
        got = ref.codes64(c[name + "_cache"])
        assert torch.equal(c[name + "_scale"].cpu().double(), scales)
        assert ((got - codes).abs() <= torch.maximum(codes.abs() / 8, torch.tensor(2.0 ** -9, dtype=torch.float64))).all()
        assert (got != codes).double().mean() < 0.01


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("layout,H,D,size", [("pages", 1, 64, 16), ("tokens", 3, 128, 32), ("pages", 8, 128, 128)])
def test_read(dtype, layout, H, D, size):
    lens = [1, 0, 77, 16, 130]
    c = make(9, lens, [0] * 5, H, D, size, layout)
    c["k_scale"].copy_(torch.rand(c["k_scale"].shape) + 0.1)
    ptr = np.concatenate([[0], np.cumsum(lens)])
    total = int(ptr[-1]) + 3
    out = tuple(torch.full((total, H, D), 5.0, dtype=dtype, device="cuda") for _ in range(2))
    got = tv.kv_read(**c, out_indptr=torch.tensor(ptr, dtype=torch.int32).cuda(), total_rows=total, out=out)
    for name in ("k", "v"):
        want = torch.full((total, H, D), 5.0, dtype=dtype)
        for b, n in enumerate(lens):
            x, _ = ref.cached(c[name + "_cache"], c[name + "_scale"], c["page_table"].cpu(), b, n)
            want[ptr[b]:ptr[b + 1]] = x.float().to(dtype)  # the product is rounded to fp32 first
        assert torch.equal(got[name].cpu(), want)


def test_read_from_the_middle_and_what_is_absent():
    lens = [50, 20, 33]
    c = make(10, lens, [0] * 3, 2, 64, 16)
    c["page_table"][0, 1] = -7
    start = torch.tensor([10, -2, 30], dtype=torch.int32).cuda()
    ptr = [2, 40, 45, 60]
    got = tv.kv_read(**c, out_indptr=torch.tensor(ptr, dtype=torch.int32).cuda(), total_rows=60, start=start,
                     dtype=torch.float32)
    for name in ("k", "v"):
        for b in range(3):
            x, there = ref.cached(c[name + "_cache"], c[name + "_scale"], c["page_table"].cpu(), b, lens[b])
            for i in range(ptr[b + 1] - ptr[b]):
                pos = int(start[b]) + i
                want = x[pos] if 0 <= pos < lens[b] and there[pos] else torch.zeros((2, 64))
                assert torch.equal(got[name][ptr[b] + i].cpu().double(), want.double())
    # a pair that does not fit is skipped
    out = tuple(torch.full((45, 2, 64), 5.0, device="cuda") for _ in range(2))
    tv.kv_read(**c, out_indptr=torch.tensor(ptr, dtype=torch.int32).cuda(), total_rows=45, start=start, out=out)
    assert (out[0][:2] == 5.0).all() and torch.equal(out[0][2:45], got["k"][2:45])


def test_append_then_read_in_a_graph_on_a_side_stream():
    c = make(11, [5, 30], [3, 3], 2, 128, 16)
    k, v = rows(11, 6, 2, 128, torch.bfloat16)
    eager = copy(c)
    tv.kv_append(k, v, **eager)
    ptr = torch.tensor([0, 8, 41], dtype=torch.int32).cuda()
    after = dict(eager, seq_lens=eager["seq_lens"] + 3)
    want = tv.kv_read(**after, out_indptr=ptr, total_rows=41)
    out = tuple(torch.empty((41, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    longer = c["seq_lens"] + 3
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        tv.kv_append(k, v, **c)
        tv.kv_read(**dict(c, seq_lens=longer), out_indptr=ptr, total_rows=41, out=out)
    for _ in range(2):  # the second replay appends the same rows to the same places
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want["k"]) and torch.equal(out[1], want["v"])
    side = copy(eager)
    tv.kv_append(k, v, **side, stream=stream)
    stream.synchronize()
    assert torch.equal(side["k_cache"].view(torch.uint8), eager["k_cache"].view(torch.uint8))
