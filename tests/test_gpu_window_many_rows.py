"""GPU: window attention of more than 32 rows of a KV head with head_dim 64, whose blocks of rows are
chosen on the device by the cached tokens; and page tables wider than the contexts, which change
nothing."""
import pytest
import torch

from speculative_decoding_verify_temp_gb300 import tsverify as tv
from tests import window_ref as ref
from tests.test_gpu_window import _built, check, make  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("windows,lens,Hq,H", [([1, 3], [30, 5], 4, 2), ([5, 6], [40, 300], 8, 2), ([12, 9], [300, 64], 8, 2),
                                               ([17, 65], [63, 129], 2, 1)])
def test_a_wider_page_table_changes_nothing(D, windows, lens, Hq, H):
    for dtype in (BF16, F16):
        s = make(71, windows, lens, Hq, H, D, 16, dtype)
        want = tv.window_attention(**s, lse=True)
        s["page_table"] = torch.cat([s["page_table"], torch.full((2, 32768), -1, dtype=torch.int32).cuda()], 1)
        got = tv.window_attention(**s, lse=True)
        assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])


def exact(s, windows, lens):
    """window_ref.attention's results, on the GPU, for chains."""
    q, (pages, H, size, D) = s["q"].double(), s["k_cache"].shape
    Hq = q.shape[1]
    scale = D ** -0.5
    out, absv = torch.zeros((2, *q.shape), dtype=torch.float64, device="cuda")
    lse, big, count, floor = torch.zeros((4, *q.shape[:2]), dtype=torch.float64, device="cuda")
    r0 = 0
    for b, (t, n) in enumerate(zip(windows, lens)):
        ids = s["page_table"][b, :-(-n // size)].long()
        rows = slice(r0, r0 + t)
        kv = []
        for name in ("k", "v"):
            x = s[name + "_cache"].view(torch.uint8)[ids].view(ref.F8).double() * s[name + "_scale"][ids][:, :, None, None].double()
            x = x.permute(1, 0, 2, 3).reshape(H, -1, D)[:, :n]
            kv.append(torch.cat([x, s[name + "_new"][rows].double().transpose(0, 1)], 1))
        seen = torch.ones((t, n + t), dtype=torch.bool, device="cuda")
        seen[:, n:] = ref.sees(t).cuda()
        for h in range(Hq):
            k, v = kv[0][h // (Hq // H)], kv[1][h // (Hq // H)]
            x = (q[rows, h] @ k.T * scale).masked_fill(~seen, -torch.inf)
            p = torch.softmax(x, -1)
            out[rows, h], absv[rows, h], lse[rows, h] = p @ v, p @ v.abs(), torch.logsumexp(x, -1)
            big[rows, h] = (q[rows, h].abs() @ k.abs().T).amax(-1) * scale
            count[rows, h] = seen.sum(-1).double()
            heads = q[rows, h // (Hq // H) * (Hq // H):(h // (Hq // H) + 1) * (Hq // H)].abs().max()
            floor[rows, h] = heads * k.abs().sum(1).max() * scale
        r0 += t
    return [x.cpu() for x in (out, lse, absv, big, count, floor)]


@pytest.mark.parametrize("windows,lens,Hq,H,dtype", [
    ([16, 5], [60000, 41111], 32, 8, BF16),           # pieces of units, joined
    ([65, 33, 40], [20011, 19000, 30003], 10, 2, F16),
    ([16] * 24, [9000 + 37 * i for i in range(24)], 8, 2, BF16),
    ([12, 40], [3000, 2000], 8, 2, F16),              # few tokens: blocks of 32 rows
])
def test_many_rows_over_long_contexts(windows, lens, Hq, H, dtype):
    s = make(72, windows, lens, Hq, H, 64, 64, dtype, garbage=False)
    check(tv.window_attention(**s, lse=True), exact(s, windows, lens), dtype, 64)
