"""GPU: verification of drafted trees against the plain 64-bit walk; the same tokens as the chain
call where the tree is a chain; the emitted token has the target's distribution."""
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


def coins(r, shape):
    return ((2 * r.integers(0, 1 << 23, shape) + 1) * 2.0 ** -24).astype(np.float32)


def make(seed, sizes, V, ld=None, sharp=3.0, width=3):
    r = np.random.default_rng(seed)
    n = sum(sizes)
    x = r.standard_normal((n, V)) * sharp
    p = np.exp(x - x.max(1, keepdims=True))
    p = (p / p.sum(1, keepdims=True)).astype(np.float32)
    full = np.zeros((n, ld or V), np.float32)
    full[:, :V] = p
    parents, tokens = [], []
    for t in sizes:
        base = len(parents)
        count = np.zeros(t, int)
        for i in range(t):
            up = -1
            if i:
                open_ = np.nonzero(count[:i] < width)[0]
                up = int(open_[max(0, len(open_) - 1 - r.integers(0, 3))])
            top = np.argsort(-p[base + max(up, 0)])[: 8]
            tokens.append(int(top[min(count[up] if i else 0, len(top) - 1)]) if r.random() < 0.8 else int(r.integers(0, V)))
            if i:
                count[up] += 1
            parents.append(up)
    ptr = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    cu = lambda a, t=torch.int32: torch.tensor(np.asarray(a), dtype=t).cuda()  # noqa: E731
    return dict(target_probs=torch.from_numpy(full).cuda()[:, :V], tokens=cu(tokens), parents=cu(parents),
                uniforms=torch.from_numpy(coins(r, n)).cuda(), qo_indptr=cu(ptr)), list(zip(ptr[:-1].tolist(), sizes))


def check(s, windows, D):
    got = tv.tree_spec_sampling(D=D, **s)
    want = ref.tree(s["target_probs"], s["tokens"], s["parents"], s["uniforms"], windows, D)
    for n in ("accept_length", "accepted_tokens", "accept_index"):
        np.testing.assert_array_equal(got[n].cpu().numpy(), want[n], err_msg=n)
    # ln of an fp32 value: logf's error of one step on the result, and its rounding
    np.testing.assert_allclose(got["logprobs"].cpu().numpy(), want["logprobs"], rtol=2 * 2.0 ** -23, atol=2.0 ** -24)
    return want


@pytest.mark.parametrize("sizes,V,ld", [
    ([8] * 4, 1024, None), ([1], 1, None), ([1, 2, 65], 7, None), ([5, 3, 1, 9], 101, None),
    ([6] * 3, 1000, 1003), ([32] * 5, 32000, None), ([13, 64], 50257, 50260), ([4] * 2, 201088, None),
    ([7] * 700, 300, None), ([20], 151936, None), ([3], 1 << 20, None),
])
def test_tree(sizes, V, ld):
    s, windows = make(sum(sizes) + V, sizes, V, ld)
    check(s, windows, max(sizes) - 1)


@pytest.mark.parametrize("V", [1024, 32000])
def test_long_paths(V):
    s, windows = make(V, [24] * 12, V, sharp=12.0)
    assert check(s, windows, 23)["accept_length"].max() > 4


def test_equal_trees_need_no_indptr():
    s, windows = make(2, [6] * 5, 500)
    a = tv.tree_spec_sampling(D=5, **s)
    s.pop("qo_indptr")
    s["tokens"], s["parents"] = s["tokens"].view(5, 6), s["parents"].view(5, 6)
    b = tv.tree_spec_sampling(D=5, **s, logprobs=False, accept_index=False)
    assert torch.equal(a["accepted_tokens"], b["accepted_tokens"]) and b["accept_index"] is None


@pytest.mark.parametrize("D", [0, 1, 2])
def test_depth_limit(D):
    s, windows = make(3, [12] * 30, 200, sharp=6.0)
    want = check(s, windows, D)
    assert want["accept_length"].max() == D + 1


def test_a_chain_gives_the_chain_calls_tokens():
    B, D, V = 64, 5, 1000
    r = np.random.default_rng(4)
    s, windows = make(4, [D + 1] * B, V, width=1, sharp=6.0)
    s["parents"] = torch.arange(-1, D, dtype=torch.int32).repeat(B).cuda()
    check(s, windows, D)
    tree = tv.tree_spec_sampling(D=D, **s)
    u = s["uniforms"].view(B, D + 1)
    chain = tv.chain_spec_sampling(s["target_probs"].contiguous(), False, D, s["tokens"].view(B, D + 1)[:, 1:].contiguous(),
                                   uniforms=torch.cat([u[:, 1:], u[:, :1]], 1).contiguous())
    # the chain call sums its draws in fp32: requests whose last coin lies near an edge may differ
    same = (tree["accepted_tokens"] == chain["accepted_tokens"]).all(1)
    assert same.float().mean() > 0.95
    assert torch.equal(tree["accept_length"], chain["accept_length"])
    assert torch.equal(tree["accept_index"], chain["accept_index"])
    assert tree["accept_length"].float().mean() > 1.5


def test_siblings_with_one_token_and_tokens_outside():
    # p = (1/2, 1/4, 1/4): all sums are exact
    p = torch.tensor([[0.5, 0.25, 0.25, 0.0]] * 6).cuda()
    parents = torch.tensor([[-1, 0, 0, 0, 0, 0]], dtype=torch.int32).cuda()
    tokens = torch.tensor([[9, 0, 0, 4, -1, 1]], dtype=torch.int32).cuda()
    for u in ([0.9, 0.75, 0.01, 0.01, 0.01, 0.4], [0.9, 0.4, 0.1, 0.1, 0.1, 0.1], [0.2, 0.75, 0.1, 0.1, 0.1, 0.75],
              [0.2, 0.5, 0.1, 0.1, 0.1, 0.5]):
        s = dict(target_probs=p, tokens=tokens, parents=parents, uniforms=torch.tensor([u]).cuda())
        check(s, [(0, 6)], 5)
        check(dict(s), [(0, 6)], 0)


def test_nothing_left_and_rows_of_one_token():
    # p has all its mass on the child that is rejected by a coin of 1 - 2^-24 of p = 1 - 2^-23
    V = 300
    p = torch.zeros((3, V)).cuda()
    p[0, 7], p[1, 5], p[2, 9] = 1 - 2.0 ** -23, 1.0, 1.0
    s = dict(target_probs=p, tokens=torch.tensor([[0, 7, 5]], dtype=torch.int32).cuda(),
             parents=torch.tensor([[-1, 0, 1]], dtype=torch.int32).cuda(),
             uniforms=torch.tensor([[0.3, 1 - 2.0 ** -24, 0.5]]).cuda())
    want = check(s, [(0, 3)], 2)
    assert want["accepted_tokens"][0].tolist() == [7, -1, -1]
    s["uniforms"][0, 1] = 0.5
    assert check(s, [(0, 3)], 2)["accepted_tokens"][0].tolist() == [7, 5, 9]


def test_parents_that_are_no_nodes_before():
    s, windows = make(6, [9] * 6, 64, sharp=6.0)
    s["parents"] = torch.tensor([0, 0, 5, -3, 1, 100, 2, 7, 1] * 6, dtype=torch.int32).cuda()
    par = s["parents"].clone().view(6, 9)
    row = torch.arange(9).cuda()
    clean = torch.where((par >= 0) & (par < row) & (row > 0), par, torch.full_like(par, -1)).view(-1)
    want = ref.tree(s["target_probs"], s["tokens"], clean, s["uniforms"], windows, 8)
    got = tv.tree_spec_sampling(D=8, **s)
    np.testing.assert_array_equal(got["accepted_tokens"].cpu().numpy(), want["accepted_tokens"])


def test_windows_that_do_not_fit():
    s, windows = make(7, [4] * 4, 100)
    s["qo_indptr"] = torch.tensor([0, 4, 2, 6, 17], dtype=torch.int32).cuda()
    got = {n: t.cpu().numpy() for n, t in tv.tree_spec_sampling(D=3, **s).items()}
    assert got["accept_length"][[1, 3]].tolist() == [0, 0] and (got["accept_length"][[0, 2]] > 0).all()
    for b in (1, 3):
        assert (got["accepted_tokens"][b] == -1).all() and (got["accept_index"][b] == -1).all()
        assert (got["logprobs"][b] == 0).all()


def test_emitted_token_has_the_targets_distribution():
    # one tree of three children, many coins: the first emitted token is a draw from p
    B, V = 60000, 6
    r = np.random.default_rng(8)
    p = np.array([0.3, 0.25, 0.2, 0.15, 0.07, 0.03], np.float32)
    s = dict(target_probs=torch.from_numpy(np.tile(p, (B * 4, 1))).cuda(),
             tokens=torch.tensor([[0, 1, 4, 0]] * B, dtype=torch.int32).cuda(),
             parents=torch.tensor([[-1, 0, 0, 0]] * B, dtype=torch.int32).cuda(),
             uniforms=torch.from_numpy(coins(r, (B, 4))).cuda())
    first = tv.tree_spec_sampling(D=1, **s)["accepted_tokens"][:, 0].cpu().numpy()
    seen = np.bincount(first, minlength=V)
    chi2 = ((seen - B * p) ** 2 / (B * p)).sum()
    assert chi2 < 25.7  # 5 degrees of freedom, 1e-4


def test_streams_and_graph():
    s, windows = make(9, [10] * 8, 5000)
    want = tv.tree_spec_sampling(D=9, **s)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = tv.tree_spec_sampling(D=9, **s, stream=stream)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = tv.tree_spec_sampling(D=9, **s)
    graph.replay()
    torch.cuda.synchronize()
    for n in want:
        assert torch.equal(got[n], want[n]) and torch.equal(captured[n], want[n])


def test_outputs_that_do_not_fit_are_refused():
    s, _ = make(10, [5] * 3, 100)
    new = lambda *shape: torch.empty(shape, dtype=torch.int32).cuda()  # noqa: E731
    good = [new(3, 5), new(3), new(3, 5), torch.empty((3, 5)).cuda()]
    tv.tree_spec_sampling(D=4, **s, outputs=good)
    for i, bad in ((0, new(3, 4)), (1, new(2)), (2, new(5, 3).t()), (3, torch.empty((3, 4)).cuda()),
                   (0, new(3, 5).long()), (3, new(3, 5)), (1, torch.empty(3, dtype=torch.int32))):
        with pytest.raises(ValueError):
            tv.tree_spec_sampling(D=4, **s, outputs=good[:i] + [bad] + good[i + 1:])
