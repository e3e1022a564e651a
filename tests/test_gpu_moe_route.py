"""The experts' router in training on the GPU against the float64 oracle."""
import numpy as np
import pytest
import torch

import fp8_scaled_matmul_amd as fm
from oracle import train

pytestmark = pytest.mark.gpu

U32, UBF = 2.0 ** -24, 2.0 ** -8
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def make(tokens, experts, dtype, seed=0):
    rng = np.random.default_rng(seed)
    l = torch.from_numpy((rng.normal(size=(tokens, experts)) * 2).astype(np.float32)).to(DTYPES[dtype])
    return l, rng


def check(l, top_k, renormalize, mask, gw, gb, r, dl):
    """Exponents off by their size (|l - max| times 2 U32) and 4 U32; sums of
    `experts` terms; a mean over the tokens with that many fp32 additions at
    most.  The gradient: a few products of such numbers, and the sums over the
    experts and the chosen ones."""
    L = l.double().cpu().numpy()
    experts = L.shape[1]
    ids, weights, counts, balance = train.route(L, top_k, renormalize, mask)
    assert np.array_equal(r.ids.cpu().numpy(), ids) and np.array_equal(r.counts.cpu().numpy(), counts)
    with np.errstate(invalid="ignore"):
        spread = np.nan_to_num(np.where(np.isfinite(L), L, 0).max(1) - np.where(np.isfinite(L), L, 0).min(1))
    rel = (2 * spread.max(initial=0) + 10 + experts) * U32
    assert (np.abs(r.weights.double().cpu().numpy() - weights) <= 2 * rel * weights + 2.0 ** -126).all()
    assert abs(r.balance.item() - balance) <= (2 * rel + len(L) * U32) * abs(balance) + U32 * abs(balance)
    GW = None if gw is None else gw.double().cpu().numpy()
    ref = train.route_backward(L, ids, counts, renormalize, GW, gb)
    # sizes of what is added up
    n = max(counts.sum() / top_k, 1)
    with np.errstate(invalid="ignore"):
        p = np.exp(L - L.max(1, keepdims=True))
        p = np.nan_to_num(p / p.sum(1, keepdims=True))
    share = abs(gb) * experts * counts / (n * n * top_k)
    size = p * (share + (p * share).sum(1, keepdims=True))
    if GW is not None:
        wg = (weights * np.abs(GW)).sum(1, keepdims=True)
        extra = weights * (np.abs(GW) + wg)
        for t in range(len(L)):
            if ids[t, 0] >= 0:
                size[t, ids[t]] += extra[t]
                size[t] += p[t] * wg[t]
    bound = (4 * rel + 8 * U32) * size + 2.0 ** -126
    bound += (UBF if l.dtype == torch.bfloat16 else U32) * np.abs(ref)
    got = dl.double().cpu().numpy()
    assert dl.dtype == l.dtype
    assert (np.abs(got - ref) <= bound).all(), (np.abs(got - ref) - bound).max()


CASES = [(1, 1, 1), (1, 64, 8), (2, 2, 2), (5, 3, 1), (7, 37, 3), (64, 65, 6), (63, 128, 8), (257, 129, 16), (1000, 16, 4),
         (33, 300, 5), (17, 512, 16), (2049, 256, 8)]


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("tokens,experts,top_k", CASES)
def test_against_oracle(tokens, experts, top_k, dtype, renormalize):
    l, rng = make(tokens, experts, dtype, seed=tokens + experts)
    mask = rng.random(tokens) < 0.75 if tokens % 2 else None
    gw = torch.from_numpy(rng.normal(size=(tokens, top_k)).astype(np.float32)).cuda()
    gb = torch.full((), 0.5, device="cuda")
    d = l.cuda()
    r = fm.moe_route(d, top_k, renormalize, mask=None if mask is None else torch.from_numpy(mask).cuda())
    check(l, top_k, renormalize, mask, gw, 0.5, r, fm.moe_route_backward(d, r, gw, gb))
    check(l, top_k, renormalize, mask, None, 0.5, r, fm.moe_route_backward(d, r, None, gb))
    check(l, top_k, renormalize, mask, gw, 0.0, r, fm.moe_route_backward(d, r, gw))
    assert (fm.moe_route_backward(d, r) == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_ties_and_signed_zeros_go_to_the_lower_expert(dtype):
    l = torch.zeros(3, 200, dtype=DTYPES[dtype])
    l[0, ::2] = -0.0
    l[1, 150:] = 1.0
    l[2] = torch.arange(200).remainder(3)
    r = fm.moe_route(l.cuda(), 5)
    assert r.ids.tolist() == [[0, 1, 2, 3, 4], [150, 151, 152, 153, 154], [2, 5, 8, 11, 14]]


@pytest.mark.parametrize("renormalize", [True, False])
def test_rows_that_leave_nothing(renormalize):
    """A row of -Inf alone counts as left out; experts at -Inf have no weight;
    the lowest finite values are values."""
    low = torch.finfo(torch.float32).min
    l = torch.zeros(6, 70)
    l[0] = -float("inf")
    l[1, 1:] = -float("inf")
    l[2] = low
    l[3, :69] = low
    l[4] = torch.arange(70.0)
    mask = torch.tensor([True, True, True, True, True, False])
    gw = torch.ones(6, 3)
    gw[5] = float("nan")
    l2 = l.clone()
    l2[5] = float("nan")        # what a token left out holds does not matter
    r = fm.moe_route(l2.cuda(), 3, renormalize, mask=mask.cuda())
    dl = fm.moe_route_backward(l2.cuda(), r, gw.cuda(), torch.ones((), device="cuda"))
    assert r.ids[0].tolist() == [-1] * 3 and r.ids[1].tolist() == [0, 1, 2] and r.ids[3].tolist() == [69, 0, 1]
    assert r.weights[0].tolist() == [0] * 3 and r.weights[1].tolist() == [1, 0, 0]
    on = [1, 2, 3, 4]
    gw[5] = 0
    ref = fm.moe_route(l[on].cuda(), 3, renormalize)
    assert torch.equal(r.ids[on], ref.ids) and torch.equal(r.weights[on], ref.weights) and torch.equal(r.counts, ref.counts)
    # the mean of 4 tokens' probabilities, added up in another order: 4 fp32
    # additions of numbers that are positive, a rounding of the result
    assert abs(r.balance.item() - ref.balance.item()) <= 2 * 5 * 2.0 ** -24 * ref.balance.item()
    assert torch.equal(dl[on], fm.moe_route_backward(l[on].cuda(), ref, gw[on].cuda(), torch.ones((), device="cuda")))
    assert (dl[[0, 5]] == 0).all()
    none = fm.moe_route(l2.cuda(), 3, renormalize, mask=torch.zeros(6, dtype=torch.bool, device="cuda"))
    assert (none.ids == -1).all() and (none.counts == 0).all() and none.balance.item() == 0
    assert (fm.moe_route_backward(l2.cuda(), none, gw.cuda(), torch.ones((), device="cuda")) == 0).all()


def test_nan_and_infinity_are_loud_in_their_rows():
    l, _ = make(4, 40, "fp32", seed=3)
    l[1, 7] = float("nan")
    l[2, 9] = float("inf")
    # over the chosen ones alone, a NaN that is not among them has no part in the sum
    assert torch.isfinite(fm.moe_route(l.cuda(), 4, renormalize=True).weights[1]).all()
    r = fm.moe_route(l.cuda(), 4, renormalize=False)
    assert 7 not in r.ids[1].tolist() and r.ids[2, 0].item() == 9
    assert torch.isnan(r.weights[1:3]).any(1).all() and torch.isfinite(r.weights[[0, 3]]).all()
    assert torch.isnan(r.balance)


def test_strides_no_tokens_and_far_rows():
    l, rng = make(50, 37, "bf16", seed=6)
    big = torch.full((52, 80), float("nan"), dtype=torch.bfloat16, device="cuda")
    v = big[1:-1, 3:40]
    v.copy_(l)
    out = torch.full((52, 80), 7.0, dtype=torch.bfloat16, device="cuda")
    gw = torch.from_numpy(rng.normal(size=(50, 4)).astype(np.float32)).cuda()
    a, b = fm.moe_route(l.cuda(), 4), fm.moe_route(v, 4)
    assert all(torch.equal(getattr(a, k), getattr(b, k)) for k in ("ids", "weights", "counts", "balance"))
    o = out[1:-1, 3:40]
    fm.moe_route_backward(v, b, gw, torch.ones(1, device="cuda"), out=o)
    assert torch.equal(o, fm.moe_route_backward(l.cuda(), a, gw, torch.ones(1, device="cuda")))
    o.fill_(7.0)
    assert (out == 7.0).all()
    r = fm.moe_route(torch.empty(0, 5, device="cuda"), 2)
    assert r.ids.shape == (0, 2) and r.counts.tolist() == [0] * 5 and r.balance.item() == 0
    assert fm.moe_route_backward(torch.empty(0, 5, device="cuda"), r).shape == (0, 5)
    # rows more than 2^32 bytes apart from the first
    far = torch.zeros((1 << 21) + 40, 1024, dtype=torch.bfloat16, device="cuda")
    far[-50:, :37] = l.cuda()
    w = far[:, :37]
    r = fm.moe_route(w, 4)
    assert torch.equal(r.ids[-50:], a.ids) and torch.equal(r.weights[-50:], a.weights)
    assert r.counts.sum().item() == 4 * len(far)


def test_captured_and_replayed_and_on_a_side_stream():
    l, rng = make(300, 100, "bf16", seed=8)
    x = l.cuda()
    gw, gb = torch.randn(300, 6, device="cuda"), torch.ones((), device="cuda")
    ws = torch.empty(fm.lib().fp8_moe_route_workspace_size(300, 100), dtype=torch.uint8, device="cuda")

    def step():
        r = fm.moe_route(x, 6, workspace=ws)
        return r, fm.moe_route_backward(x, r, gw, gb)

    step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        s, sd = step()
    side.synchronize()
    r, d = step()
    assert torch.equal(sd, d) and torch.equal(s.balance, r.balance)
    graphs, held = [], []
    for _ in range(2):              # two graphs, one workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append(step())
        graphs.append(g)
    for rep in range(3):
        for g, (r, d) in zip(graphs, held):
            x.copy_(x.roll(1, 1))
            want, wd = step()
            want = [v.clone() for v in (want.ids, want.weights, want.counts, want.balance, wd)]
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip((r.ids, r.weights, r.counts, r.balance, d), want):
                assert torch.equal(a, b), rep


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_nan_among_nothing_but_minus_infinity_is_loud(dtype, renormalize):
    l, _ = make(5, 40, dtype, seed=3)
    l[2] = -float("inf")
    l[2, 7] = float("nan")
    l[3] = -float("inf")
    r = fm.moe_route(l.cuda(), 4, renormalize)
    assert r.ids[2].tolist() == [0, 1, 2, 3] and torch.isnan(r.weights[2]).all() and torch.isnan(r.balance)
    assert r.ids[3].tolist() == [-1] * 4
    dl = fm.moe_route_backward(l.cuda(), r, torch.ones_like(r.weights))
    assert torch.isnan(dl[2]).any() and torch.isfinite(dl[[0, 1, 3, 4]]).all()


@pytest.mark.parametrize("tokens,experts,top_k", [(1, 1, 1), (70, 37, 3), (5000, 512, 16), (9000, 128, 8)])
def test_what_the_workspace_holds_does_not_matter(tokens, experts, top_k):
    l, _ = make(tokens, experts, "bf16", seed=experts)
    l = l.cuda()
    need = fm.lib().fp8_moe_route_workspace_size(tokens, experts)
    room = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    a, b = fm.moe_route(l, top_k, workspace=room[:need]), fm.moe_route(l, top_k)
    assert (room[need:] == 0xFF).all()
    for name in ("ids", "weights", "counts", "balance"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name
