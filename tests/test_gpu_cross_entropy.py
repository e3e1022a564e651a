"""The vocabulary loss on the GPU against the float64 oracle: sizes where tiles,
reads and pieces end, targets that do not count, strides, graphs, streams."""
import numpy as np
import pytest
import torch

import fp8_scaled_matmul_amd as fm
from oracle import train

pytestmark = pytest.mark.gpu

U32, UBF = 2.0 ** -24, 2.0 ** -8        # half a step of fp32 and bf16, relative


def make(tokens, vocab, hidden, seed=0, ignored=0.2, scale=2.0):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.normal(size=(tokens, hidden)).astype(np.float32)).bfloat16()
    w = torch.from_numpy((rng.normal(size=(vocab, hidden)) * scale * hidden ** -0.5).astype(np.float32)).bfloat16()
    t = rng.integers(0, vocab, size=tokens)
    t[rng.random(tokens) < ignored] = -100
    g = rng.normal(size=tokens).astype(np.float32)
    return x, w, torch.from_numpy(t), torch.from_numpy(g)


def expect(x, w, t, g, softcap):
    """Reference and error bounds of every output.

    A logit is a sum of `hidden` exact products in fp32: off by (hidden + 1)
    U32 sum |x w| at most; the cap adds 8 U32 softcap.  lse: the largest logit
    error; each term's exponent (its size times U32) and 4 U32; at most
    vocab / 64 + 90 additions; the logarithm.  p = exp(z - lse) is off by the
    sum of these, relatively; dl by that, the slope's error and bf16's rounding;
    dx and dw by the errors of dl through the other operand, `vocab` or `tokens`
    fp32 additions and bf16's rounding."""
    X, W, T, G = x.double().numpy(), w.double().numpy(), t.numpy(), g.double().numpy()
    loss, lse = train.cross_entropy(X, W, T, softcap)
    z, slope = train.logits(X, W, softcap)
    e_z = (X.shape[1] + 1) * U32 * (np.abs(X) @ np.abs(W).T) + 8 * U32 * softcap
    e_lse = e_z.max(1) + U32 * (W.shape[0] / 64 + 94 + 2 * np.abs(z).max(1) + 2 * np.abs(lse))
    on = (T >= 0) & (T < len(W))
    e_loss = np.where(on, e_lse + e_z[np.arange(len(T)), np.where(on, T, 0)] + U32 * np.abs(np.nan_to_num(loss)), 0)
    d, p = train.logits_grad(X, W, T, G, softcap)
    e_p = e_z + e_lse[:, None] + U32 * (2 * np.abs(z) + 2 * np.abs(lse)[:, None] + 4)
    # numbers below the smallest normal one, 2^-126, count as 0: an exponential,
    # then its product with the gradient
    e_d = p * e_p + np.abs(d) * (UBF + 4 * U32) + on[:, None] * 2.0 ** -126 * (1 + np.abs(G))[:, None]
    if softcap:
        full = np.abs(np.divide(d, slope, out=np.zeros_like(d), where=slope > 0))
        e_d += full * (2 * np.abs(z) * e_z / softcap ** 2 + 4 * U32)
    Xon = np.where(on[:, None], X, 0)
    dx, dw = d @ W, d.T @ Xon
    e_dx = e_d @ np.abs(W) + (len(W) + 2) * U32 * (np.abs(d) @ np.abs(W)) + UBF * np.abs(dx)
    e_dw = e_d.T @ np.abs(Xon) + (len(X) + 2) * U32 * (np.abs(d).T @ np.abs(Xon)) + UBF * np.abs(dw)
    return dict(loss=(loss, e_loss), lse=(lse, e_lse), dx=(dx, e_dx), dw=(dw, e_dw))


def check(got, want, name):
    ref, bound = want[name]
    a = got.double().cpu().numpy()
    bad = np.isnan(ref)
    assert np.array_equal(np.isnan(a), bad), name
    # 2^-126: the smallest normal number
    excess = np.abs(a - ref)[~bad] - (bound[~bad] if bound.shape == ref.shape else bound) - 2.0 ** -126
    assert excess.size == 0 or excess.max() <= 0, f"{name}: {excess.max()} over the bound"


def run(x, w, t, g, softcap=0.0, **kw):
    loss, lse = fm.linear_cross_entropy(x, w, t, softcap=softcap)
    dx, dw = fm.linear_cross_entropy_backward(x, w, t, lse, g, softcap=softcap, **kw)
    return dict(loss=loss, lse=lse, dx=dx, dw=dw)


SIZES = [(1, 1, 1), (1, 257, 8), (2, 2, 3), (3, 1000, 33), (31, 300, 64), (32, 64, 32), (33, 513, 72), (64, 777, 200),
         (65, 256, 96), (128, 255, 31), (129, 1025, 40), (257, 511, 264), (300, 2049, 1000), (513, 130, 520)]


@pytest.mark.parametrize("softcap", [0.0, 3.0])
@pytest.mark.parametrize("tokens,vocab,hidden", SIZES)
def test_against_oracle(tokens, vocab, hidden, softcap):
    x, w, t, g = make(tokens, vocab, hidden, seed=tokens + vocab)
    want = expect(x, w, t, g, softcap)
    got = run(x.cuda(), w.cuda(), t.cuda(), g.cuda(), softcap)
    for name in got:
        check(got[name], want, name)


def test_more_tiles_than_whole_rounds():
    """More tiles of 256 x 256 than compute units, in each product: the rows behind
    the last whole round have a launch of their own (257 tokens: two tiles across)."""
    x, w, t, g = make(257, 65700, 72, seed=3)
    want = expect(x, w, t, g, 0.0)
    got = run(x.cuda(), w.cuda(), t.cuda(), g.cuda())
    for name in got:
        check(got[name], want, name)


def test_large_logits_and_cap():
    """Logits of some hundreds: one token of the vocabulary takes all."""
    for softcap in (0.0, 20.0):
        x, w, t, g = make(70, 600, 128, seed=5, scale=60.0)
        want = expect(x, w, t, g, softcap)
        got = run(x.cuda(), w.cuda(), t.cuda(), g.cuda(), softcap)
        for name in got:
            check(got[name], want, name)


@pytest.mark.parametrize("tokens", [5, 70, 300])
def test_tokens_that_do_not_count_add_nothing(tokens):
    """Their x, their gradient may hold anything; targets past the vocabulary
    are loud in the loss and count for nothing."""
    x, w, t, g = make(tokens, 400, 64, seed=9, ignored=0.0)
    t[1::5] = -1
    t[2::5] = 400
    t[3::5] = 1 << 40
    want = expect(x, w, t, g, 0.0)
    off = (t < 0) | (t >= 400)
    x2, g2 = x.clone(), g.clone()
    x2[off] = float("nan")
    x2[off, 0] = float("inf")
    g2[off] = float("nan")
    got = run(x2.cuda(), w.cuda(), t.cuda(), g2.cuda())
    on = ~off
    assert (got["loss"].cpu()[t < 0] == 0).all() and torch.isnan(got["loss"].cpu()[t >= 400]).all()
    assert (got["dx"].cpu()[off] == 0).all()
    check(got["dw"], want, "dw")
    for name in ("loss", "lse", "dx"):
        ref, bound = want[name]
        check(got[name][on.cuda()], {name: (ref[on.numpy()], bound[on.numpy()])}, name)
    all_off = torch.full_like(t, -100)
    dx, dw = fm.linear_cross_entropy_backward(x2.cuda(), w.cuda(), all_off.cuda(), got["lse"], g2.cuda())
    assert (dx == 0).all() and (dw == 0).all()


@pytest.mark.parametrize("tokens,vocab,hidden", [(5, 300, 64), (70, 259, 40), (300, 600, 1000)])
def test_strides_and_alignment(tokens, vocab, hidden):
    """Views of larger tensors at any element; rows and columns beside the
    outputs stay as they were."""
    x, w, t, g = make(tokens, vocab, hidden, seed=3)
    want = expect(x, w, t, g, 0.0)
    plain = run(x.cuda(), w.cuda(), t.cuda(), g.cuda())
    for pad in (1, 8):
        def view(a):
            big = torch.full((a.shape[0] + 2, a.shape[1] + 2 * pad), float("nan"), dtype=a.dtype, device="cuda")
            v = big[1:-1, pad:-pad]
            v.copy_(a)
            return big, v

        _, xv = view(x)
        _, wv = view(w)
        bx, ox = view(torch.zeros_like(x))
        bw, ow = view(torch.zeros_like(w))
        bx.fill_(7.0)
        bw.fill_(7.0)
        gv = torch.zeros(2 * tokens, device="cuda")[::2]
        gv.copy_(g)
        got = run(xv, wv, t.cuda(), gv, out_x=ox, out_w=ow)
        assert got["dx"] is ox and got["dw"] is ow
        for name in got:
            check(got[name], want, name)
            assert torch.equal(got[name], plain[name]), name
        for big, v in ((bx, ox), (bw, ow)):
            v.fill_(7.0)
            assert (big == 7.0).all()


def test_one_gradient_for_all_and_one_side():
    x, w, t, g = [a.cuda() for a in make(100, 500, 96, seed=4)]
    loss, lse = fm.linear_cross_entropy(x, w, t)
    one = torch.full((), 0.25, device="cuda")
    a = fm.linear_cross_entropy_backward(x, w, t, lse, one.expand(100))
    b = fm.linear_cross_entropy_backward(x, w, t, lse, one.repeat(100))
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    dx, none = fm.linear_cross_entropy_backward(x, w, t, lse, one.expand(100), want_w=False)
    assert none is None and torch.equal(dx, a[0])
    none, dw = fm.linear_cross_entropy_backward(x, w, t, lse, one.expand(100), want_x=False)
    assert none is None and torch.equal(dw, a[1])


def test_no_tokens():
    w = torch.ones(30, 24, dtype=torch.bfloat16, device="cuda")
    x = torch.empty(0, 24, dtype=torch.bfloat16, device="cuda")
    t = torch.empty(0, dtype=torch.int64, device="cuda")
    got = run(x, w, t, torch.empty(0, device="cuda"))
    assert got["loss"].shape == (0,) and got["dx"].shape == (0, 24) and (got["dw"] == 0).all()


def test_empty_vocabulary_rows():
    """A vocabulary row of -Inf logits (a word that cannot come) adds nothing."""
    x = torch.ones(3, 16, dtype=torch.bfloat16)
    w = torch.zeros(300, 16, dtype=torch.bfloat16)
    w[::3] = -float("inf")
    w[1::3] = 0.25
    loss, lse = fm.linear_cross_entropy(x.cuda(), w.cuda(), torch.tensor([1, 2, 0]).cuda())
    ref = np.log(100 * np.exp(4.0) + 100)
    assert np.abs(lse.cpu().numpy() - ref).max() < 1e-5 and loss[2].item() == float("inf")


@pytest.mark.parametrize("softcap", [0.0, 15.0])
def test_tokens_in_pieces_and_vocabulary_in_pieces(softcap):
    """More tokens than a forward pass takes at once, more logits than a piece
    holds; the reference in float64 on the GPU."""
    tokens, vocab, hidden = 70001, 4501, 64
    x, w, t, g = [a.cuda() for a in make(tokens, vocab, hidden, seed=8)]
    got = run(x, w, t, g, softcap)
    X, W = x.double(), w.double()
    z, slope = X @ W.t(), 1.0
    if softcap:
        th = torch.tanh(z / softcap)
        z, slope = softcap * th, 1 - th * th
    lse = torch.logsumexp(z, 1)
    on = t >= 0
    at = t.clamp(min=0)
    loss = torch.where(on, lse - z.gather(1, at[:, None])[:, 0], 0.0)
    d = torch.exp(z - lse[:, None])
    d.scatter_add_(1, at[:, None], torch.full_like(lse, -1.0)[:, None])
    d *= torch.where(on, g.double(), 0.0)[:, None] * slope
    del z, slope
    # logits: 65 U32 sum |x w|, about 65 * 2^-24 * 64 * 0.8 * 0.2; see expect()
    assert (got["lse"].double() - lse).abs().max() < 2e-4
    assert (got["loss"].double() - loss).abs().max() < 4e-4
    dx, dw = d @ W, d.t() @ X
    ax, aw = d.abs() @ W.abs(), d.abs().t() @ X.abs()
    # dl: bf16's rounding, 4e-4 from the logits; sums of 4501 and 70001 terms in fp32
    assert ((got["dx"].double() - dx).abs() <= (UBF + 4e-4 + 4501 * U32) * ax + UBF * dx.abs()).all()
    assert ((got["dw"].double() - dw).abs() <= (UBF + 4e-4 + 70001 * U32) * aw + UBF * dw.abs()).all()
    again = run(x, w, t, g, softcap)
    assert all(torch.equal(got[k], again[k]) for k in got)


def test_gradient_matches_differences_of_the_loss():
    """Along a direction of x and of w, by the kernel's own losses: fp32 losses
    of about 6 over steps of 2^-4 limit it to 2^-23 * 6 * 40 / 2^-4; the step's third
    derivative and bf16's rounding of dl and of the results to 2%."""
    x, w, t, g = make(40, 300, 64, seed=12, ignored=0.0)
    g = torch.ones(40)
    loss, lse = fm.linear_cross_entropy(x.cuda(), w.cuda(), t.cuda())
    dx, dw = fm.linear_cross_entropy_backward(x.cuda(), w.cuda(), t.cuda(), lse, g.cuda())
    rng = np.random.default_rng(0)
    for a, grad, which in ((x, dx, 0), (w, dw, 1)):
        ref = train.cross_entropy_backward(x.double().numpy(), w.double().numpy(), t.numpy(), np.ones(40))[which]
        direction = np.sign(ref) * (rng.random(a.shape) < 0.5) * 2.0 ** -6
        up, down = (a.double().numpy() + direction), (a.double().numpy() - direction)
        up, down = torch.from_numpy(up).bfloat16(), torch.from_numpy(down).bfloat16()
        moved = (up.double() - down.double()).numpy()
        both = [fm.linear_cross_entropy(*(((m, w) if which == 0 else (x, m))[i].cuda() for i in (0, 1)), t.cuda())[0]
                for m in (up, down)]
        change = (both[0].double() - both[1].double()).sum().item()
        along = (grad.double().cpu().numpy() * moved).sum()
        assert abs(change - along) < 0.02 * abs(along) + 40 * 6 * 2.0 ** -23 * 4


def test_captured_and_replayed():
    """Two captured steps share a workspace, replayed in turn with eager work
    between; each replay reads the inputs anew."""
    a = [v.cuda() for v in make(90, 700, 128, seed=21)]
    b = [v.cuda() for v in make(300, 300, 72, seed=22)]
    need = max(fm.lib().fp8_linear_ce_workspace_size(s[0].shape[0], s[1].shape[0], s[0].shape[1], back)
               for s in (a, b) for back in (0, 1))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    outs = [dict(dx=torch.empty_like(s[0]), dw=torch.empty_like(s[1])) for s in (a, b)]

    def step(s, o):
        x, w, t, g = s
        loss, lse = fm.linear_cross_entropy(x, w, t, softcap=5.0, workspace=ws)
        fm.linear_cross_entropy_backward(x, w, t, lse, g, softcap=5.0, out_x=o["dx"], out_w=o["dw"], workspace=ws)
        return loss, lse

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for s, o in zip((a, b), outs):
            step(s, o)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs, held = [], []
    for s, o in zip((a, b), outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held.append(step(s, o))
        graphs.append(graph)
    for rep in range(3):
        for s, o, graph, h in zip((a, b), outs, graphs, held):
            s[0].copy_(s[0].roll(1, 0))
            want = run(*s, 5.0)
            for v in o.values():
                v.zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            for name, v in (("loss", h[0]), ("lse", h[1]), ("dx", o["dx"]), ("dw", o["dw"])):
                assert torch.equal(v, want[name]), (rep, name)


def test_on_a_side_stream():
    x, w, t, g = [v.cuda() for v in make(200, 900, 256, seed=31)]
    want = run(x, w, t, g)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = run(x, w, t, g)
    side.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want)


def test_an_infinite_gradient_is_loud_in_its_token():
    x, w, t, g = make(70, 300, 64, seed=4, ignored=0.0)
    for bad in (float("inf"), float("nan")):
        g2 = g.clone()
        g2[9] = bad
        got = run(x.cuda(), w.cuda(), t.cuda(), g2.cuda())
        want = expect(x, w, t, g, 0.0)
        assert not torch.isfinite(got["dx"][9]).any()
        on = np.arange(70) != 9
        check(got["dx"][torch.from_numpy(on).cuda()], {"dx": (want["dx"][0][on], want["dx"][1][on])}, "dx")


@pytest.mark.parametrize("tokens,vocab,hidden", [(1, 257, 8), (5, 4100, 33), (70, 2059, 40), (257, 65700, 72), (300, 2049, 1000)])
def test_what_the_workspace_holds_does_not_matter(tokens, vocab, hidden):
    """Full of NaN, and no larger than asked for: nothing behind it is written."""
    x, w, t, g = [v.cuda() for v in make(tokens, vocab, hidden, seed=vocab)]
    want = run(x, w, t, g)
    size = fm.lib().fp8_linear_ce_workspace_size
    got = {}
    for back in (0, 1):
        need = size(tokens, vocab, hidden, back)
        room = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
        if back:
            got["dx"], got["dw"] = fm.linear_cross_entropy_backward(x, w, t, got["lse"], g, workspace=room[:need])
        else:
            got["loss"], got["lse"] = fm.linear_cross_entropy(x, w, t, workspace=room[:need])
        assert (room[need:] == 0xFF).all()
        with pytest.raises(ValueError, match="workspace"):
            if back:
                fm.linear_cross_entropy_backward(x, w, t, got["lse"], g, workspace=room[:need - 1])
            else:
                fm.linear_cross_entropy(x, w, t, workspace=room[:need - 1])
    for name in want:
        assert torch.equal(got[name], want[name]), name


@pytest.mark.parametrize("softcap", [0.0, 3.0])
@pytest.mark.parametrize("tokens,vocab,hidden", [(20, 30001, 24), (50, 30003, 40), (100, 25002, 72), (300, 13001, 40), (600, 20005, 33)])
def test_each_tile_of_the_logits(tokens, vocab, hidden, softcap):
    """Enough vocabulary for each tile: 128 x 32, 128 x 64, 256 x 128 (of up to 128
    tokens and of more), 256 x 256."""
    x, w, t, g = make(tokens, vocab, hidden, seed=tokens)
    want = expect(x, w, t, g, softcap)
    got = run(x.cuda(), w.cuda(), t.cuda(), g.cuda(), softcap)
    for name in got:
        check(got[name], want, name)
