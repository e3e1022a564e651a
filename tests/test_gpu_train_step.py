"""The training operators as a step uses them: dropout onto a residual stream, an
expert router with its balance loss, the vocabulary loss, and back; against
torch's float64 autograd on the same values, and captured."""
import pytest
import torch

import fp8_scaled_matmul_amd as fm
from oracle import train

pytestmark = pytest.mark.gpu

RATE, TOP_K, CAP = 0.25, 2, 15.0


def inputs(tokens, hidden, experts, vocab):
    gen = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen)
    h, res = r(tokens, hidden).bfloat16(), r(tokens, hidden).bfloat16()
    router, w = (r(experts, hidden) * hidden ** -0.5).bfloat16(), (r(vocab, hidden) * hidden ** -0.5).bfloat16()
    t = torch.randint(0, vocab, (tokens,), generator=gen)
    t[::7] = -100
    return [a.cuda() for a in (h, res, router, w, t)]


def step(h, res, router, w, t, seed, grad):
    """The loss' mean, balance, and gradients of h, res, router, w.  The router's
    small product is torch's; its experts are left out (each token's weight stands
    for them)."""
    x = fm.dropout(h, RATE, seed, residual=res)
    logits = x.float() @ router.float().t()
    r = fm.moe_route(logits, TOP_K)
    loss, lse = fm.linear_cross_entropy(x, w, t, softcap=CAP)
    total = (loss * grad).sum() + 0.01 * r.balance + r.weights[:, 0].sum() * 1e-3
    dx, dw = fm.linear_cross_entropy_backward(x, w, t, lse, grad, softcap=CAP)
    gw = torch.zeros_like(r.weights)
    gw[:, 0] = 1e-3
    dl = fm.moe_route_backward(logits, r, gw, torch.full((), 0.01, device="cuda"))
    dx = (dx.float() + dl @ router.float()).bfloat16()
    return total, x, fm.dropout(dx, RATE, seed), dx, dl.t() @ x.float(), dw


def test_against_autograd():
    h, res, router, w, t = inputs(96, 128, 8, 500)
    seed = torch.tensor([77], device="cuda")
    grad = torch.full((96,), 1.0, device="cuda") / (t >= 0).sum()
    total, x, dh, dres, drouter, dw = step(h, res, router, w, t, seed, grad)

    keep = torch.from_numpy(train.dropout_bits(96, 128, 77) >= 16384).cuda()
    leaves = [a.double().requires_grad_() for a in (h, res, router, w)]
    H, R, Q, W = leaves
    X = torch.where(keep, H * (4.0 / 3.0), 0.0) + R
    X = X + (x.double() - X).detach()           # bf16's rounding passed through
    logits = X @ Q.t()
    p = torch.softmax(logits, 1)
    top = torch.argsort(-logits, dim=1, stable=True)[:, :TOP_K]
    weights = torch.softmax(logits.gather(1, top), 1)
    f = torch.bincount(top.flatten(), minlength=8).double() / (96 * TOP_K)
    z = CAP * torch.tanh(X @ W.t() / CAP)
    on = t >= 0
    loss = torch.nn.functional.cross_entropy(z[on], t[on], reduction="sum") / on.sum()
    want = loss + 0.01 * 8 * (f * p.mean(0)).sum() + 1e-3 * weights[:, 0].sum()
    want.backward()
    assert abs(total.item() - want.item()) < 1e-5 * abs(want.item())
    # dl and dx are bf16: 2^-8 of what is added up, which exceeds the sums' norm by
    # the random signs' factor at most
    for got, leaf in ((dh, H), (dres, R), (drouter, Q), (dw, W)):
        err = (got.double() - leaf.grad).norm() / leaf.grad.norm()
        assert err.item() < 2.0 ** -7, err.item()


def test_two_captured_steps_replayed_in_turn():
    args = inputs(200, 256, 16, 1000)
    seed = torch.tensor([5], device="cuda")
    grad = torch.full((200,), 1 / 200, device="cuda")
    step(*args, seed, grad)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(*args, seed, grad))
        graphs.append(g)
    for rep in range(3):
        for g, out in zip(graphs, outs):
            seed.add_(1)
            want = [v.clone() for v in step(*args, seed, grad)]
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(out, want):
                assert torch.equal(a, b), rep


def test_the_short_way_and_the_checked_way_agree(monkeypatch):
    """Calls that are in order go through the extension module, the others through
    ctypes: the same kernels on the same arguments."""
    args = inputs(70, 128, 16, 600)
    seed = torch.tensor([5], device="cuda")
    grad = torch.randn(70, generator=torch.Generator().manual_seed(1)).cuda()
    short = step(*args, seed, grad)
    monkeypatch.setattr(fm, "_ext_module", fm._NoExt())
    for a, b in zip(short, step(*args, seed, grad)):
        assert torch.equal(a, b)


def test_two_threads_on_two_streams():
    import threading
    cases = [(inputs(n, 256, 16, 1000), torch.tensor([n], device="cuda"), torch.full((n,), 1 / n, device="cuda"))
             for n in (33, 300)]
    want = [[v.clone() for v in step(*a, s, g)] for a, s, g in cases]
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        a, s, g = cases[i]
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(10):
                got[i].append(step(*a, s, g))
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in range(2):
        assert len(got[i]) == 10
        for out in got[i]:
            for a, b in zip(out, want[i]):
                assert torch.equal(a, b)


def test_refusals_are_the_same_on_the_device():
    h, res, router, w, t = inputs(8, 64, 8, 100)
    f = torch.zeros(8, device="cuda")
    seed = torch.tensor([5], device="cuda")
    r = fm.moe_route(h, 2)
    for call in (
        lambda: fm.dropout(h, 1.5, seed),
        lambda: fm.dropout(h, float("nan"), seed),
        lambda: fm.dropout(h, 0.1, seed, residual=res[:, :32]),
        lambda: fm.linear_cross_entropy(h, w, t, softcap=1e-50),
        lambda: fm.linear_cross_entropy_backward(h, w, t, f, f, softcap=1e-50),
        lambda: fm.linear_cross_entropy(h, w, t[:7]),
        lambda: fm.linear_cross_entropy(h, w, t.cpu()),
        lambda: fm.linear_cross_entropy_backward(h, w, t, f[:7], f),
        lambda: fm.moe_route(h, 65),
        lambda: fm.moe_route(h, 2, mask=torch.ones(7, dtype=torch.bool, device="cuda")),
        lambda: fm.moe_route_backward(h[:4], r),
    ):
        with pytest.raises(ValueError):
            call()
    # what any true value says
    a = fm.moe_route_backward(h, fm.Route(r.ids, r.weights, r.counts, r.balance, 1), torch.ones_like(r.weights))
    assert torch.equal(a, fm.moe_route_backward(h, r, torch.ones_like(r.weights)))
