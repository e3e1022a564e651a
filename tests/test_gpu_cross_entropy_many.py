"""The vocabulary loss with many tiles for each workgroup, against its definition
in float64 on the GPU."""
import pytest
import torch

import fp8_scaled_matmul_amd as fm

pytestmark = pytest.mark.gpu

U32, UBF = 2.0 ** -24, 2.0 ** -8        # half a step of fp32 and bf16, relative
TINY = 2.0 ** -126                      # smaller numbers count as 0


def make(tokens, vocab, hidden, seed, ignored=0.1):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(tokens, hidden, generator=gen, device="cuda").bfloat16()
    w = (torch.randn(vocab, hidden, generator=gen, device="cuda") * 2 * hidden ** -0.5).bfloat16()
    t = torch.randint(0, vocab, (tokens,), generator=gen, device="cuda")
    t[torch.rand(tokens, generator=gen, device="cuda") < ignored] = -100
    return x, w, t, torch.randn(tokens, generator=gen, device="cuda")


def run(x, w, t, g, softcap):
    loss, lse = fm.linear_cross_entropy(x, w, t, softcap=softcap)
    dx, dw = fm.linear_cross_entropy_backward(x, w, t, lse, g, softcap=softcap)
    return dict(loss=loss, lse=lse, dx=dx, dw=dw)


def expect(x, w, t, g, softcap):
    """Reference and bound of every output.

    A logit is a sum of `hidden` exact products in fp32: off by (hidden + 1) U32
    sum |x w| at most; the cap adds 8 U32 softcap.  lse: the largest logit error,
    each exponent's rounding, vocab / 64 + 90 additions, the logarithm.  dl: the
    errors of z and lse relative to p, the slope's, bf16's rounding.  dx and dw: dl's
    errors through the other operand, fp32 additions of `vocab` and `tokens` terms,
    bf16's rounding."""
    X, W, G = x.double(), w.double(), g.double()
    on = (t >= 0) & (t < len(w))
    at = torch.where(on, t, 0)[:, None]
    z = X @ W.t()
    e_z = (X.shape[1] + 1) * U32 * (X.abs() @ W.abs().t()) + 8 * U32 * softcap
    slope = None
    if softcap:
        th = torch.tanh(z / softcap)
        z, slope = softcap * th, 1 - th * th
    lse = torch.logsumexp(z, 1)
    loss = torch.where(on, lse - z.gather(1, at)[:, 0], 0.0)
    e_lse = e_z.amax(1) + U32 * (len(w) / 64 + 94 + 2 * z.abs().amax(1) + 2 * lse.abs())
    e_loss = torch.where(on, e_lse + e_z.gather(1, at)[:, 0] + U32 * loss.abs(), 0.0)
    p = torch.exp(z - lse[:, None])
    G = torch.where(on, G, 0.0)[:, None]
    full = p.scatter_add(1, at, -on.double()[:, None]) * G          # without the slope
    d = full if slope is None else full * slope
    e_d = p * G.abs() * (e_z + e_lse[:, None] + U32 * (2 * z.abs() + 2 * lse.abs()[:, None] + 4))
    e_d += d.abs() * (UBF + 4 * U32) + 2 * TINY * G.abs().amax()
    if slope is not None:
        e_d += full.abs() * (2 * z.abs() * e_z / softcap ** 2 + 4 * U32)
    e_d *= on[:, None]
    del p, full, slope, z, e_z
    X = torch.where(on[:, None], X, 0.0)
    dx, dw = d @ W, d.t() @ X
    a = d.abs()
    e_dx = (e_d + (len(w) + 2) * U32 * a) @ W.abs() + UBF * dx.abs() + TINY
    e_dw = (e_d + (len(x) + 2) * U32 * a).t() @ X.abs() + UBF * dw.abs() + TINY
    return dict(loss=(loss, e_loss), lse=(lse, e_lse), dx=(dx, e_dx), dw=(dw, e_dw))


def check(got, want):
    for name, (ref, bound) in want.items():
        excess = ((got[name].double() - ref).abs() - bound).amax().item()
        assert excess <= 0, f"{name}: {excess} over the bound"


@pytest.mark.parametrize("softcap", [0.0, 3.0])
@pytest.mark.parametrize("tokens,vocab,hidden", [(8192, 16384, 32), (8192, 16384, 31), (8190, 16400, 8), (1300, 100003, 16),
                                                 (4100, 30001, 33), (4100, 30001, 1)])
def test_one_and_two_stages_of_k_and_many_tiles(tokens, vocab, hidden, softcap):
    """Widths of one stage of K (and of two) with 7 to 9 tiles of 256 x 256 a
    workgroup, of changing tokens: each tile's epilogue has its own tokens' targets,
    sums and gradients."""
    args = make(tokens, vocab, hidden, seed=hidden)
    want = expect(*args, softcap)
    got = run(*args, softcap)
    check(got, want)
    again = run(*args, softcap)
    assert all(torch.equal(got[k], again[k]) for k in got)


@pytest.mark.parametrize("softcap", [0.0, 3.0])
@pytest.mark.parametrize("tokens,vocab,hidden", [(1, 300, 64), (20, 5000, 33), (70, 4101, 64), (120, 700, 40), (300, 600, 64),
                                                 (600, 20005, 33), (2000, 9000, 40), (70001, 4501, 64)])
def test_a_word_that_cannot_come_and_tokens_that_do_not_count(tokens, vocab, hidden, softcap):
    """A vocabulary row of -Inf is as one of -2^20, whose exponentials are 0 as well:
    tokens that do not count still add nothing to dw, and their dx is 0."""
    x, w, t, g = make(tokens, vocab, hidden, seed=tokens)
    x = x.abs() + 0.5
    t = t.clamp(max=vocab - 2)          # the last one is the word
    if tokens > 1:
        t[::3] = -1
        t[1::7] = vocab
    on = (t >= 0) & (t < vocab)
    got = {}
    for name, value in (("finite", -2.0 ** 20), ("infinite", -float("inf"))):
        w2, x2 = w.clone(), x.clone()
        w2[-1] = value
        x2[~on] = float("nan")
        got[name] = run(x2, w2, t, g, softcap)
    a, b = got["finite"], got["infinite"]
    assert torch.equal(a["dw"], b["dw"]) and torch.isfinite(b["dw"]).all()
    assert torch.equal(a["loss"][on], b["loss"][on]) and torch.equal(a["lse"][on], b["lse"][on])
    assert (a["dx"][~on] == 0).all() and (b["dx"][~on] == 0).all()
    if not softcap:                     # the word adds nothing
        assert (b["dw"][-1] == 0).all()
        if tokens * vocab < 1 << 25:
            t2 = torch.where(on, t, -1)
            want = expect(x, w[:-1], t2, g, softcap)
            check({"dw": a["dw"][:-1]}, {"dw": want["dw"]})
            check({"dx": a["dx"]}, {"dx": want["dx"]})


@pytest.mark.parametrize("softcap", [0.0, 3.0])
@pytest.mark.parametrize("tokens,vocab,hidden", [(4096, 70000, 64), (4099, 66001, 33)])
def test_pieces_of_the_vocabulary_with_split_sums(tokens, vocab, hidden, softcap):
    """dx of two pieces of the vocabulary (512 MiB of dl each at most), each summed in
    16 parts."""
    args = make(tokens, vocab, hidden, seed=vocab)
    got = run(*args, softcap)
    check(got, expect(*args, softcap))


def rounded(v):
    return v.float().bfloat16().double()


@pytest.mark.parametrize("kind", ["mean", "each"])
@pytest.mark.parametrize("softcap", [0.0, 15.0])
@pytest.mark.parametrize("tokens,vocab,hidden", [(50, 4100, 256), (700, 9000, 200), (3000, 5000, 256)])
def test_gradients_lose_one_rounding_of_the_logits_gradient_and_one_of_their_own(tokens, vocab, hidden, softcap, kind):
    """The norm of dx's and dw's error.  What the documentation gives away: dl over
    the largest |gradient| is rounded to bf16, and so is the result.  Both are made
    here in float64; their errors are independent, so their squares add up.  Of at
    least 12800 entries the norms of either and of their sum are within 1 / sqrt(12800)
    of that; logits in fp32 add some 1e-6.  5 %: one more rounding of either kind, or a
    bit less in one, adds 15 % or more wherever that rounding counts."""
    x, w, t, g = make(tokens, vocab, hidden, seed=tokens)
    on = t >= 0
    x += (3 * torch.rand(tokens, 1, device="cuda") * w[t.clamp(min=0)].float()).bfloat16()
    if kind == "mean":
        g = torch.full_like(g, 1.0) / on.sum()
    X, W = torch.where(on[:, None], x.double(), 0.0), w.double()
    z, slope = X @ W.t(), 1.0
    if softcap:
        th = torch.tanh(z / softcap)
        z, slope = softcap * th, 1 - th * th
    d = torch.softmax(z, 1)
    d.scatter_add_(1, t.clamp(min=0)[:, None], -on.double()[:, None])
    d *= torch.where(on, g.double(), 0.0)[:, None] * slope
    by = torch.where(on, g.abs(), 0.0).amax().double()
    off = rounded(d / by) * by - d
    got = run(x, w, t, g, softcap)
    for name, ref, via in (("dx", d @ W, off @ W), ("dw", d.t() @ X, off.t() @ X)):
        own = rounded(ref) - ref
        want = (own.norm() ** 2 + via.norm() ** 2).sqrt() / ref.norm()
        err = (got[name].double() - ref).norm() / ref.norm()
        assert err.item() <= 1.05 * want.item()
