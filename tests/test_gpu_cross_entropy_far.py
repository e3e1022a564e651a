"""The vocabulary loss where offsets pass 32 bits: a weight, and hidden states, of
more than 4 GiB; the reference in float64 on the GPU, by pieces."""
import pytest
import torch

import fp8_scaled_matmul_amd as fm

pytestmark = pytest.mark.gpu

U32, UBF = 2.0 ** -24, 2.0 ** -8


def _reference(x, w, t, g, rows=65536):
    """loss, lse, dx, dw (bf16's worth of it), and sums of sizes for the bounds."""
    X = x.double()
    z = torch.cat([X @ w[i:i + rows].double().t() for i in range(0, len(w), rows)], 1)
    lse = torch.logsumexp(z, 1)
    loss = lse - z.gather(1, t[:, None])[:, 0]
    d = torch.exp(z - lse[:, None])
    d.scatter_add_(1, t[:, None], torch.full_like(lse, -1.0)[:, None])
    d *= g.double()[:, None]
    return loss, lse, d


def test_a_weight_past_4_gib():
    tokens, vocab, hidden = 3, 600001, 4096
    gen = torch.Generator(device="cuda").manual_seed(1)
    w = torch.empty(vocab, hidden, dtype=torch.bfloat16, device="cuda")
    for i in range(0, vocab, 100000):
        w[i:i + 100000] = torch.randn(len(w[i:i + 100000]), hidden, generator=gen, device="cuda") * hidden ** -0.5
    x = torch.randn(tokens, hidden, generator=gen, device="cuda").bfloat16()
    t = torch.tensor([0, vocab - 1, 555555], device="cuda")
    g = torch.tensor([1.0, -2.0, 0.5], device="cuda")
    loss, lse = fm.linear_cross_entropy(x, w, t)
    dx, dw = fm.linear_cross_entropy_backward(x, w, t, lse, g)
    rl, rs, d = _reference(x, w, t, g)
    # logits: 4097 U32 sum |x w|, about 4097 * 2^-24 * 4096 * 0.8 * 0.0125 = 0.01 at
    # the very most; what random signs leave is 100 times less
    assert (lse.double() - rs).abs().max() < 1e-4 and (loss.double() - rl).abs().max() < 2e-4
    size = torch.zeros(tokens, hidden, dtype=torch.float64, device="cuda")
    ref = torch.zeros_like(size)
    for i in range(0, vocab, 65536):
        part = w[i:i + 65536].double()
        ref += d[:, i:i + 65536] @ part
        size += d[:, i:i + 65536].abs() @ part.abs()
    assert ((dx.double() - ref).abs() <= (UBF + 3e-4 + 600003 * U32) * size + UBF * ref.abs()).all()
    for i in (0, 262144, 524288, vocab - 1000):
        want = d[:, i:i + 1000].t() @ x.double()
        big = d[:, i:i + 1000].abs().t() @ x.double().abs()
        assert ((dw[i:i + 1000].double() - want).abs() <= (UBF + 3e-4) * big + UBF * want.abs() + 2.0 ** -126).all()


def test_hidden_states_past_4_gib():
    tokens, vocab, hidden = 530001, 300, 4096
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.empty(tokens, hidden, dtype=torch.bfloat16, device="cuda")
    for i in range(0, tokens, 100000):
        x[i:i + 100000] = torch.randn(len(x[i:i + 100000]), hidden, generator=gen, device="cuda")
    w = (torch.randn(vocab, hidden, generator=gen, device="cuda") * hidden ** -0.5).bfloat16()
    t = torch.randint(0, vocab, (tokens,), generator=gen, device="cuda")
    g = torch.randn(tokens, generator=gen, device="cuda")
    loss, lse = fm.linear_cross_entropy(x, w, t)
    dx, dw = fm.linear_cross_entropy_backward(x, w, t, lse, g)
    ref = torch.zeros(vocab, hidden, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(ref)
    for i in range(0, tokens, 50000):
        part = slice(i, i + 50000)
        rl, rs, d = _reference(x[part], w, t[part], g[part])
        assert (lse[part].double() - rs).abs().max() < 1e-4 and (loss[part].double() - rl).abs().max() < 2e-4
        ref += d.t() @ x[part].double()
        size += d.abs().t() @ x[part].double().abs()
        want = d @ w.double()
        big = d.abs() @ w.double().abs()
        assert ((dx[part].double() - want).abs() <= (UBF + 3e-4 + 302 * U32) * big + UBF * want.abs()).all()
    # fp32 sums of 530001 terms: a bound of 530003 U32 = 0.03 of the summed sizes;
    # the sums here are of about the square root of their terms
    assert ((dw.double() - ref).abs() <= (UBF + 3e-4 + 530003 * U32) * size + UBF * ref.abs()).all()
    assert ((dw.double() - ref).norm() / ref.norm()).item() < 0.01
