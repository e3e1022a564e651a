"""The mixture-of-experts layer with 4-bit weights against the float64 oracle."""
import numpy as np
import pytest
import torch

import fp8_scaled_matmul_amd as fm
from oracle import mx4

pytestmark = pytest.mark.gpu


def _experts(e, rows, cols, rng, std):
    """Random codes and scales of e matrices: (Mx4 on the GPU, float64 values)."""
    codes = rng.integers(0, 16, (e * rows, cols)).astype(np.uint8)
    mid = 127 + int(np.floor(np.log2(std / 3)))
    sb = rng.integers(mid - 2, mid + 2, (e * rows, -(-cols // 32))).astype(np.uint8)
    q, s = mx4.pack(codes, sb)
    s = np.ascontiguousarray(s.reshape(s.shape[0], e, rows, 16).transpose(1, 0, 2, 3))
    held = fm.Mx4(torch.from_numpy(q.reshape(e, rows, -1)).cuda(), torch.from_numpy(s).cuda(), cols)
    return held, mx4.values(codes, sb).reshape(e, rows, cols)


class Layer:
    def __init__(self, t, e, k, h, i, renormalize, seed=0, **kw):
        rng = np.random.default_rng([t, e, k, h, i, seed])
        self.rng, self.k, self.renormalize = rng, k, renormalize
        self.w1, self.v1 = _experts(e, 2 * i, h, rng, h ** -0.5)
        self.w2, self.v2 = _experts(e, h, i, rng, i ** -0.5)
        self.router = torch.from_numpy(rng.standard_normal((e, h)) * h ** -0.5).bfloat16()
        self.moe = fm.MoeMx4(self.router.cuda(), self.w1, self.w2, k, max_tokens=t, renormalize=renormalize, **kw)

    def x(self, t, h, scale=1.0):
        return torch.from_numpy(self.rng.standard_normal((t, h)) * scale).bfloat16()

    def check(self, x, got):
        """ids equal; weights within their fp32 roundings; y within what the
        roundings of the formula's steps add up to."""
        y, ids, weights = [v.cpu() for v in got]
        xv, rv = x.double().numpy(), self.router.double().numpy()
        want, wid, wp = mx4.moe(xv, rv, self.v1, self.v2, self.k, self.renormalize)
        assert np.array_equal(ids.numpy(), wid)
        e, h = rv.shape
        i = self.v2.shape[2]
        logits = xv @ rv.T
        z = np.abs(np.take_along_axis(logits, wid, 1) - logits.max(1, keepdims=True))
        # exponent argument, exp, the sum's additions and the quotient
        # (a weight below fp32's smallest number is 0)
        held = wp.astype(np.float32).astype(np.float64)
        assert (np.abs(weights.double().numpy() - held) <= (z + 16 + e) * 2.0 ** -24 * wp).all()
        blk = np.abs(np.pad(xv, ((0, 0), (0, -h % 32)))).reshape(len(xv), -1, 32).max(2).repeat(32, 1)[:, :h]
        bound = 2.0 ** -8 * np.abs(want) + 2.0 ** -134
        for t in range(len(xv)):
            for j in range(self.k):
                w1, w2 = self.v1[wid[t, j]], self.v2[wid[t, j]]
                gu = w1 @ xv[t]
                # fp32 sums of h terms (doubled for their order), x's small elements
                d = np.abs(w1) @ (2 * h * 2.0 ** -24 * np.abs(xv[t]) + 2.0 ** -21 * blk[t])
                g, u = gu[:i], gu[i:]
                with np.errstate(over="ignore"):
                    silu = g / (1 + np.exp(-g))
                a = wp[t, j] * silu * u
                # silu's slope is under 1.1; a dozen roundings besides
                da = wp[t, j] * (1.1 * d[:i] * np.abs(u) + (np.abs(silu) + 1.1 * d[:i]) * d[i:])
                da += (z[t, j] + 32 + e + np.abs(g)) * 2.0 ** -24 * np.abs(a)
                # a's pieces, and fp32 sums of k i terms
                ab = np.abs(np.pad(a, (0, -i % 32))).reshape(-1, 32).max(1).repeat(32)[:i]
                da += 2.0 ** -12 * np.abs(a) + 2.0 ** -25 * ab + 2 * self.k * i * 2.0 ** -24 * np.abs(a)
                bound[t] += np.abs(w2) @ da
        err = np.abs(y.double().numpy() - want)
        assert (err <= bound).all(), f"worst {np.max(err / bound):.3g} of the bound"


SIZES = [(1, 1, 1, 1, 1), (1, 4, 1, 32, 32), (1, 64, 8, 256, 100), (2, 37, 3, 1000, 531), (3, 5, 5, 70, 33),
         (7, 37, 3, 264, 65), (16, 8, 2, 520, 64), (17, 8, 2, 256, 257), (33, 20, 1, 96, 40), (64, 16, 4, 512, 300),
         (64, 4, 4, 300, 128), (40, 130, 16, 264, 96), (5, 512, 10, 128, 64), (64, 100, 8, 64, 32)]


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("t,e,k,h,i", SIZES)
def test_moe(t, e, k, h, i, renormalize):
    m = Layer(t, e, k, h, i, renormalize)
    x = m.x(t, h)
    got = m.moe(x.cuda())
    m.check(x, got)
    # the same bits again, and fewer tokens through the same layer
    assert all(torch.equal(a, b) for a, b in zip(got, m.moe(x.cuda())))
    few = x[: t // 2 + 1]
    m.check(few, m.moe(few.cuda()))
    m.check(x, m.moe(x.cuda()))


@pytest.mark.parametrize("h", [2, 7, 9, 11, 39, 46, 61, 516, 525, 1031])
def test_moe_row_ends(h):
    """Rows of x and router that end anywhere in a read of eight, and rows
    shorter than one, their elements after other rows' (NaN there)."""
    m = Layer(20, 18, 3, h, 40, True)
    x = m.x(20, h)
    m.check(x, m.moe(x.cuda()))
    wide = torch.full((20, h + 3), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 1:-2] = x.cuda()
    m.check(x, m.moe(wide[:, 1:-2]))


def test_moe_every_token_to_one_expert():
    """64 tokens reach the same experts: four columns tiles of 16, and the
    other experts none."""
    m = Layer(64, 9, 2, 320, 96, True)
    m.router[:] = 0
    m.router[3] = 1
    m.router[7] = 0.5
    m.moe.router.copy_(m.router)
    x = m.x(64, 320).abs()
    got = m.moe(x.cuda())
    assert (got[1].cpu() == torch.tensor([3, 7])).all()
    m.check(x, got)


def test_moe_ties_go_to_the_lower_expert():
    m = Layer(4, 150, 6, 64, 32, True)
    m.router[:] = m.router[:1]
    m.router[100:] *= 2
    m.moe.router.copy_(m.router)
    x = m.x(4, 64)
    got = m.moe(x.cuda())
    m.check(x, got)
    up = (x.double() @ m.router[0].double()) > 0
    assert torch.equal(got[1].cpu()[:, 0], torch.where(up, 100, 0).int())
    x[:] = 0                    # every logit 0
    got = m.moe(x.cuda())
    assert (got[1].cpu() == torch.arange(6)).all() and (got[0] == 0).all()
    m.check(x, got)


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e4, 1e15])
def test_moe_far_ranges(scale):
    """Blocks at both ends of the range; outliers beside small elements."""
    m = Layer(6, 12, 3, 300, 70, True)
    x = m.x(6, 300, 1.0)
    x[:, ::50] *= 1000
    x[:, 1::50] *= 1e-6
    m.router /= 64
    m.moe.router.copy_(m.router)
    if scale > 1:
        m.router /= scale
        m.moe.router.copy_(m.router)
    x = (x.float() * scale).bfloat16()
    m.check(x, m.moe(x.cuda()))


def test_moe_nonfinite_rows():
    """A token that holds an Inf or NaN is NaN throughout, valid ids all the
    same; the other tokens are as without it, and the outputs are counted."""
    ctr = fm.Counters()
    m = Layer(20, 30, 4, 200, 96, True, counters=ctr)
    x = m.x(20, 200)
    want = [v.clone() for v in m.moe(x.cuda())]
    assert ctr.read()["nonfinite_out"] == 0
    bad = x.clone()
    bad[3, 17] = float("nan")
    bad[11, 199] = float("inf")
    y, ids, weights = m.moe(bad.cuda())
    ok = [t for t in range(20) if t not in (3, 11)]
    assert torch.isnan(y[[3, 11]]).all() and ctr.read()["nonfinite_out"] == 400
    assert torch.equal(y[ok], want[0][ok]) and torch.equal(ids[ok], want[1][ok])
    assert ((ids >= 0) & (ids < 30)).all() and all(len(set(r.tolist())) == 4 for r in ids)
    # a NaN block of one expert reaches the tokens that chose it, in its row alone
    e, row = int(ids[0, 0]), 5
    m.w2.s[e, 0, row, 1] = 255
    y2, ids2, _ = m.moe(x.cuda())
    hit = (want[1] == e).any(1)
    nan = torch.isnan(y2)
    assert torch.equal(nan[:, row], hit) and int(nan.sum()) == int(hit.sum())


def test_moe_strides_and_outputs_given():
    m = Layer(9, 20, 3, 200, 96, False)
    x = m.x(9, 200)
    want = m.moe(x.cuda())
    for pitch in (203, 208):
        wide = torch.zeros(9, pitch, dtype=torch.bfloat16, device="cuda")
        wide[:, :200] = x.cuda()
        buf = torch.full((9, pitch), 7.0, dtype=torch.bfloat16, device="cuda")
        got = m.moe(wide[:, :200], out=buf[:, :200])
        assert torch.equal(buf[:, :200], want[0]) and (buf[:, 200:] == 7).all()
        assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    # experts of a larger stack (a shard), rows of codes further apart
    q1 = torch.zeros(22, 192, 144, dtype=torch.uint8, device="cuda")
    q1[1:21, :, :128] = m.w1.q
    s1 = torch.zeros(22, 1, 200, 16, dtype=torch.uint8, device="cuda")
    s1[1:21, :, :192] = m.w1.s
    w1 = fm.Mx4(q1[1:21, :, :128], s1[1:21, :, :192], 200)
    got = fm.MoeMx4(m.router.cuda(), w1, m.w2, 3, max_tokens=9, renormalize=False)(x.cuda())
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    y, ids, weights = m.moe(x[:0].cuda())
    assert y.shape == (0, 200) and ids.shape == (0, 3) and weights.shape == (0, 3)


def test_moe_on_another_stream_and_captured():
    m = Layer(12, 40, 4, 256, 128, True)
    x = m.x(12, 256).cuda()
    want = [v.clone() for v in m.moe(x)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = m.moe(x)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = m.moe(x)
    for i in range(4):
        x.copy_(m.x(12, 256))
        want = [v.clone() for v in m.moe(x)]
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_moe_is_what_quantize_and_product_give():
    """The layer on weights that the library quantized, against the library's
    own products, expert by expert, on activations that 4 bits hold exactly."""
    t, e, h, i = 4, 3, 128, 64
    rng = np.random.default_rng(1)
    w1 = torch.from_numpy(rng.standard_normal((e, 2 * i, h))).bfloat16().cuda()
    w2 = torch.from_numpy(rng.standard_normal((e, h, i))).bfloat16().cuda()
    h1 = [fm.mx4_quantize(w)[0] for w in w1]
    h2 = [fm.mx4_quantize(w)[0] for w in w2]
    stack = lambda a, c: fm.Mx4(torch.stack([v.q for v in a]), torch.stack([v.s for v in a]), c)    # noqa: E731
    x = torch.from_numpy(mx4.VALUES[rng.integers(0, 16, (t, h))]).bfloat16().cuda()
    x[:, ::32] = 6
    router = torch.from_numpy(rng.standard_normal((e, h)) / 16).bfloat16().cuda()
    y, ids, weights = fm.MoeMx4(router, stack(h1, h), stack(h2, i), 1)(x)
    xq, _ = fm.mx4_quantize(x)
    for tok in range(t):
        gu = fm.mx4_mm(xq, h1[ids[tok, 0]]).float()[tok]
        a = torch.nn.functional.silu(gu[:i]) * gu[i:] * weights[tok, 0]
        want = fm.mx4_dequantize(h2[ids[tok, 0]], torch.float32) @ a
        size = fm.mx4_dequantize(h2[ids[tok, 0]], torch.float32).abs() @ a.abs()
        # gate and up rounded to bf16 (silu's relative slope is at most 1 + |g|), y too, a to 2^-12
        slope = 2 + gu[:i].abs().max()
        assert ((y[tok].float() - want).abs() <= 2.0 ** -8 * (want.abs() + slope * size) + 2.0 ** -12 * size).all()


def test_moe_inner_activations_keep_their_precision():
    """Outputs that are differences of nearly equal inner activations show the
    precision those are held to: fp32."""
    t, h, i = 3, 256, 64
    rng = np.random.default_rng(19)

    def held(codes):        # every scale 1
        q, s = mx4.pack(codes, np.full((codes.shape[0], -(-codes.shape[1] // 32)), 127, np.uint8))
        return fm.Mx4(torch.from_numpy(q[None]).cuda(), torch.from_numpy(s[None]).cuda(), codes.shape[1])

    # g = x[0]; u = x[0] + a little that differs, of blocks of its own: both exact in fp32
    c1 = np.zeros((2 * i, h), np.uint8)
    c1[:, 0] = 2
    c1[i:, 32] = rng.integers(0, 16, i)
    c1[i:, 64] = rng.integers(0, 16, i)
    c2 = np.zeros((h, i), np.uint8)
    for r in range(h):
        c2[r, rng.choice(i, 2, replace=False)] = 2, 10      # 1, -1
    x = np.zeros((t, h))
    x[:, 0] = 1.75, 3.125, 0.8125
    x[:, 32] = 1.25 * 2.0 ** -12
    x[:, 64] = 1.625 * 2.0 ** -14
    layer = fm.MoeMx4(torch.ones(1, h, dtype=torch.bfloat16, device="cuda"), held(c1), held(c2), 1, max_tokens=t)
    y = layer(torch.from_numpy(x).bfloat16().cuda())[0].cpu().double().numpy()
    gu = x @ mx4.VALUES[c1].T
    a = gu[:, :i] / (1 + np.exp(-gu[:, :i])) * gu[:, i:]
    # exp, sum, quotient and two products in fp32 (four units in the last place for exp and quotient)
    da = 12 * 2.0 ** -23 * np.abs(a)
    w2 = mx4.VALUES[c2]
    want = a @ w2.T
    bound = 2.0 ** -8 * np.abs(want) + da @ np.abs(w2).T + 2.0 ** -24 * np.abs(a) @ np.abs(w2).T
    assert (np.abs(y - want) <= bound).all(), np.max(np.abs(y - want) / bound)


def test_moe_sums_of_far_apart_terms_keep_their_precision():
    """A sum's terms of very different size beside each other: what the small
    ones add up to shows once the large ones cancel.  Both layers, bounds of
    fp32 sums."""
    t, h, i = 16, 512, 512
    rng = np.random.default_rng(23)

    def held(codes):
        q, s = mx4.pack(codes, np.full((codes.shape[0], -(-codes.shape[1] // 32)), 127, np.uint8))
        return fm.Mx4(torch.from_numpy(q[None]).cuda(), torch.from_numpy(s[None]).cuda(), codes.shape[1])

    # every fourth element of x is large, in pairs that the weights 1 and -1 cancel exactly
    x = rng.standard_normal((t, h))
    x[:, ::8] = 192.0 * (1 + rng.integers(0, 4, (t, h // 8)))
    x[:, 4::8] = x[:, ::8]
    c1 = rng.integers(0, 16, (2 * i, h)).astype(np.uint8)
    c1[:, ::8], c1[:, 4::8] = 2, 10
    xb = torch.from_numpy(x).bfloat16()
    xv = xb.double().numpy()
    c2 = rng.integers(0, 16, (h, i)).astype(np.uint8)
    layer = fm.MoeMx4(torch.ones(1, h, dtype=torch.bfloat16, device="cuda"), held(c1), held(c2), 1, max_tokens=t)
    y = layer(xb.cuda())[0].cpu().double().numpy()
    w1, w2 = mx4.VALUES[c1], mx4.VALUES[c2]
    gu, size = xv @ w1.T, np.abs(xv) @ np.abs(w1).T
    # an instruction's sum of 32 products is off by 2^-22 of their sizes at most (measured), 16 of them and three more
    # sums of waves by 2^-24 of the sizes so far each
    d = (2.0 ** -22 + 19 * 2.0 ** -24) * size
    g, u, dg, du = gu[:, :i], gu[:, i:], d[:, :i], d[:, i:]
    silu = g / (1 + np.exp(-g))
    a = silu * u
    da = 1.1 * dg * np.abs(u) + (np.abs(silu) + 1.1 * dg) * du + (12 + np.abs(g)) * 2.0 ** -23 * np.abs(a)
    want, ysize = a @ w2.T, np.abs(a) @ np.abs(w2).T
    # the rounding of y, its sums; the errors of a are independent, so that five deviations of their sum bound it
    bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -22 + 40 * 2.0 ** -24) * ysize + 5 * np.sqrt((da ** 2) @ (w2 ** 2).T)
    assert (np.abs(y - want) <= bound).all(), np.max(np.abs(y - want) / bound)


@pytest.mark.parametrize("most,t,e,k,h,i", [(9, 8, 512, 1, 520, 64), (11, 10, 400, 2, 600, 512)])
def test_moe_fewer_tokens_through_a_layer_for_more(most, t, e, k, h, i):
    """Where fewer tokens take more splits of the router's sums."""
    m = Layer(most, e, k, h, i, True)
    for n in (t, most):
        x = m.x(n, h)
        m.check(x, m.moe(x.cuda()))


def test_moe_a_single_row_may_have_any_row_stride():
    m = Layer(1, 1, 1, 200, 96, True)
    x = m.x(1, 200).cuda()
    want = [v.clone() for v in m.moe(x)]
    column = x.reshape(200, 1).clone().t()
    assert column.stride() == (1, 1)
    m.moe.router = m.router.cuda().reshape(200, 1).t()
    m.moe = fm.MoeMx4(m.moe.router, m.w1, m.w2, 1, max_tokens=1)
    out = torch.zeros(200, 1, dtype=torch.bfloat16, device="cuda").t()
    for got in (m.moe(column), m.moe(column, out=out)):
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_moe_built_on_a_busy_stream_and_called_on_another():
    """The layer's workspace is ready when it has been built, whatever its
    stream still had to do."""
    m = Layer(5, 12, 3, 256, 96, True)
    x = m.x(5, 256).cuda()
    router = m.router.cuda()
    want = [v.clone() for v in m.moe(x)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    # memory that is not zero, for the allocator to hand out again
    torch.full((m.moe._ws.numel(),), 0x5A, dtype=torch.uint8, device="cuda")
    torch.cuda._sleep(20_000_000)
    layer = fm.MoeMx4(router, m.w1, m.w2, 3, max_tokens=5)
    with torch.cuda.stream(side):
        got = layer(x)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("t,e,k,h,i", [(16, 512, 4, 2100, 16), (64, 128, 8, 4096, 16), (1, 300, 5, 4100, 16),
                                       (5, 512, 3, 1600, 16), (3, 200, 2, 9000, 8)])
def test_moe_router_takes_several_rounds(t, e, k, h, i):
    """Long rows and many experts: one split and three rounds of reads with a
    ragged end, two reads a round, eight splits, sums of several splits for
    every number of experts a lane."""
    m = Layer(t, e, k, h, i, False)
    x = m.x(t, h)
    m.check(x, m.moe(x.cuda()))


def test_moe_other_tokens_change_a_token_within_its_bound_alone():
    """Without the tokens that hold an Inf or NaN the others choose the same
    experts with the same weights; their sums may take another order."""
    m = Layer(20, 30, 4, 200, 96, True, seed=3)
    x = m.x(20, 200)
    bad = x.clone()
    bad[3, 17] = float("nan")
    bad[11, 199] = float("inf")
    got = m.moe(bad.cuda())
    ok = [t for t in range(20) if t not in (3, 11)]
    m.check(x[ok], [v[ok] for v in got])
    want = m.moe(x.cuda())
    assert torch.equal(got[1][ok], want[1][ok]) and torch.equal(got[2][ok], want[2][ok])


def test_moe_counts_only_the_outputs_there_are():
    """Rows and tokens that fill no tile, with counts asked for, in either of
    the second layer's forms."""
    for t, e, k, h, i in ((3, 5, 2, 70, 33), (64, 8, 4, 2050, 1100)):
        ctr = fm.Counters()
        m = Layer(t, e, k, h, i, True, counters=ctr)
        x = m.x(t, h)
        y, ids, _ = m.moe(x.cuda())
        assert torch.isfinite(y).all() and ctr.read()["nonfinite_out"] == 0
        m.w2.s[int(ids[0, 0]), 0, h - 1, 0] = 255
        y, ids2, _ = m.moe(x.cuda())
        hit = (ids2 == ids[0, 0]).any(1)
        assert torch.equal(torch.isnan(y)[:, h - 1], hit) and torch.isnan(y).sum() == hit.sum()
        assert ctr.read()["nonfinite_out"] == int(hit.sum())
