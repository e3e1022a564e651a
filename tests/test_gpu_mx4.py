"""The 4-bit quantizer, dequantizer and product against the float64 oracle."""
import numpy as np
import pytest
import torch

import fp8_scaled_matmul_amd as fm
from oracle import mx4

pytestmark = pytest.mark.gpu


def _x(rows, cols, dtype=torch.bfloat16, seed=0, spread=True):
    g = torch.Generator().manual_seed(seed + 1000003 * rows + cols)
    x = torch.randn(rows, cols, generator=g)
    if spread:      # blocks of very different size
        x *= torch.exp2(torch.randint(-30, 30, (rows, cols // 16 + 1), generator=g).float()).repeat_interleave(16, 1)[:, :cols]
    return x.to(dtype)


def _f64(t):
    return t.detach().cpu().double().numpy()


def _check_quantize(x, seed=None, want_t=True, ld=None):
    """Codes, scale bytes, padding and counters equal the oracle's."""
    rows, cols = x.shape
    dev = x.cuda()
    if ld:
        dev = torch.zeros(rows, ld, dtype=x.dtype, device="cuda")[:, :cols].copy_(x)
    sd = None if seed is None else torch.tensor([seed], dtype=torch.int64, device="cuda")
    ctr = fm.Counters()
    q, qt = fm.mx4_quantize(dev, want_t=want_t, seed=sd, counters=ctr)
    bits = None if seed is None else mx4.random_bits(rows, cols, seed)
    codes, sb, want = mx4.quantize(_f64(x), bits)
    eq, es = mx4.pack(codes, sb)
    assert np.array_equal(q.s.cpu().numpy(), es), "scale bytes"
    assert np.array_equal(q.q.cpu().numpy(), eq), "codes"
    got = ctr.read()
    assert all(got[f] == want[f] for f in ("saturated", "underflow", "nan")), (got, want)
    if want_t:
        codes, sb, _ = mx4.quantize(_f64(x).T, None if bits is None else bits.T)
        eq, es = mx4.pack(codes, sb)
        assert np.array_equal(qt.s.cpu().numpy(), es), "transposed scale bytes"
        assert np.array_equal(qt.q.cpu().numpy(), eq), "transposed codes"
    # without counters: the same codes
    q2, _ = fm.mx4_quantize(dev, want_t=want_t, seed=sd)
    assert torch.equal(q.q, q2.q) and torch.equal(q.s, q2.s)


SHAPES = [(1, 1), (1, 32), (3, 33), (1, 4096), (31, 31), (33, 255), (257, 256), (70, 513), (512, 512), (100, 1030),
          (513, 136)]


@pytest.mark.parametrize("seed", [None, 0x123456789ABCDEF])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize(rows, cols, dtype, seed):
    _check_quantize(_x(rows, cols, dtype), seed, want_t=True)
    _check_quantize(_x(rows, cols, dtype, 1), seed, want_t=False)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_strided_rows(dtype):
    _check_quantize(_x(40, 96, dtype), ld=104)
    _check_quantize(_x(40, 95, dtype), 7, ld=101)


@pytest.mark.parametrize("seed", [None, 99])
@pytest.mark.parametrize("want_t", [False, True])
def test_quantize_every_bf16_pattern(want_t, seed):
    """All 65536 bf16 values, Inf and NaN and subnormals among them: sorted by
    pattern (blocks of one magnitude) and mixed (blocks of every magnitude)."""
    b = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    _check_quantize(b.reshape(128, 512), seed, want_t)
    _check_quantize(b.reshape(512, 128).t().contiguous(), seed, want_t)


@pytest.mark.parametrize("want_t", [False, True])
def test_quantize_fp32_extremes(want_t):
    """Subnormals, the largest values, signed zeros, Inf and NaN in fp32, and
    amax on both sides of the step between two scales."""
    rng = np.random.default_rng(5)
    bits = rng.integers(0, 1 << 32, (64, 96), dtype=np.uint64).astype(np.uint32)
    bits[:16] &= 0x807FFFFF                       # subnormals
    bits[16:24] = 0x7F7FFFFF                      # the largest
    bits[24:28] = 0x80000000                      # -0
    bits[28] = 0x7F800000                         # only Inf
    x = torch.from_numpy(bits.view(np.float32).copy())
    x[32:36] = 0.1
    for i, v in enumerate((6.0, np.nextafter(np.float32(6.0), np.float32(7.0)), 1.5, 1.5000001)):
        x[32 + i, ::32] = float(v)
    for seed in (None, 5):
        _check_quantize(x, seed, want_t)


def test_quantize_empty_and_outputs_given():
    for shape in [(0, 64), (5, 0)]:
        q, qt = fm.mx4_quantize(torch.empty(shape, dtype=torch.bfloat16, device="cuda"), want_t=True)
        assert q.shape == shape and qt.shape == shape[::-1]
        assert fm.mx4_dequantize(q).shape == shape
    x = _x(64, 300).cuda()
    # rows of codes and scale panels further apart, what lies between untouched
    qb = torch.full((64, 384), 0x5A, dtype=torch.uint8, device="cuda")
    sb = torch.full((1, 80, 16), 0x5A, dtype=torch.uint8, device="cuda")
    out = fm.Mx4(qb[:, :256], sb[:, :64], 300)
    got, _ = fm.mx4_quantize(x, out=out)
    want, _ = fm.mx4_quantize(x)
    assert got is out and torch.equal(out.q, want.q) and torch.equal(out.s, want.s)
    assert (qb[:, 256:] == 0x5A).all() and (sb[:, 64:] == 0x5A).all()
    assert torch.equal(fm.mx4_dequantize(out, torch.float32), fm.mx4_dequantize(want, torch.float32))


def test_quantize_seed_is_read_on_the_device():
    """The same call draws anew when the seed tensor changes; equal seeds give
    equal codes; the mean over seeds approaches the value."""
    x = torch.full((64, 64), 0.3, dtype=torch.float32, device="cuda")
    x[:, ::32] = 6.0
    x[::32] = 6.0
    seed = torch.tensor([1], dtype=torch.int64, device="cuda")
    a = fm.mx4_quantize(x, seed=seed)[0].q.clone()
    assert torch.equal(a, fm.mx4_quantize(x, seed=seed)[0].q)
    mean = torch.zeros_like(x)
    for i in range(64):
        seed.fill_(1000 + i)
        mean += fm.mx4_dequantize(fm.mx4_quantize(x, seed=seed)[0], torch.float32) / 64
    assert not torch.equal(a, fm.mx4_quantize(x, seed=seed)[0].q)
    inner = mean[x == 0.3 * torch.ones_like(x)]
    # 0.3 = 0.5 * 0.6: std of the mean of n * 64 draws is 0.5 sqrt(0.24 / (64 n))
    n = inner.numel() * 64
    assert abs(inner.mean().item() - 0.3) < 5 * 0.5 * (0.24 / n) ** 0.5


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_dequantize_every_code_and_scale(dtype):
    sb = np.arange(256, dtype=np.uint8)[:, None]
    codes = np.tile(np.arange(16, dtype=np.uint8), 2)[None, :].repeat(256, 0)
    q, s = mx4.pack(codes, sb)
    a = fm.Mx4(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), 32)
    got = _f64(fm.mx4_dequantize(a, dtype))
    with np.errstate(over="ignore"):
        want = mx4.values(codes, sb)
        want = want.astype(np.float32).astype(np.float64)       # past the range: Inf
    assert np.array_equal(got, want, equal_nan=True)
    assert np.array_equal(np.signbit(got[1:255]), np.signbit(want[1:255]))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (5, 33), (7, 520), (6, 1032)])
def test_dequantize_ragged(rows, cols, dtype):
    rng = np.random.default_rng(rows * cols)
    codes = rng.integers(0, 16, (rows, cols)).astype(np.uint8)
    sb = rng.integers(100, 150, (rows, -(-cols // 32))).astype(np.uint8)
    q, s = mx4.pack(codes, sb)
    a = fm.Mx4(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), cols)
    buf = torch.full((rows, cols + 3), 7.0, dtype=dtype, device="cuda")
    fm.mx4_dequantize(a, out=buf[:, :cols])
    assert np.array_equal(_f64(buf[:, :cols]), mx4.values(codes, sb)) and (buf[:, cols:] == 7).all()
    assert np.array_equal(_f64(fm.mx4_dequantize(a, dtype)), mx4.values(codes, sb))


# ------------------------------------------------------------------ product
def _operand(rows, k, seed, lo=110, hi=140):
    """Random codes and scales: (Mx4 on the GPU, float64 values)."""
    rng = np.random.default_rng([rows, k, seed])
    codes = rng.integers(0, 16, (rows, k)).astype(np.uint8)
    sb = rng.integers(lo, hi, (rows, -(-k // 32))).astype(np.uint8)
    q, s = mx4.pack(codes, sb)
    return fm.Mx4(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), k), mx4.values(codes, sb)


def _check_mm(y, va, vb):
    """One rounding to bf16 (2^-8 of the value, 2^-134 where it is subnormal)
    and k additions in fp32 (2^-24 of what is summed each, doubled for the
    order)."""
    ref, size = mx4.mm(va, vb)
    bound = 2.0 ** -8 * np.abs(ref) + 2 * va.shape[1] * 2.0 ** -24 * size + 2.0 ** -134
    err = np.abs(_f64(y) - ref)
    assert (err <= bound).all(), f"worst {np.max(err / bound):.3g} of the bound"


MM = [(1, 1, 1), (1, 8, 32), (1, 300, 513), (2, 64, 256), (5, 1000, 4096), (16, 100, 70), (17, 33, 700),
      (32, 4096, 512), (33, 65, 1025), (64, 64, 512), (65, 129, 96), (100, 70, 3100), (128, 128, 256),
      (200, 513, 1100), (257, 255, 800), (333, 1000, 1568), (700, 700, 512), (4, 4, 20000), (130, 70, 9000)]


@pytest.mark.parametrize("m,n,k", MM)
def test_mm(m, n, k):
    a, va = _operand(m, k, 0)
    b, vb = _operand(n, k, 1)
    y = fm.mx4_mm(a, b)
    _check_mm(y, va, vb)
    # the same bits again
    assert torch.equal(y, fm.mx4_mm(a, b))
    # strided output of odd pitch: nothing past its columns is written
    buf = torch.full((m, n + 3), 7.0, dtype=torch.bfloat16, device="cuda")
    fm.mx4_mm(a, b, out=buf[:, :n])
    assert torch.equal(buf[:, :n], y) and (buf[:, n:] == 7).all()


@pytest.mark.parametrize("m,n,k", [(512, 768, 2048), (1024, 1024, 1000), (2048, 4096, 512), (4100, 2050, 300)])
def test_mm_large(m, n, k):
    a, va = _operand(m, k, 2)
    b, vb = _operand(n, k, 3)
    _check_mm(fm.mx4_mm(a, b), va, vb)


@pytest.mark.parametrize("m,n,k", [(3400, 4100, 700), (4097, 3585, 1024), (6000, 2100, 130), (4096, 4096, 1300)])
def test_mm_many_tiles(m, n, k):
    """Enough output for the largest tiles: ragged edges, one to five panels
    of scales, an odd pitch."""
    a, va = _operand(m, k, 8)
    b, vb = _operand(n, k, 9)
    y = fm.mx4_mm(a, b)
    _check_mm(y, va, vb)
    buf = torch.full((m, n + 1), 7.0, dtype=torch.bfloat16, device="cuda")
    fm.mx4_mm(a, b, out=buf[:, :n])
    assert torch.equal(buf[:, :n], y) and (buf[:, n:] == 7).all()


@pytest.mark.parametrize("m,n,k", [(1900, 2000, 700), (1536, 2048, 256), (2000, 1600, 31), (3000, 2600, 1300),
                                   (2900, 1537, 256)])
def test_mm_some_tiles(m, n, k):
    """About one and two middle-sized tiles a CU: fewer steps than the ring
    has stages, ragged edges, an odd pitch."""
    a, va = _operand(m, k, 10)
    b, vb = _operand(n, k, 11)
    y = fm.mx4_mm(a, b)
    _check_mm(y, va, vb)
    buf = torch.full((m, n + 1), 7.0, dtype=torch.bfloat16, device="cuda")
    fm.mx4_mm(a, b, out=buf[:, :n])
    assert torch.equal(buf[:, :n], y) and (buf[:, n:] == 7).all()


@pytest.mark.parametrize("m,n,k", [(12, 16000, 300), (9, 12345, 96), (3000, 50, 800), (2000, 300, 1000), (500, 300, 1040),
                                   (100, 700, 9000), (1500, 1500, 256), (16, 64, 33), (1300, 1300, 511)])
def test_mm_every_shape_of_tile(m, n, k):
    """Few rows or columns, long and short K: the tiles that such products take."""
    a, va = _operand(m, k, 12)
    b, vb = _operand(n, k, 13)
    y = fm.mx4_mm(a, b)
    _check_mm(y, va, vb)
    buf = torch.full((m, n + 1), 7.0, dtype=torch.bfloat16, device="cuda")
    fm.mx4_mm(a, b, out=buf[:, :n])
    assert torch.equal(buf[:, :n], y) and (buf[:, n:] == 7).all()


@pytest.mark.parametrize("m", [1, 40, 300])
def test_mm_scales_at_their_ends(m):
    """Scale bytes over the whole range, each product within bf16's range."""
    k, n = 544, 96
    rng = np.random.default_rng(m)
    for lo, hi in ((0, 30), (230, 254)):
        codes = rng.integers(0, 16, (m, k)).astype(np.uint8)
        sb = rng.integers(lo, hi, (m, 17)).astype(np.uint8)
        q, s = mx4.pack(codes, sb)
        a = fm.Mx4(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), k)
        b, vb = _operand(n, k, m, *((214, 224) if lo == 0 else (100, 110)))
        _check_mm(fm.mx4_mm(a, b), mx4.values(codes, sb), vb)


@pytest.mark.parametrize("m,n", [(1, 70), (33, 40), (150, 300), (600, 520)])
def test_mm_nan_scale_and_overflow(m, n):
    """A NaN block makes its whole row (or column) NaN, and outputs past
    bf16's range are Inf; both are counted, and nothing else is."""
    k = 640
    a, va = _operand(m, k, 4)
    b, vb = _operand(n, k, 5)
    a.s[0, m // 2, 3] = 255
    b.s[1, n - 1, 1] = 255
    ctr = fm.Counters()
    y = _f64(fm.mx4_mm(a, b, counters=ctr))
    nan = np.zeros((m, n), bool)
    nan[m // 2] = True
    nan[:, n - 1] = True
    assert np.array_equal(np.isnan(y), nan) and ctr.read()["nonfinite_out"] == nan.sum()
    one = torch.full((m, k), 4.0, device="cuda", dtype=torch.bfloat16)
    big, _ = fm.mx4_quantize(one * 2.0 ** 100)
    w, _ = fm.mx4_quantize(torch.full((n, k), 2.0 ** 100, device="cuda", dtype=torch.bfloat16))
    ctr = fm.Counters()
    y = fm.mx4_mm(big, w, counters=ctr)
    assert torch.isinf(y).all() and ctr.read()["nonfinite_out"] == m * n


def test_mm_k_zero_and_empty():
    e = fm.mx4_mm(fm.Mx4.empty(3, 0), fm.Mx4.empty(5, 0))
    assert e.shape == (3, 5) and (e == 0).all()
    assert fm.mx4_mm(fm.Mx4.empty(0, 64), fm.Mx4.empty(5, 64)).shape == (0, 5)
    assert fm.mx4_mm(fm.Mx4.empty(3, 64), fm.Mx4.empty(0, 64)).shape == (3, 0)


def test_mm_views_of_larger_operands():
    """Rows of a larger operand (a shard): codes with a row distance and scale
    panels further apart than their rows."""
    a, va = _operand(64, 1200, 6)
    b, vb = _operand(300, 1200, 7)
    wide = torch.zeros(300, 720, dtype=torch.uint8, device="cuda")
    wide[:, :640] = b.q
    shard = fm.Mx4(wide[100:250, :640], b.s[:, 100:250], 1200)
    _check_mm(fm.mx4_mm(a, shard), va, vb[100:250])
    _check_mm(fm.mx4_mm(shard, a), vb[100:250], va)


def test_on_another_stream():
    x = _x(300, 700).cuda()
    w = _x(200, 700, seed=9).cuda()
    torch.cuda.synchronize()
    want = fm.mx4_mm(fm.mx4_quantize(x)[0], fm.mx4_quantize(w)[0])
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        got = fm.mx4_mm(fm.mx4_quantize(x)[0], fm.mx4_quantize(w)[0])
    st.synchronize()
    assert torch.equal(got, want)


def test_graph_replays_follow_inputs_and_seed():
    """A training step's quantizations and products in a captured graph: every
    replay equals the eager step on the inputs and the seed of that moment."""
    x, dy = _x(256, 512, spread=False).cuda(), _x(256, 384, seed=1, spread=False).cuda()
    w, wt = fm.mx4_quantize(_x(384, 512, seed=2, spread=False).cuda(), want_t=True)
    seed = torch.tensor([5], dtype=torch.int64, device="cuda")

    def step():
        xq, xqt = fm.mx4_quantize(x, want_t=True)
        dq, dqt = fm.mx4_quantize(dy, want_t=True, seed=seed)
        return fm.mx4_mm(xq, w), fm.mx4_mm(dq, wt), fm.mx4_mm(dqt, xqt)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for i in range(4):
        x.copy_(_x(256, 512, seed=20 + i, spread=False))
        dy.copy_(_x(256, 384, seed=40 + i, spread=False))
        seed.fill_(i)
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_linear_gradients_against_formula_and_differences():
    """dX = dY W and dW = dY^T X on operands that 4 bits hold exactly, against
    float64 and against central differences of sum(dY * (X W^T)), which is
    linear in each entry, so that a difference is exact but for roundings."""
    rng = np.random.default_rng(3)
    m, n, k = 64, 96, 160

    def grid(r, c):     # every block (of rows and of columns) holds a 6: scale 1
        v = mx4.VALUES[rng.integers(0, 16, (r, c))]
        v[:, ::32] = 6.0
        v[::32] = 6.0
        return v

    x, w, dy = grid(m, k), grid(n, k), grid(m, n)
    dev = lambda v: torch.from_numpy(v).bfloat16().cuda()   # noqa: E731
    xq, xqt = fm.mx4_quantize(dev(x), want_t=True)
    _, wqt = fm.mx4_quantize(dev(w), want_t=True)
    dq, dqt = fm.mx4_quantize(dev(dy), want_t=True)
    dx, dw = _f64(fm.mx4_mm(dq, wqt)), _f64(fm.mx4_mm(dqt, xqt))
    # sums of products of multiples of 0.25 below 2^22 are exact in fp32: one rounding
    assert (np.abs(dx - dy @ w) <= 2.0 ** -8 * np.abs(dy @ w)).all()
    assert (np.abs(dw - dy.T @ x) <= 2.0 ** -8 * np.abs(dy.T @ x)).all()
    for r, c in [(0, 0), (5, 7), (63, 95)]:
        step = np.zeros_like(w)
        step[c, 3] = 1.0
        d = ((dy * (x @ (w + step).T)).sum() - (dy * (x @ (w - step).T)).sum()) / 2
        assert abs(dw[c, 3] - d) <= 2.0 ** -8 * abs(d) + 1e-6
        step = np.zeros_like(x)
        step[r, 3] = 1.0
        d = ((dy * ((x + step) @ w.T)).sum() - (dy * ((x - step) @ w.T)).sum()) / 2
        assert abs(dx[r, 3] - d) <= 2.0 ** -8 * abs(d) + 1e-6


def test_same_results_with_and_without_outputs_given():
    """The calls that the extension module takes whole and those the Python
    code takes give the same, parameters that require gradients among them."""
    x = torch.nn.Parameter(_x(100, 300).cuda())
    seed = torch.tensor([3], dtype=torch.int64, device="cuda")
    for sd in (None, seed):
        q, qt = fm.mx4_quantize(x, want_t=True, seed=sd)
        o, ot = fm.mx4_quantize(x, want_t=True, seed=sd, out=fm.Mx4.empty(100, 300), out_t=fm.Mx4.empty(300, 100))
        assert all(torch.equal(a, b) for a, b in ((q.q, o.q), (q.s, o.s), (qt.q, ot.q), (qt.s, ot.s)))
        assert fm.mx4_quantize(x, seed=sd)[1] is None and not q.q.requires_grad
    for dtype in (torch.bfloat16, torch.float32):
        y = torch.empty(100, 300, dtype=dtype, device="cuda")
        assert torch.equal(fm.mx4_dequantize(q, dtype), fm.mx4_dequantize(q, out=y))
    y = torch.empty(100, 100, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(fm.mx4_mm(q, q), fm.mx4_mm(q, q, out=y))


@pytest.mark.parametrize("m,n,k", [(1500, 1500, 512), (1300, 1202, 40), (3000, 3000, 512), (2998, 3002, 300),
                                   (3001, 2999, 512)])
def test_mm_counts_only_the_outputs_there_are(m, n, k):
    """NaN blocks of either operand reach the places past the edges of a tile
    too; those are no outputs.  Ragged products of the 128 x 128 and the 256 x
    256 tile, even and odd n."""
    a, _ = _operand(m, k, 14)
    b, _ = _operand(n, k, 15)
    ctr = fm.Counters()
    assert torch.isfinite(fm.mx4_mm(a, b, counters=ctr)).all() and ctr.read()["nonfinite_out"] == 0
    nan = torch.zeros(m, n, dtype=torch.bool)
    for rows, cols in (((), (n - 1, 5)), ((0, m - 1), ()), ((m // 2,), (n // 3,))):
        a.s[0, list(rows), 0] = 255
        b.s[0, list(cols), (k - 1) // 32 % 16] = 255
        nan[list(rows)] = True
        nan[:, list(cols)] = True
        ctr = fm.Counters()
        y = fm.mx4_mm(a, b, counters=ctr)
        assert torch.equal(torch.isnan(y).cpu(), nan) and ctr.read()["nonfinite_out"] == int(nan.sum())


def test_calls_let_other_threads_run():
    """A call releases the interpreter while it enqueues: another thread gets
    on although the switch interval never ends."""
    import sys
    import threading
    import time
    x = _x(64, 512).cuda()
    q, _ = fm.mx4_quantize(x)
    turns, stop, started = [0], threading.Event(), threading.Event()

    def count():
        started.set()
        while not stop.is_set():
            turns[0] += 1
            time.sleep(1e-5)

    old = sys.getswitchinterval()
    thread = threading.Thread(target=count)
    thread.start()
    started.wait()
    sys.setswitchinterval(1000.0)
    try:
        got = []
        for call in (lambda: fm.mx4_quantize(x), lambda: fm.mx4_dequantize(q), lambda: fm.mx4_mm(q, q)):
            before = turns[0]
            for _ in range(3000):
                call()
            got.append(turns[0] - before)
    finally:
        sys.setswitchinterval(old)
        stop.set()
        thread.join()
    torch.cuda.synchronize()
    assert min(got) >= 30, got      # once in a hundred calls


def test_same_results_without_the_extension(monkeypatch):
    x = _x(70, 300).cuda()
    seed = torch.tensor([9], dtype=torch.int64, device="cuda")

    def calls():
        q, qt = fm.mx4_quantize(x, want_t=True, seed=seed)
        a = fm.Mx4(q.q, q.s, 300)
        e = fm.Mx4(torch.stack([qt.q[:140], qt.q[140:280]]), torch.stack([qt.s[:, :140], qt.s[:, 140:280]]), 70)
        w2 = fm.Mx4(q.q[:, :128][None].repeat(2, 1, 1).contiguous(), q.s[None].repeat(2, 1, 1, 1), 70)
        layer = fm.MoeMx4(torch.ones(2, 70, dtype=torch.bfloat16, device="cuda"), e, w2, 1, max_tokens=3)
        return [q.q, q.s, qt.q, qt.s, fm.mx4_dequantize(a, torch.float32), fm.mx4_mm(a, q), *layer(x[:3, :70])]

    want = calls()
    monkeypatch.setattr(fm, "_ext_module", fm._NoExt())
    # outputs past the range are NaN on both sides
    assert all(torch.equal(g.view(torch.uint8), w.view(torch.uint8)) for g, w in zip(calls(), want))


def test_a_single_row_may_have_any_row_stride():
    """A column turned into a row: stride 1 between rows that there are not."""
    x = _x(300, 1).cuda().t()
    assert x.shape == (1, 300) and x.stride() == (1, 1)
    same = x.contiguous().as_strided((1, 300), (300, 1))
    want, want_t = fm.mx4_quantize(same, want_t=True)
    for kw in ({}, {"counters": fm.Counters()}):
        q, qt = fm.mx4_quantize(x, want_t=True, **kw)
        assert all(torch.equal(a, b) for a, b in ((q.q, want.q), (q.s, want.s), (qt.q, want_t.q), (qt.s, want_t.s)))
    row = torch.zeros(300, 1, dtype=torch.bfloat16, device="cuda").t()
    assert torch.equal(fm.mx4_dequantize(q, out=row), fm.mx4_dequantize(q))
    y = torch.zeros(1, 1, dtype=torch.bfloat16, device="cuda").expand(1, 1)
    assert torch.equal(fm.mx4_mm(q, q, out=y), fm.mx4_mm(q, q))
