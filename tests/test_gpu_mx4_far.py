"""The 4-bit operators where offsets pass 2^31 bytes: large tensors, and small
ones whose rows, panels or experts lie far apart."""
import numpy as np
import pytest
import torch

import fp8_scaled_matmul_amd as fm
from oracle import mx4
from test_gpu_mx4 import _check_mm, _f64, _operand
from test_gpu_mx4_moe import Layer

pytestmark = pytest.mark.gpu
FAR = 1 << 31


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def _apart(t, dim, stride):
    """t with `stride` elements between its entries along dim."""
    strides = [0] * t.dim()
    near = 1
    for d in reversed(range(t.dim())):
        if d != dim:
            strides[d] = near
            near *= t.shape[d]
    assert stride >= near
    strides[dim] = stride
    buf = torch.empty((t.shape[dim] - 1) * stride + near, dtype=t.dtype, device="cuda")
    out = buf.as_strided(t.shape, strides)
    out.copy_(t)
    return out


def test_large_tensor_both_ways():
    rows, cols, last = 70000, 32768, 69632          # 2.3 e9 elements; the last panel of rows and what follows
    x = torch.randn(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[last:] *= torch.exp2(torch.arange(rows - last, device="cuda") % 40 - 20.0).bfloat16()[:, None]
    seed = torch.tensor([77], dtype=torch.int64, device="cuda")
    q, qt = fm.mx4_quantize(x, want_t=True)
    w, wt = fm.mx4_quantize(x[last:], want_t=True)
    assert torch.equal(q.q[last:], w.q) and torch.equal(q.s[:, last:], w.s)
    assert torch.equal(qt.q[:, last // 2:], wt.q) and torch.equal(qt.s[last // 512:], wt.s)
    only, _ = fm.mx4_quantize(x)
    assert torch.equal(only.q, q.q) and torch.equal(only.s, q.s)
    for dtype in (torch.bfloat16, torch.float32):
        y = fm.mx4_dequantize(q, dtype)
        assert torch.equal(y[last:], fm.mx4_dequantize(w, dtype))
        del y
    r, rt = fm.mx4_quantize(x, want_t=True, seed=seed)
    row, n = rows - 2, 704
    codes, sb, _ = mx4.quantize(_f64(x[row:, :n]), mx4.random_bits(2, n, 77, row))
    eq, es = mx4.pack(codes, sb)
    assert np.array_equal(r.q[row:, :n // 2].cpu().numpy(), eq[:, :n // 2])
    assert np.array_equal(r.s[0, row:].cpu().numpy(), es[0][:, :16])
    # the same bits in the transposed copy: the last whole block of rows, one column
    b0 = rows // 32 * 32 - 32
    codes, sb, _ = mx4.quantize(_f64(x[b0:b0 + 32, 32766:]).T, mx4.random_bits(32, 32768, 77, b0)[:, 32766:].T)
    eq, _ = mx4.pack(codes, sb)
    assert np.array_equal(rt.q[32766:, b0 // 2:b0 // 2 + 16].cpu().numpy(), eq[:, :16])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_and_panels_far_apart(dtype):
    x = torch.randn(4, 1100, device="cuda").to(dtype)
    far = _apart(x, 0, FAR // x.element_size() // 2 + 8)
    want, want_t = fm.mx4_quantize(x, want_t=True)

    o = fm.Mx4(_apart(want.q, 0, FAR // 2 + 16), _apart(want.s, 0, FAR + 16), want.cols)
    for v in (o.q, o.s):
        v.zero_()
    fm.mx4_quantize(far, out=o)
    assert torch.equal(o.q, want.q) and torch.equal(o.s, want.s)
    q, qt = fm.mx4_quantize(far, want_t=True)
    assert torch.equal(q.q, want.q) and torch.equal(qt.q, want_t.q) and torch.equal(qt.s, want_t.s)
    y = _apart(torch.zeros(4, 1100, dtype=dtype, device="cuda"), 0, FAR // x.element_size() // 2 + 8)
    fm.mx4_dequantize(o, out=y)
    assert torch.equal(y, fm.mx4_dequantize(want, dtype))


def test_mm_large_operand_and_output():
    m, k = 70000, 65536
    codes = torch.randint(0, 256, (m, k // 2), dtype=torch.uint8, device="cuda")
    scales = torch.randint(120, 130, (k // 512, m, 16), dtype=torch.uint8, device="cuda")
    a = fm.Mx4(codes, scales, k)
    last = m - 40
    va = mx4.values(*mx4.unpack(codes[last:].cpu().numpy(), scales[:, last:].contiguous().cpu().numpy(), k))
    for n in (16, 600):
        b, vb = _operand(n, k, 20, 120, 130)
        _check_mm(fm.mx4_mm(a, b)[last:], va, vb)
    n, k = 20000, 64
    a, va = _operand(m, k, 21)
    b, vb = _operand(n, k, 22)
    y = fm.mx4_mm(a, b)
    for rows in (slice(0, 40), slice(last, m)):
        _check_mm(y[rows], va[rows], vb)


@pytest.mark.parametrize("m,n", [(3, 700), (600, 520), (1500, 1500), (3000, 3000)])
def test_mm_rows_and_panels_far_apart(m, n):
    """Each kind of tile, at the largest distances it takes."""
    k = 700
    a, va = _operand(m, k, 23)
    b, vb = _operand(n, k, 24)
    want = fm.mx4_mm(a, b)
    _check_mm(want, va, vb)
    far_a = fm.Mx4(_apart(a.q, 0, (1 << 22) - 16), _apart(a.s, 0, FAR + 16), k)
    assert torch.equal(fm.mx4_mm(far_a, b), want)
    del far_a
    far_b = fm.Mx4(_apart(b.q, 0, (1 << 22) - 16), _apart(b.s, 0, FAR + 16), k)
    assert torch.equal(fm.mx4_mm(a, far_b), want)
    del far_b
    for ldc in ((1 << 21) - 2, (1 << 21) - 1):
        y = _apart(torch.zeros(m, n, dtype=torch.bfloat16, device="cuda"), 0, ldc)
        fm.mx4_mm(a, b, out=y)
        assert torch.equal(y, want)
        del y


def test_moe_experts_and_rows_far_apart():
    m = Layer(6, 4, 2, 1100, 600, True)
    x = m.x(6, 1100).cuda()
    want = m.moe(x)
    m.check(x.cpu(), want)

    def far(w):
        return fm.Mx4(_apart(w.q, 0, FAR // 2 + 16), _apart(w.s, 0, FAR // 2 + 16), w.cols)

    w1, w2 = far(m.w1), far(m.w2)
    # scale panels far apart, experts between them
    s = torch.empty(3 * (1 << 20) + 2 * (FAR + (1 << 24)), dtype=torch.uint8, device="cuda")
    e, panels, rows, _ = m.w2.s.shape
    s = s.as_strided((e, panels, rows, 16), (1 << 20, FAR + (1 << 24), 16, 1))
    s.copy_(m.w2.s)
    router = _apart(m.router.cuda(), 0, FAR // 4 + 8)
    far_x = _apart(x, 0, FAR // 4 + 8)
    out = _apart(torch.zeros_like(x), 0, FAR // 4 + 8)
    for second in (w2, fm.Mx4(w2.q, s, w2.cols)):
        got = fm.MoeMx4(router, w1, second, 2, max_tokens=6)(far_x, out=out)
        assert all(torch.equal(g, w) for g, w in zip(got, want))
