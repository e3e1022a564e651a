"""Refusals of the 4-bit entry points, on the CPU: the C ABI rejects bad
arguments before it touches the device, the binding before it calls it."""
import pytest
import torch

import fp8_scaled_matmul_amd as fm

BAD = 0x1000        # non-null, aligned, never dereferenced: every call fails before


@pytest.fixture(scope="module", autouse=True)
def _built():
    import os
    if not os.path.exists(fm.LIB_PATH):
        from fp8_scaled_matmul_amd import build
        build.build()


@pytest.mark.parametrize("args,code", [
    (dict(dtype=5), fm.FP8_ERR_INVALID_ARG),
    (dict(rows=-1), fm.FP8_ERR_INVALID_ARG),
    (dict(ld=10), fm.FP8_ERR_INVALID_ARG),
    (dict(x=None), fm.FP8_ERR_INVALID_ARG),
    (dict(x=BAD + 1), fm.FP8_ERR_INVALID_ARG),
    (dict(q=None), fm.FP8_ERR_INVALID_ARG),
    (dict(q=BAD + 8), fm.FP8_ERR_INVALID_ARG),
    (dict(ldq=255), fm.FP8_ERR_INVALID_ARG),
    (dict(ldq=264), fm.FP8_ERR_INVALID_ARG),
    (dict(ldq=128), fm.FP8_ERR_INVALID_ARG),
    (dict(s=None), fm.FP8_ERR_INVALID_ARG),
    (dict(s=BAD + 4), fm.FP8_ERR_INVALID_ARG),
    (dict(cols=513, ld=513, ldq=384, ps=16 * 63), fm.FP8_ERR_INVALID_ARG),
    (dict(q_t=BAD), fm.FP8_ERR_INVALID_ARG),
    (dict(s_t=BAD), fm.FP8_ERR_INVALID_ARG),
    (dict(q_t=BAD, s_t=BAD, ldq_t=64), fm.FP8_ERR_INVALID_ARG),
    (dict(seed=BAD + 4), fm.FP8_ERR_INVALID_ARG),
    (dict(rows=1 << 31), fm.FP8_ERR_UNSUPPORTED_SHAPE),
])
def test_quantize_rejects_before_device(args, code):
    a = dict(x=BAD, dtype=fm.BF16, rows=64, cols=512, ld=513, q=BAD, ldq=256, s=BAD, ps=1024, q_t=None, ldq_t=0,
             s_t=None, ps_t=0, seed=None, ctr=None)
    a.update(args)
    assert fm.fp8_mx4_quantize(*a.values(), None) == code, fm.lib().fp8_last_error()


@pytest.mark.parametrize("args,code", [
    (dict(dtype=3), fm.FP8_ERR_INVALID_ARG),
    (dict(q=None), fm.FP8_ERR_INVALID_ARG),
    (dict(y=None), fm.FP8_ERR_INVALID_ARG),
    (dict(ldy=511), fm.FP8_ERR_INVALID_ARG),
    (dict(y=BAD + 2, dtype=fm.FP32), fm.FP8_ERR_INVALID_ARG),
])
def test_dequantize_rejects_before_device(args, code):
    a = dict(q=BAD, ldq=256, s=BAD, ps=1024, rows=64, cols=512, y=BAD, dtype=fm.BF16, ldy=512)
    a.update(args)
    assert fm.fp8_mx4_dequantize(*a.values(), None) == code, fm.lib().fp8_last_error()


@pytest.mark.parametrize("args,code", [
    (dict(m=-1), fm.FP8_ERR_INVALID_ARG),
    (dict(a=None), fm.FP8_ERR_INVALID_ARG),
    (dict(b=BAD + 8), fm.FP8_ERR_INVALID_ARG),
    (dict(sb=None), fm.FP8_ERR_INVALID_ARG),
    (dict(lda=128), fm.FP8_ERR_INVALID_ARG),
    (dict(psb=16 * 47), fm.FP8_ERR_INVALID_ARG),
    (dict(psb=16 * 48 + 8), fm.FP8_ERR_INVALID_ARG),
    (dict(c=None), fm.FP8_ERR_INVALID_ARG),
    (dict(c=BAD + 1), fm.FP8_ERR_INVALID_ARG),
    (dict(ldc=47), fm.FP8_ERR_INVALID_ARG),
    (dict(lda=1 << 22), fm.FP8_ERR_UNSUPPORTED_SHAPE),
    (dict(ldc=1 << 21), fm.FP8_ERR_UNSUPPORTED_SHAPE),
    (dict(k=1 << 31), fm.FP8_ERR_UNSUPPORTED_SHAPE),
])
def test_mm_rejects_before_device(args, code):
    a = dict(a=BAD, lda=384, sa=BAD, psa=16 * 32, b=BAD, ldb=384, sb=BAD, psb=16 * 48, m=32, n=48, k=768, c=BAD,
             ldc=48, ctr=None)
    a.update(args)
    assert fm.fp8_mx4_mm(*a.values(), None) == code, fm.lib().fp8_last_error()


def _mx4(rows, cols):
    return fm.Mx4.empty(rows, cols, "cpu")


def test_mx4_layout_is_checked():
    q, s = torch.zeros(5, 256, dtype=torch.uint8), torch.zeros(1, 5, 16, dtype=torch.uint8)
    assert fm.Mx4(q, s, 500).shape == (5, 500)
    for bad in [(q.short(), s, 500), (q, s, 256), (q, s, 513), (q, s.reshape(5, 1, 16), 500),
                (q.t().contiguous().t(), s, 500), (q, s.expand(1, 5, 16)[..., ::1].transpose(1, 2), 500)]:
        with pytest.raises(ValueError):
            fm.Mx4(*bad)


def test_binding_rejects():
    x = torch.zeros(8, 64, dtype=torch.bfloat16)
    for kw in [dict(x=x.half()), dict(x=x[0]), dict(x=x.t()), dict(seed=torch.zeros(1)),
               dict(seed=torch.zeros(2, dtype=torch.int64)), dict(out=_mx4(8, 65)), dict(out=x),
               dict(out_t=_mx4(64, 8)), dict(want_t=True, out_t=_mx4(8, 64))]:
        with pytest.raises(ValueError):
            fm.mx4_quantize(**{"x": x, **kw})
    with pytest.raises(ValueError, match="CUDA"):
        fm.mx4_quantize(x)
    with pytest.raises(ValueError, match="out must"):
        fm.mx4_dequantize(_mx4(8, 64), out=torch.zeros(8, 63))
    with pytest.raises(ValueError, match="dtype"):
        fm.mx4_dequantize(_mx4(8, 64), torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        fm.mx4_dequantize(_mx4(8, 64))
    with pytest.raises(ValueError, match="disagree"):
        fm.mx4_mm(_mx4(8, 64), _mx4(8, 65))
    with pytest.raises(ValueError, match="a must be an Mx4"):
        fm.mx4_mm(x, _mx4(8, 64))
    with pytest.raises(ValueError, match="out must"):
        fm.mx4_mm(_mx4(8, 64), _mx4(9, 64), out=torch.zeros(8, 9))
    with pytest.raises(ValueError, match="CUDA"):
        fm.mx4_mm(_mx4(8, 64), _mx4(9, 64))


@pytest.mark.parametrize("args,code", [
    (dict(tokens=-1), fm.FP8_ERR_INVALID_ARG),
    (dict(top_k=0), fm.FP8_ERR_INVALID_ARG),
    (dict(top_k=9), fm.FP8_ERR_INVALID_ARG),
    (dict(experts=0), fm.FP8_ERR_INVALID_ARG),
    (dict(inner=0), fm.FP8_ERR_INVALID_ARG),
    (dict(x=None), fm.FP8_ERR_INVALID_ARG),
    (dict(x=BAD + 1), fm.FP8_ERR_INVALID_ARG),
    (dict(ldx=255), fm.FP8_ERR_INVALID_ARG),
    (dict(router=None), fm.FP8_ERR_INVALID_ARG),
    (dict(ldr=255), fm.FP8_ERR_INVALID_ARG),
    (dict(y=None), fm.FP8_ERR_INVALID_ARG),
    (dict(ldy=255), fm.FP8_ERR_INVALID_ARG),
    (dict(ids=None), fm.FP8_ERR_INVALID_ARG),
    (dict(weights=None), fm.FP8_ERR_INVALID_ARG),
    (dict(w1=None), fm.FP8_ERR_INVALID_ARG),
    (dict(w1=(BAD, None, 128, 24576, 6144, 6144)), fm.FP8_ERR_INVALID_ARG),
    (dict(w1=(BAD, BAD, 64, 24576, 6144, 6144)), fm.FP8_ERR_INVALID_ARG),
    (dict(w2=(BAD, BAD, 128, 24584, 6144, 6144)), fm.FP8_ERR_INVALID_ARG),
    (dict(w2=(BAD, BAD, 128, 24576, 6144, -16)), fm.FP8_ERR_INVALID_ARG),
    (dict(ws=None), fm.FP8_ERR_INVALID_ARG),
    (dict(ws=BAD + 8), fm.FP8_ERR_INVALID_ARG),
    (dict(wsb=1024), fm.FP8_ERR_INVALID_ARG),
    (dict(tokens=65), fm.FP8_ERR_UNSUPPORTED_SHAPE),
    (dict(w1=(BAD, BAD, 1 << 26, 24576, 6144, 6144)), fm.FP8_ERR_UNSUPPORTED_SHAPE),
    (dict(w2=(BAD, BAD, 1 << 26, 24576, 6144, 6144)), fm.FP8_ERR_UNSUPPORTED_SHAPE),
    (dict(experts=513), fm.FP8_ERR_UNSUPPORTED_SHAPE),
    (dict(experts=20, top_k=17), fm.FP8_ERR_UNSUPPORTED_SHAPE),
    (dict(hidden=1 << 24, ldx=1 << 24, ldr=1 << 24, ldy=1 << 24), fm.FP8_ERR_UNSUPPORTED_SHAPE),
])
def test_moe_rejects_before_device(args, code):
    held = (BAD, BAD, 128, 24576, 6144, 6144)
    a = dict(x=BAD, tokens=4, hidden=256, ldx=256, router=BAD, ldr=256, w1=held, w2=held, experts=8, inner=96, top_k=2,
             renormalize=1, y=BAD, ldy=256, ids=BAD, weights=BAD, ws=BAD, wsb=1 << 30, ctr=None)
    a.update(args)
    for w in ("w1", "w2"):
        a[w] = fm.Mx4Experts(*a[w]) if a[w] else None
    assert fm.fp8_mx4_moe(*a.values(), None) == code, fm.lib().fp8_last_error()


def test_moe_binding_rejects():
    e, h, i = 4, 64, 32
    router = torch.zeros(e, h, dtype=torch.bfloat16)
    stack = lambda r, c: fm.Mx4(torch.zeros(e, r, 128, dtype=torch.uint8),      # noqa: E731
                                torch.zeros(e, 1, r, 16, dtype=torch.uint8), c)
    w1, w2 = stack(2 * i, h), stack(h, i)
    for bad in [(router.float(), w1, w2, 1), (router, _mx4(2 * i, h), w2, 1), (router, w2, w1, 1),
                (router[:3], w1, w2, 1), (router, w1, w2, 0), (router, w1, w2, 5), (router, w1, w2, 1, 65),
                (router, w1, w2, 1, 0), (router, w1.q, w2, 1)]:
        with pytest.raises(ValueError):
            fm.MoeMx4(*bad)
    with pytest.raises(ValueError, match="CUDA"):
        fm.MoeMx4(router, w1, w2, 2)


def test_extension_leaves_other_calls_to_python():
    """Calls that are not all in order get None from the extension module, so
    that the Python code refuses or handles them."""
    ext = fm._ext()
    x = torch.zeros(8, 64, dtype=torch.bfloat16)
    q, s = torch.zeros(5, 256, dtype=torch.uint8), torch.zeros(1, 5, 16, dtype=torch.uint8)
    assert ext.mx4_held(q, s, 500) == (256, 80)
    wide = torch.zeros(5, 300, dtype=torch.uint8)[:, :256]
    assert ext.mx4_held(wide, s, 500) == (300, 80)
    for args in [(q.short(), s, 500), (q, s, 256), (q, s, 513), (q, s[0], 500), (q, s, 500.0), (q, None, 500),
                 (q[0], s, 500), (q, s.expand(2, 5, 16), 500), (q, s), (q[:0], s[:, :0], 500)]:
        assert ext.mx4_held(*args) is None
    for args in [(x, False, None), (None, False, None), (x[0], False, None), (x, False, 5), (x,)]:
        assert ext.mx4_quantize(*args) is None
    a = _mx4(8, 64)
    assert ext.mx4_dequantize(a.q, a.s, a._held, a.cols, False) is None
    assert ext.mx4_mm(a.q, a.s, a._held, a.cols, a.q, a.s, a._held, a.cols) is None
    assert ext.mx4_mm(a.q, a.s, a._held, a.cols, a.q, a.s, a._held, 65) is None
    assert ext.mx4_moe(x, x, a.q, 0, 0, 8, 32, 1, 0, 8) is None


def test_extension_passes_errors_of_its_arguments_on():
    a = _mx4(8, 64)
    with pytest.raises(OverflowError):
        fm._ext().mx4_held(a.q, a.s, 1 << 70)


def test_moe_workspace_grows_with_tokens():
    """A workspace for some tokens serves every call of fewer."""
    import random
    rng = random.Random(3)
    sizes = [(512, 1, 520, 64), (400, 2, 600, 512), (1, 1, 1, 1), (512, 16, 9000, 64), (300, 3, 4100, 32)]
    sizes += [(rng.randint(1, 512), 1, rng.randint(1, 9000), rng.randint(1, 3000)) for _ in range(300)]
    for experts, top_k, hidden, inner in sizes:
        size = [fm.lib().fp8_mx4_moe_workspace_size(t, experts, top_k, hidden, inner) for t in range(1, 65)]
        assert size[0] > 0 and all(a <= b for a, b in zip(size, size[1:])), (experts, top_k, hidden, inner)


@pytest.mark.parametrize("rows,cols,want_t", [
    ((1 << 28) + 1, 1, False), ((1 << 19) + 1, 1 << 19, False), ((1 << 31) - 1, 1, False), ((1 << 29) + 1, 1, True),
    (1, (1 << 29) + 1, True), (1 << 19, (1 << 19) + 1, True)])
def test_tensors_too_large_for_one_launch(rows, cols, want_t):
    """A launch holds fewer than 2^32 work-items: larger tensors are refused
    as such."""
    ldq, ldt = 128 * -(-cols // 256), 128 * -(-rows // 256)
    st = fm.fp8_mx4_quantize(BAD, fm.BF16, rows, cols, cols, BAD, ldq, BAD, 16 * rows, BAD if want_t else None, ldt,
                             BAD if want_t else None, 16 * cols, None, None, None)
    assert st == fm.FP8_ERR_UNSUPPORTED_SHAPE
    if not want_t:
        st = fm.fp8_mx4_dequantize(BAD, ldq, BAD, 16 * rows, rows, cols, BAD, fm.BF16, cols, None)
        assert st == fm.FP8_ERR_UNSUPPORTED_SHAPE


def test_outputs_and_layers_too_large_for_one_launch():
    m, n = (1 << 31) - 1, (1 << 21) - 1
    st = fm.fp8_mx4_mm(BAD, 128, BAD, 0, BAD, 128, BAD, 0, m, n, 32, BAD, n, None, None)
    assert st == fm.FP8_ERR_UNSUPPORTED_SHAPE
    # 512 experts and 64 tokens' groups of 32-row tiles: 576 * 2^15 workgroups
    assert fm.lib().fp8_mx4_moe_workspace_size(64, 512, 16, 64, 1 << 20) == 0
    assert fm.lib().fp8_mx4_moe_workspace_size(64, 8, 2, 64, 1 << 20) > 0
    inner = 1 << 20
    w1 = fm.Mx4Experts(BAD, BAD, 128, 1 << 30, 32 * inner, 1 << 30)
    w2 = fm.Mx4Experts(BAD, BAD, inner // 2, 1 << 30, 1024, 1 << 30)
    st = fm.fp8_mx4_moe(BAD, 64, 64, 64, BAD, 64, w1, w2, 512, inner, 16, 1, BAD, 64, BAD, BAD, BAD, 1 << 60, None, None)
    assert st == fm.FP8_ERR_UNSUPPORTED_SHAPE


def test_without_the_extension_python_takes_every_call(monkeypatch):
    import sys
    monkeypatch.setitem(sys.modules, fm.__name__ + "._fp8mi_torch", None)      # as if it had not been built
    monkeypatch.setattr(fm, "_ext_module", None)
    q, s = torch.zeros(5, 256, dtype=torch.uint8), torch.zeros(1, 5, 16, dtype=torch.uint8)
    with pytest.warns(RuntimeWarning, match="not there"):
        a = fm.Mx4(q, s, 500)
    assert a.shape == (5, 500) and a._held == (256, 80)
    test_mx4_layout_is_checked()
    test_binding_rejects()
    test_moe_binding_rejects()
