"""Refusals of the vocabulary loss, the experts' router and dropout, on the CPU:
the C ABI rejects bad arguments before it touches the device, the binding before
it calls it."""
import pytest
import torch

import fp8_scaled_matmul_amd as fm

BAD = 0x1000        # non-null, aligned, never dereferenced: every call fails before
INVALID, SHAPE = fm.FP8_ERR_INVALID_ARG, fm.FP8_ERR_UNSUPPORTED_SHAPE


@pytest.fixture(scope="module", autouse=True)
def _built():
    import os
    if not os.path.exists(fm.LIB_PATH):
        from fp8_scaled_matmul_amd import build
        build.build()


HEAD = [
    (dict(tokens=-1), INVALID), (dict(vocab=0), INVALID), (dict(hidden=0), INVALID), (dict(x=None), INVALID),
    (dict(w=None), INVALID), (dict(ldx=63), INVALID), (dict(ldw=63), INVALID), (dict(x=BAD + 1), INVALID),
    (dict(w=BAD + 1), INVALID), (dict(targets=None), INVALID), (dict(targets=BAD + 4), INVALID),
    (dict(softcap=-1.0), INVALID), (dict(softcap=float("nan")), INVALID), (dict(softcap=float("inf")), INVALID),
    (dict(tokens=1 << 24), SHAPE), (dict(vocab=1 << 24), SHAPE), (dict(ldx=1 << 21), SHAPE), (dict(ldw=1 << 21), SHAPE),
    (dict(ws=None), INVALID), (dict(ws=BAD + 8), INVALID), (dict(wsb=1000), INVALID),
]


@pytest.mark.parametrize("args,code", HEAD + [(dict(loss=None), INVALID), (dict(lse=BAD + 2), INVALID)])
def test_linear_ce_rejects_before_device(args, code):
    a = dict(x=BAD, ldx=64, w=BAD, ldw=64, tokens=32, vocab=100, hidden=64, targets=BAD, softcap=0.0, loss=BAD, lse=BAD,
             ws=BAD, wsb=1 << 40)
    a.update(args)
    assert fm.fp8_linear_ce(*a.values(), None) == code, fm.lib().fp8_last_error()


@pytest.mark.parametrize("args,code", HEAD + [
    (dict(lse=None), INVALID), (dict(grad=None), INVALID), (dict(grad=BAD + 2), INVALID), (dict(step=-1), INVALID),
    (dict(lddx=63), INVALID), (dict(lddw=63), INVALID), (dict(dx=BAD + 1), INVALID), (dict(dw=BAD + 1), INVALID),
    (dict(lddx=1 << 21), SHAPE), (dict(lddw=1 << 21), SHAPE)])
def test_linear_ce_backward_rejects_before_device(args, code):
    a = dict(x=BAD, ldx=64, w=BAD, ldw=64, tokens=32, vocab=100, hidden=64, targets=BAD, softcap=0.0, lse=BAD, grad=BAD,
             step=1, dx=BAD, lddx=64, dw=BAD, lddw=64, ws=BAD, wsb=1 << 40)
    a.update(args)
    assert fm.fp8_linear_ce_backward(*a.values(), None) == code, fm.lib().fp8_last_error()


def test_linear_ce_workspace():
    size = fm.lib().fp8_linear_ce_workspace_size
    for back in (0, 1):
        assert size(0, 100, 64, back) == 0 and size(10, 0, 64, back) == 0 and size(10, 100, 0, back) == 0
        assert size(1 << 24, 100, 64, back) == 0 and size(10, 1 << 24, 64, back) == 0 and size(10, 100, 1 << 21, back) == 0
        assert 0 < size(1, 1, 1, back) <= size(100, 1000, 64, back)
    # the logits' gradient is held in pieces: far below all of it
    assert size(65536, 131072, 1024, 1) < 65536 * 131072 * 2 // 8


ROUTE = [
    (dict(dtype=2), INVALID), (dict(tokens=-1), INVALID), (dict(experts=0), INVALID), (dict(top_k=0), INVALID),
    (dict(top_k=65), INVALID), (dict(logits=None), INVALID), (dict(ld=63), INVALID), (dict(logits=BAD + 1), INVALID),
    (dict(dtype=fm.FP32, logits=BAD + 2), INVALID), (dict(experts=513, ld=513), SHAPE), (dict(top_k=17), SHAPE),
    (dict(tokens=1 << 27), SHAPE), (dict(ids=None), INVALID), (dict(weights=None), INVALID), (dict(counts=None), INVALID),
    (dict(ids=BAD + 2), INVALID), (dict(weights=BAD + 1), INVALID), (dict(counts=BAD + 2), INVALID),
]


@pytest.mark.parametrize("args,code", ROUTE + [
    (dict(balance=None), INVALID), (dict(balance=BAD + 2), INVALID), (dict(ws=None), INVALID), (dict(ws=BAD + 4), INVALID),
    (dict(wsb=16), INVALID)])
def test_route_rejects_before_device(args, code):
    a = dict(logits=BAD, dtype=fm.BF16, tokens=32, experts=64, ld=64, top_k=4, renormalize=1, mask=None, ids=BAD, weights=BAD,
             counts=BAD, balance=BAD, ws=BAD, wsb=1 << 40)
    a.update(args)
    assert fm.fp8_moe_route(*a.values(), None) == code, fm.lib().fp8_last_error()


@pytest.mark.parametrize("args,code", ROUTE + [
    (dict(dlogits=None), INVALID), (dict(dlogits=BAD + 1), INVALID), (dict(ldd=63), INVALID), (dict(gw=BAD + 2), INVALID),
    (dict(gb=BAD + 2), INVALID)])
def test_route_backward_rejects_before_device(args, code):
    a = dict(logits=BAD, dtype=fm.BF16, tokens=32, experts=64, ld=64, top_k=4, renormalize=1, ids=BAD, weights=BAD,
             counts=BAD, gw=BAD, gb=BAD, dlogits=BAD, ldd=64)
    a.update(args)
    assert fm.fp8_moe_route_backward(*a.values(), None) == code, fm.lib().fp8_last_error()


def test_route_workspace():
    size = fm.lib().fp8_moe_route_workspace_size
    assert size(0, 64) == 0 and size(10, 0) == 0 and size(10, 513) == 0 and size(1 << 27, 64) == 0
    assert 0 < size(1, 1) <= size(100, 64)


@pytest.mark.parametrize("args,code", [
    (dict(dtype=2), INVALID), (dict(rows=-1), INVALID), (dict(x=None), INVALID), (dict(y=None), INVALID),
    (dict(ld=31), INVALID), (dict(ldr=31), INVALID), (dict(ldy=31), INVALID), (dict(x=BAD + 1), INVALID),
    (dict(residual=BAD + 1), INVALID), (dict(y=BAD + 1), INVALID), (dict(dtype=fm.FP32, y=BAD + 2), INVALID),
    (dict(rate=-0.1), INVALID), (dict(rate=1.1), INVALID), (dict(rate=float("nan")), INVALID), (dict(seed=None), INVALID),
    (dict(seed=BAD + 4), INVALID), (dict(rows=1 << 31), SHAPE), (dict(cols=1 << 31, ld=1 << 31, ldr=1 << 31, ldy=1 << 31), SHAPE)])
def test_dropout_rejects_before_device(args, code):
    a = dict(x=BAD, dtype=fm.BF16, rows=64, cols=32, ld=32, residual=BAD, ldr=32, rate=0.1, seed=BAD, y=BAD, ldy=32)
    a.update(args)
    assert fm.fp8_dropout(*a.values(), None) == code, fm.lib().fp8_last_error()


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_binding_refuses_what_is_wrong_with_a_head():
    x, w, t, f = bf(4, 16), bf(30, 16), torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    back = fm.linear_cross_entropy_backward
    for call in (
        lambda: fm.linear_cross_entropy(x.float(), w, t),
        lambda: fm.linear_cross_entropy(x, w.float(), t),
        lambda: fm.linear_cross_entropy(x, bf(30, 17), t),
        lambda: fm.linear_cross_entropy(x, w, t.int()),
        lambda: fm.linear_cross_entropy(x, w, t[:3]),
        lambda: fm.linear_cross_entropy(x, w, torch.zeros(8, dtype=torch.int64)[::2]),
        lambda: fm.linear_cross_entropy(x, bf(16, 30).t(), t),
        lambda: fm.linear_cross_entropy(bf(4, 2, 16), w, t),
        lambda: fm.linear_cross_entropy(x, w, t, softcap=-1),
        lambda: fm.linear_cross_entropy(x, w, t, softcap=float("nan")),
        lambda: fm.linear_cross_entropy(x, w, t, workspace=f),
        lambda: back(x, w, t, f.double(), f),
        lambda: back(x, w, t, f[:2], f),
        lambda: back(x, w, t, f, f.bfloat16()),
        lambda: back(x, w, t, f, torch.zeros(())),
        lambda: back(x, w, t, f, f, out_x=bf(4, 15)),
        lambda: back(x, w, t, f, f, out_w=w.float()),
        lambda: back(x, w, t, f, f, want_x=False, out_x=x),
        lambda: fm.linear_cross_entropy(x, w, t),           # on the CPU
        lambda: back(x, w, t, f, f),
    ):
        with pytest.raises(ValueError):
            call()


def test_binding_refuses_what_is_wrong_with_a_route():
    l, f = bf(4, 16), torch.zeros(4, 2)
    r = fm.Route(torch.zeros(4, 2, dtype=torch.int32), f, torch.zeros(16, dtype=torch.int32), torch.zeros(()), True)
    for call in (
        lambda: fm.moe_route(l.half(), 2),
        lambda: fm.moe_route(l, 0),
        lambda: fm.moe_route(l, 17),
        lambda: fm.moe_route(l.t(), 2),
        lambda: fm.moe_route(l, 2, mask=torch.ones(4)),
        lambda: fm.moe_route(l, 2, mask=torch.ones(5, dtype=torch.bool)),
        lambda: fm.moe_route(l, 2, workspace=f),
        lambda: fm.moe_route_backward(l, None),
        lambda: fm.moe_route_backward(l[:3], r),
        lambda: fm.moe_route_backward(bf(4, 17), r),
        lambda: fm.moe_route_backward(l, r, f.double()),
        lambda: fm.moe_route_backward(l, r, f[:, :1]),
        lambda: fm.moe_route_backward(l, r, f, torch.zeros(2)),
        lambda: fm.moe_route_backward(l, r, f, out=l.float()),
        lambda: fm.moe_route(l, 2),                         # on the CPU
        lambda: fm.moe_route_backward(l, r, f),
    ):
        with pytest.raises(ValueError):
            call()


def test_binding_refuses_what_is_wrong_with_a_dropout():
    x, s = bf(4, 16), torch.zeros(1, dtype=torch.int64)
    for call in (
        lambda: fm.dropout(x.half(), 0.1, s),
        lambda: fm.dropout(x[0], 0.1, s),
        lambda: fm.dropout(x.t(), 0.1, s),
        lambda: fm.dropout(x, -0.1, s),
        lambda: fm.dropout(x, 1.5, s),
        lambda: fm.dropout(x, float("nan"), s),
        lambda: fm.dropout(x, 0.1, s.int()),
        lambda: fm.dropout(x, 0.1, torch.zeros(2, dtype=torch.int64)),
        lambda: fm.dropout(x, 0.1, s, residual=x.float()),
        lambda: fm.dropout(x, 0.1, s, out=bf(4, 15)),
        lambda: fm.dropout(x, 0.1, s),                      # on the CPU
    ):
        with pytest.raises(ValueError):
            call()


def test_caps_that_are_no_caps():
    """Too small for its square in fp32, or for fp32 at all."""
    assert fm.fp8_linear_ce(BAD, 64, BAD, 64, 32, 100, 64, BAD, 1e-31, BAD, BAD, BAD, 1 << 40, None) == INVALID
    for cap in (1e-31, 1e-50):
        with pytest.raises(ValueError, match="softcap"):
            fm.linear_cross_entropy(bf(4, 16), bf(30, 16), torch.zeros(4, dtype=torch.int64), softcap=cap)
