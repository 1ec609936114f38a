"""Checks of the 8-bit path's C entry points that need no GPU: bad arguments are
refused synchronously, before any launch, with a status and a message; empty
calls are no-ops.  And of the tests' own oracle, on borders worked by hand."""

import ctypes
import math

import numpy as np
import pytest

wq = pytest.importorskip("bit_weight_only_wq_amd")
torch = pytest.importorskip("torch")
from bit_weight_only_wq_amd import _lib  # noqa: E402
import w8_util  # noqa: E402

FAKE = 0x100000  # 16-byte aligned, never dereferenced (validation fails first)
OK, BAD, UNSUP, MIS = _lib.WQ_OK, _lib.WQ_ERR_INVALID_ARG, _lib.WQ_ERR_UNSUPPORTED, _lib.WQ_ERR_MISALIGNED


def at(i):
    return FAKE + (i << 24)


def rows(x=at(0), xs=64, g=at(1), gs=64, R=3, K=64, dt=0, c=at(2), cs=64, s=at(3)):
    return wq.load().wq_quantize_rows(x, xs, g, gs, R, K, dt, c, cs, s, None)


def normq(x=at(0), xs=64, r=at(1), rs=64, w=at(2), R=3, K=64, dt=0, eps=1e-6, t=at(3), ts=64, c=at(4), cs=64, s=at(5)):
    return wq.load().wq_rmsnorm_quantize(x, xs, r, rs, w, R, K, dt, eps, t, ts, c, cs, s, None)


def normv(x=at(0), xs=64, r=at(1), rs=64, w=at(2), R=3, K=64, dt=0, eps=1e-6, t=at(3), ts=64, c=at(4), cs=64):
    return wq.load().wq_rmsnorm(x, xs, r, rs, w, R, K, dt, eps, t, ts, c, cs, None)


def gemm(A=at(0), as_=64, sa=at(1), W=at(2), ws_=64, sw=at(3), bias=0, Y=at(4), ys=32, B=3, K=64, N=32, dt=0, p=0, n=0):
    return wq.load().wq_gemm_w8a8(A, as_, sa, W, ws_, sw, bias, Y, ys, B, K, N, dt, p, n, None)


SHAPES = [(dict(R=-1), BAD), (dict(K=0), BAD), (dict(dt=2), BAD), (dict(dt=-1), BAD), (dict(R=1 << 24), UNSUP),
          (dict(K=(1 << 20) + 1, xs=1 << 21, cs=1 << 21), UNSUP), (dict(xs=-1), BAD), (dict(xs=1 << 38), BAD),
          (dict(cs=63), BAD), (dict(cs=-1, R=1), BAD), (dict(x=0), BAD), (dict(c=0), BAD), (dict(x=at(0) + 1), MIS),
          (dict(R=0, x=0, c=0), OK)]


@pytest.mark.parametrize("kw,want", SHAPES + [(dict(gs=-1), BAD), (dict(s=0), BAD), (dict(g=at(1) + 1), MIS),
                                              (dict(s=at(3) + 2), MIS)])
def test_rows_refusals(kw, want):
    assert rows(**kw) == want
    assert (want == OK) == (wq.load().wq_last_error() == b"")


NORMS = SHAPES + [(dict(rs=-1), BAD), (dict(ts=63), BAD), (dict(w=0), BAD), (dict(r=0), BAD), (dict(t=0), BAD),
                  (dict(eps=0.0), BAD), (dict(eps=-1.0), BAD), (dict(eps=math.nan), BAD), (dict(eps=math.inf), BAD),
                  (dict(eps=1e-39), BAD), (dict(t=at(0), xs=128), BAD), (dict(t=at(1), rs=128), BAD),
                  (dict(w=at(2) + 1), MIS), (dict(r=at(1) + 1), MIS), (dict(t=at(3) + 1), MIS)]


@pytest.mark.parametrize("kw,want", NORMS + [(dict(s=0), BAD), (dict(s=at(5) + 1), MIS)])
def test_norm_codes_refusals(kw, want):
    assert normq(**kw) == want
    assert (want == OK) == (wq.load().wq_last_error() == b"")


@pytest.mark.parametrize("kw,want", NORMS + [(dict(c=at(4) + 1), MIS)])
def test_norm_values_refusals(kw, want):
    assert normv(**kw) == want
    assert (want == OK) == (wq.load().wq_last_error() == b"")


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), BAD), (dict(N=-1), BAD), (dict(K=0), BAD), (dict(K=8), UNSUP), (dict(K=72, as_=80, ws_=80), UNSUP),
    (dict(K=1 << 17, as_=1 << 17, ws_=1 << 17), UNSUP), (dict(B=(1 << 20) + 1), UNSUP),
    (dict(N=(1 << 24) + 1, ys=1 << 25), UNSUP), (dict(dt=2), BAD), (dict(as_=48), BAD), (dict(ws_=48), BAD),
    (dict(ys=31), BAD), (dict(as_=1 << 23), BAD), (dict(ws_=1 << 23), BAD), (dict(ys=1 << 38), BAD),
    (dict(as_=-16, B=1), BAD), (dict(A=0), BAD), (dict(W=0), BAD), (dict(sa=0), BAD), (dict(sw=0), BAD), (dict(Y=0), BAD),
    (dict(A=at(0) + 8), MIS), (dict(W=at(2) + 4), MIS), (dict(as_=72), MIS), (dict(ws_=72), MIS), (dict(sa=at(1) + 2), MIS),
    (dict(sw=at(3) + 1), MIS), (dict(bias=at(5) + 1), MIS), (dict(Y=at(4) + 1), MIS), (dict(n=64), BAD),
    (dict(p=at(6) + 4, n=1 << 40), MIS), (dict(B=0, A=0, sa=0, Y=0), OK), (dict(N=0, W=0, sw=0, Y=0), OK)])
def test_gemm_refusals(kw, want):
    assert gemm(**kw) == want
    assert (want == OK) == (wq.load().wq_last_error() == b"")


def test_gemm_workspace_size():
    lib, n = wq.load(), ctypes.c_size_t(7)
    assert lib.wq_gemm_w8a8_workspace_size(3, 64, 32, None) == BAD
    assert lib.wq_gemm_w8a8_workspace_size(0, 64, 32, ctypes.byref(n)) == OK and n.value == 0
    assert lib.wq_gemm_w8a8_workspace_size(3, 60, 32, ctypes.byref(n)) == UNSUP and n.value == 0
    assert lib.wq_gemm_w8a8_workspace_size(-1, 64, 32, ctypes.byref(n)) == BAD and n.value == 0
    for B, K, N in ((1, 64, 16), (48, 8192, 1024), (333, 11008, 4096), (8192, 8192, 28672)):
        assert lib.wq_gemm_w8a8_workspace_size(B, K, N, ctypes.byref(n)) == OK
        if n.value:                              # one byte too few is refused before any launch
            assert gemm(B=B, K=K, N=N, as_=K, ws_=K, ys=N, p=at(6), n=n.value - 1) == BAD


def test_oracle_borders():
    """127 t / max with max = 127: codes are the nearest whole numbers, ties to even."""
    t = np.array([[127.0, 0.5, 1.5, -0.5, -1.5, 2.5, 126.5, 0.4999999999, -2.5000001, 0.0], [0.0] * 10])
    codes, top = w8_util.nearest_codes(t)
    assert codes[0].tolist() == [127, 0, 2, 0, -2, 2, 126, 0, -3, 0] and top[0] == 127
    assert not codes[1].any() and top[1] == 0
    x = torch.tensor([[3.0, -4.0]]).half()
    y, codes, scales, h = w8_util.norm(x, torch.tensor([1.0, 0.5]).half(), None, 1.0)
    r = 1 / math.sqrt(13.5)
    assert np.allclose(y, [[3 * r, -2 * r]], rtol=1e-15) and codes.tolist() == [[127, -85]]
    assert math.isclose(scales[0], 3 * r / 127, rel_tol=1e-15) and h is x
    a = np.array([[1, -128]], np.int8)
    y = w8_util.product(a, np.array([0.5], np.float32), np.array([[2, 127]], np.int8), np.array([0.25], np.float32),
                        torch.tensor([0.75]).half(), torch.float16)
    assert y.tolist() == [[(2 - 128 * 127) * 0.125 + 0.75]]


def test_product_bytes():
    from bit_weight_only_wq_amd import roofline as rl
    assert rl.gemm_w8a8_bytes(3, 5, 16) == 48 + 80 + 4 * 8 + 30


def test_cpu_tensors_are_refused():
    """The binding never hands host memory to a kernel."""
    h, i8 = torch.ones((4, 64)).half(), torch.ones((4, 64), dtype=torch.int8)
    one = torch.ones(4)
    for bad in [lambda: wq.quantize_rows(h), lambda: wq.rmsnorm(h, h[0]), lambda: wq.rmsnorm_quantize(h, h[0], residual=h),
                lambda: wq.gemm_w8a8(i8, one, i8, one), lambda: wq.gemm_w8a8(i8, one, i8, one, out=h[:, :4]),
                lambda: wq.quantize_rows(h.numpy()), lambda: wq.gemm_w8a8(None, one, i8, one)]:
        with pytest.raises(ValueError):
            bad()
