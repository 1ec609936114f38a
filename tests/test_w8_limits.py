"""Limits of the 8-bit path's C entry points that need no GPU: every call here is
refused, or empty, before anything is launched."""

import ctypes

import pytest

wq = pytest.importorskip("bit_weight_only_wq_amd")
from bit_weight_only_wq_amd import _lib  # noqa: E402
from test_w8_abi import FAKE, at, gemm, normq, normv  # noqa: E402

# 48 rows on 1024 x 8192: K is split, so the workspace is written.  Rows of A and W a
# little apart, Y too.
B, K, N = 48, 8192, 1024
CALL = dict(B=B, K=K, N=N, as_=K + 16, ws_=K + 32, ys=N + 8, bias=at(5))
SPANS = {"A": (at(0), (B - 1) * (K + 16) + K), "W": (at(2), (N - 1) * (K + 32) + K), "Y": (at(4), 2 * ((B - 1) * (N + 8) + N)),
         "a_scales": (at(1), 4 * B), "w_scales": (at(3), 4 * N), "bias": (at(5), 2 * N)}


@pytest.mark.parametrize("name", list(SPANS))
def test_workspace_over_an_operand(name):
    n = ctypes.c_size_t(0)
    assert wq.load().wq_gemm_w8a8_workspace_size(B, K, N, ctypes.byref(n)) == _lib.WQ_OK and n.value > 0
    first, size = SPANS[name]
    last = (first + size - 1) // 16 * 16
    for p in (first, last, (first + last) // 32 * 16, first - n.value // 32 * 16, first - (n.value - 1) // 16 * 16):
        assert gemm(**CALL, p=p, n=n.value) == _lib.WQ_ERR_INVALID_ARG, (name, p - FAKE)
        assert b"overlaps" in wq.load().wq_last_error()


LARGEST = 3.4028234663852886e38                                # fp32's


@pytest.mark.parametrize("eps,want", [(2.0 ** -126, _lib.WQ_OK), (1e-6, _lib.WQ_OK), (3.4e38, _lib.WQ_OK), (3.4025e38, _lib.WQ_OK),
                                      (LARGEST, _lib.WQ_OK), (float("inf"), _lib.WQ_ERR_INVALID_ARG),
                                      (2.0 ** -126 - 2.0 ** -149, _lib.WQ_ERR_INVALID_ARG)])
def test_eps_from_end_to_end(eps, want):
    """Calls of no rows: eps is looked at, nothing is launched."""
    assert normq(R=0, eps=eps) == want and normv(R=0, eps=eps) == want


def test_type_numbers():
    """The binding's numbers of the 16-bit types are wq.h's."""
    import os
    import re
    header = open(os.path.join(os.path.dirname(__file__), "..", "include", "wq.h")).read()
    for name in ("WQ_FP16", "WQ_BF16"):
        assert int(re.search(name + r" = (\d+)", header).group(1)) == getattr(_lib, name)
