"""GPU tests of the 8-bit path at the ends of what it takes: inputs whose rows
repeat or overlap, bf16 products past fp32's range on either side, streams.

Tolerances as in test_gpu_w8_rows: a scale of quantize_rows within 2^-22, of the
norm within 2^-21, values half a step of their type and 2^-22."""

import numpy as np
import pytest

import w8_util
from gpu_util import device, note
from test_gpu_w8_rows import check_codes, check_values, randn
from w8_util import TYPES, bits

import bit_weight_only_wq_amd as wq

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def same(got, want):
    for g, w in zip(got, want):
        assert (g is None) == (w is None)
        if g is not None:
            assert g.shape == w.shape and g.is_contiguous()
            assert torch.equal(g, w) if g.dtype != torch.bfloat16 else torch.equal(bits(g), bits(w))


# Windows of a line one, two and K values apart, and one row repeated: rows fewer
# and more than values.
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("R,K", [(4, 8), (8, 4), (5, 9), (10, 64), (64, 10), (3, 4096), (4096, 3), (1, 7), (7, 1), (2, 40000)])
@pytest.mark.parametrize("step", [0, 1, 2, "K"])
def test_rows_that_overlap(dt, R, K, step):
    dev, dtype = device(), TYPES[dt]
    step = K if step == "K" else step
    note(f"overlapping rows R={R} K={K} step={step} {dt}")
    line = randn(R + K + step, (R - 1) * step + K).to(dtype).to(dev)
    x = line.as_strided((R, K), (step, 1))
    other = randn(1, R, K).to(dtype).to(dev)
    w = (1 + 0.3 * randn(2, K)).to(dtype).to(dev)
    plain = x.contiguous()
    same(wq.quantize_rows(x), wq.quantize_rows(plain))
    same(wq.quantize_rows(x, gate=other), wq.quantize_rows(plain, gate=other))
    same(wq.quantize_rows(other, gate=x), wq.quantize_rows(other, gate=plain))
    for fn in (wq.rmsnorm_quantize, wq.rmsnorm):
        same(fn(x, w), fn(plain, w))
        same(fn(x, w, residual=other), fn(plain, w, residual=other))
        same(fn(other, w, residual=x), fn(other, w, residual=plain))
        same(fn(x, w, residual=x), fn(plain, w, residual=plain))
