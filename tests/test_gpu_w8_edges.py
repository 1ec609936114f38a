"""GPU tests of the 8-bit path at the ends of what it takes: inputs whose rows
repeat or overlap, bf16 products past fp32's range on either side, streams.

Tolerances as in test_gpu_w8_rows: a scale of quantize_rows within 2^-22, of the
norm within 2^-21, values half a step of their type and 2^-22."""

import numpy as np
import pytest

import w8_util
from gpu_util import device, note
import test_gpu_w8_rows as rows_tests
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


def odd_norm_rows(K, seed):
    """bf16 rows h and weights w whose products leave what fp32 holds exactly, on
    either side: past its largest, below its smallest normal, below its smallest, of
    mixed sizes, rows of zeros and ordinary ones between them."""
    h = randn(seed, 8, K)
    h[0] *= 2.0 ** 125                                       # h w past fp32 where w > 2
    h[1] *= 3e-24
    h[2] *= 2.0 ** -100
    h[3] *= torch.exp2(torch.linspace(-120, 0, K))           # a few large, most tiny
    h[4] = 0.0
    h[5] = 0.0
    h[5, K // 2] = 2.0 ** 126
    h[7, ::2] = 0.0
    return h.bfloat16()


WEIGHTS = {"large": 8.0, "tiny": 1e-18, "least": 2.0 ** -60, "ordinary": 1.0}


@pytest.mark.parametrize("K", [1, 7, 64, 1000, 2048, 5000, 8192, 12288, 16384, 20000, 32768, 40000])
@pytest.mark.parametrize("size", list(WEIGHTS))
@pytest.mark.parametrize("residual", [False, True])
def test_values_past_fp32_products(K, size, residual):
    """The norm's values where h w is no fp32 number but h w / rms is a bf16 one."""
    dev = device()
    note(f"norm values, products past fp32, K={K} {size} residual={residual}")
    h = odd_norm_rows(K, K)
    w = (WEIGHTS[size] * (1 + 0.3 * randn(K + 1, K))).bfloat16()
    res = None
    if residual:
        h = h / 2                                            # (the sum is what h was)
        res = h.clone()
    for eps in (1e-6, 2.0 ** -126):
        y, _, _, total = w8_util.norm(h, w, res, eps)
        got, t = wq.rmsnorm(h.to(dev), w.to(dev), residual=res.to(dev) if residual else None, eps=eps)
        assert np.isfinite(y).all() and np.abs(y).max() < 3e38
        check_values(got, y, torch.bfloat16, (K, size, eps))
        assert not residual or torch.equal(bits(t), bits(total))


@pytest.mark.parametrize("K", [1, 7, 64, 1000, 2048, 5000, 8192, 12288, 16384, 20000, 32768, 40000])
@pytest.mark.parametrize("size", ["tiny", "least", "ordinary"])
@pytest.mark.parametrize("residual", [False, True])
def test_codes_of_products_below_fp32(K, size, residual):
    """The norm's codes where a row's largest h w is subnormal in fp32, or nothing."""
    dev = device()
    note(f"norm codes, products below fp32, K={K} {size} residual={residual}")
    h = odd_norm_rows(K, K)
    w = (WEIGHTS[size] * (1 + 0.3 * randn(K + 1, K))).bfloat16()
    res = None
    if residual:
        h = h / 2
        res = h.clone()
    for eps in (1e-6, 2.0 ** -126):
        _, codes, scales, total = w8_util.norm(h, w, res, eps)
        c, s, t = wq.rmsnorm_quantize(h.to(dev), w.to(dev), residual=res.to(dev) if residual else None, eps=eps)
        bad = np.argwhere(c.cpu().numpy() != codes)
        assert not len(bad), (len(bad), bad[0], c.cpu().numpy()[tuple(bad[0])], codes[tuple(bad[0])])
        # A scale below fp32's smallest normal number: half a step of its own, and the same again for a product before it.
        got = s.cpu().numpy().astype(np.float64)
        assert np.all(np.abs(got - scales) <= np.maximum(2.0 ** -21 * scales, 2.0 ** -149)), (got, scales)
        assert not residual or torch.equal(bits(t), bits(total))


def test_codes_next_to_a_border_below_fp32():
    """127 t / max is 89.228 where the products themselves, rounded to fp32, give 89.243."""
    dev = device()
    h = torch.tensor([[3.0e-24, 2.1e-24] + [0.0] * 6]).bfloat16()
    w = torch.full((8,), 1e-18).bfloat16()
    rng = np.random.default_rng(5)
    many = torch.from_numpy(rng.uniform(-3e-24, 3e-24, (64, 2048)).astype(np.float32)).bfloat16()
    note("codes next to a border below fp32")
    for x, wt in ((h, w), (many, w[:1].repeat(2048))):
        _, codes, scales, _ = w8_util.norm(x, wt, None, 2.0 ** -126)
        c, s, _ = wq.rmsnorm_quantize(x.to(dev), wt.to(dev), eps=2.0 ** -126)
        check_codes(c, s, codes, scales, 2.0 ** -21, "codes")


@pytest.mark.parametrize("K", [1024, 2000, 8192, 20000, 40000])
def test_scale_of_a_lone_large_value(K):
    """Rows of zeros but for one place: r max is sqrt(K) w there, past fp32, and a
    127th of it is not."""
    dev = device()
    h = torch.zeros((6, K), dtype=torch.bfloat16)
    w = torch.ones(K, dtype=torch.bfloat16)
    for i, (value, weight) in enumerate(((4.0, 2.0 ** 125), (2.0 ** -3, 2.0 ** 127), (1.0, -(2.0 ** 127)), (-3.0, 2.0 ** 126),
                                         (2.0 ** 60, 2.0 ** 67), (1.0, 1.0))):
        h[i, 7 * i], w[7 * i] = value, weight
    note(f"scale of a lone large value K={K}")
    _, codes, scales, _ = w8_util.norm(h, w, None, 1e-6)
    assert np.isfinite(scales.astype(np.float32)).all() and scales.max() * 127 > 3.5e38
    c, s, _ = wq.rmsnorm_quantize(h.to(dev), w.to(dev))
    check_codes(c, s, codes, scales, 2.0 ** -21, K)


def test_workspace_beside_the_operands():
    """A workspace right between a and w of one buffer, and right behind Y, is used; over
    them it is refused."""
    dev = device()
    B, K, N = 48, 8192, 1024
    n = wq.gemm_w8a8_workspace(B, N, K).numel()
    assert n > 0 and n % 16 == 0
    y_bytes = 2 * B * N
    buf = torch.empty(B * K + n + N * K + y_bytes + n, dtype=torch.uint8, device=dev)
    a = buf[:B * K].view(torch.int8).view(B, K)
    ws = buf[B * K:B * K + n]
    w = buf[B * K + n:B * K + n + N * K].view(torch.int8).view(N, K)
    y = buf[B * K + n + N * K:][:y_bytes].view(torch.float16).view(B, N)
    ws2 = buf[-n:]
    rng = np.random.default_rng(1)
    ha, hw = rng.integers(-128, 128, (B, K)).astype(np.int8), rng.integers(-128, 128, (N, K)).astype(np.int8)
    sa, sw = torch.full((B,), 2.0 ** -7, device=dev), torch.full((N,), 2.0 ** -9, device=dev)
    a.copy_(torch.from_numpy(ha))
    w.copy_(torch.from_numpy(hw))
    want = w8_util.product(ha, sa.cpu().numpy(), hw, sw.cpu().numpy(), None, torch.float16)
    for space in (ws, ws2):
        note("workspace beside the operands")
        y.zero_()
        wq.gemm_w8a8(a, sa, w, sw, out=y, workspace=space)
        assert torch.equal(bits(y), bits(want))
        assert (a.cpu().numpy() == ha).all() and (w.cpu().numpy() == hw).all()
    for lo in (0, B * K - 16, B * K + 16, B * K + n + N * K - 16, buf.numel() - n - 16):
        with pytest.raises(wq.WQError):
            wq.gemm_w8a8(a, sa, w, sw, out=y, workspace=buf[lo:lo + n])


@pytest.mark.parametrize("eps", [2.0 ** -126, 3.4028234663852886e38])
def test_eps_at_its_ends(eps):
    dev = device()
    x, w = randn(1, 5, 1000).bfloat16(), (1 + 0.3 * randn(2, 1000)).bfloat16()
    y, codes, scales, _ = w8_util.norm(x, w, None, eps)
    note(f"eps {eps}")
    check_values(wq.rmsnorm(x.to(dev), w.to(dev), eps=eps)[0], y, torch.bfloat16, "values")
    check_codes(*wq.rmsnorm_quantize(x.to(dev), w.to(dev), eps=eps)[:2], codes, scales, 2.0 ** -21, "codes")


# Both ends of every class of widths that a row's threads and vectors are chosen by,
# where the sizes of test_gpu_w8_rows have a gap.
WIDTHS = [(3, 511), (3, 513), (3, 1023), (5, 1024), (3, 1025), (4, 1536), (3, 2047), (5, 2048), (3, 2049), (2, 4095), (2, 6143),
          (2, 8191), (2, 8193), (2, 12287), (2, 16383), (2, 24575), (2, 32767), (2, 32769)]


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("R,K", WIDTHS)
@pytest.mark.parametrize("gate", [False, True])
def test_rows_at_the_widths_ends(R, K, dt, gate):
    rows_tests.test_rows_match_definition(R, K, dt, gate)


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("R,K", WIDTHS)
@pytest.mark.parametrize("residual", [False, True])
def test_norms_at_the_widths_ends(R, K, dt, residual):
    rows_tests.test_norms_match_definition(R, K, dt, residual)


def test_calls_follow_their_stream():
    """Inputs that a stream of its own writes late: every call on it waits for them, as a
    launch on another stream would not."""
    dev, side = device(), torch.cuda.Stream()
    R, K, N = 6, 4096, 256
    busy = torch.zeros((4096, 4096), dtype=torch.float16, device=dev)
    new_x, new_r = randn(1, R, K).half(), randn(2, R, K).half()
    x, r = torch.zeros((R, K), dtype=torch.float16, device=dev), torch.zeros((R, K), dtype=torch.float16, device=dev)
    from_x, from_r = new_x.to(dev), new_r.to(dev)
    w = (1 + 0.3 * randn(3, K)).half()
    wd = w.to(dev)
    mat, mat_scales = wq.quantize_rows((0.02 * randn(4, N, K)).half().to(dev))
    torch.mm(busy, busy)
    torch.cuda.synchronize()
    note("calls on a stream of their own")
    with torch.cuda.stream(side):
        for _ in range(100):
            torch.mm(busy, busy)
        x.copy_(from_x)
        r.copy_(from_r)
        codes, scales, total = wq.rmsnorm_quantize(x, wd, residual=r)
        values, total2 = wq.rmsnorm(x, wd, residual=r)
        c2, s2 = wq.quantize_rows(total, gate=x)
        y = wq.gemm_w8a8(codes, scales, mat, mat_scales)
    side.synchronize()
    want, want_codes, want_scales, h = w8_util.norm(new_x, w, new_r, 1e-6)
    check_codes(codes, scales, want_codes, want_scales, 2.0 ** -21, "codes")
    check_values(values, want, torch.float16, "values")
    assert torch.equal(bits(total), bits(h)) and torch.equal(bits(total2), bits(h))
    check_codes(c2, s2, *w8_util.rows(h, new_x), 2.0 ** -22, "gated")
    product = w8_util.product(codes.cpu().numpy(), scales.cpu().numpy(), mat.cpu().numpy(), mat_scales.cpu().numpy(), None,
                              torch.float16)
    assert torch.equal(bits(y), bits(product))


@pytest.mark.parametrize("K", [64, 2048, 11008, 28672, 40000])
def test_gates_below_the_smallest_normal(K):
    """bf16 gates that are subnormal, times values so large that the products are ordinary
    numbers: every code as the exact quotient decides it."""
    dev = device()
    rng = np.random.default_rng(K)
    g = (rng.integers(-127, 128, (6, K)) * 2.0 ** -133).astype(np.float32)
    g = torch.from_numpy(g).bfloat16()
    x = randn(K, 6, K) * 2.0 ** 90
    x[1] = 2.0 ** 75 * randn(K + 1, K)
    x[2] = 2.0 ** 120
    x[3] *= 2.0 ** -80
    g[4] *= 2.0 ** 4
    g[5, ::2] = 3.0
    x[5, ::2] = 2.0 ** -44
    x = x.bfloat16()
    note(f"subnormal gates K={K}")
    codes, scales = wq.quantize_rows(x.to(dev), gate=g.to(dev))
    check_codes(codes, scales, *w8_util.rows(x, g), 2.0 ** -22, K)
