"""GPU rows to 8 bits and the root-mean-square norm against their definitions in
float64: codes exactly, scales and values within counted roundings.

Tolerances.  A scale of quantize_rows is max|t| / 127 rounded, where fp32's max|t|
may itself be rounded: 2 * 2^-24, taken as 2^-22.  The norm's factor r takes a
division, a square root and a conversion in fp32 at most (mean and sum in 64
bits), its scale two more steps: under 6 * 2^-24, taken as 2^-21.  A value is t
(exact) times r, under 2^-22 together, then rounded to its type: half a step of
the type relative, or half of its smallest subnormal."""

import numpy as np
import pytest

import w8_util
from gpu_util import device, note
from w8_util import TYPES, bits, half_step

import bit_weight_only_wq_amd as wq

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# rows, K: lengths from one value up, odd ones, those at and past what one wave
# (512 values a step) or one workgroup holds, models' widths.
SIZES = [(1, 1), (3, 2), (2, 7), (5, 8), (4, 9), (3, 63), (9, 64), (7, 100), (1, 512), (6, 520), (33, 896), (5, 1000),
         (1, 4096), (17, 4096), (3, 4100), (2, 4104), (1, 4864), (3, 5000), (1, 8192), (9, 8192), (2, 8200), (1, 11008),
         (3, 11008), (2, 16384), (1, 20001), (2, 28672), (1, 32768), (2, 32776), (1, 70000), (1, 131077),
         (2, 4097), (2, 6144), (2, 6145), (2, 12288), (2, 12289), (2, 16385), (2, 24576), (2, 24577)]


def randn(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed))


def check_codes(codes, scales, want_codes, want_scales, rel, what):
    got = codes.cpu().numpy()
    bad = np.argwhere(got != want_codes)
    assert not len(bad), (what, len(bad), bad[0], got[tuple(bad[0])], want_codes[tuple(bad[0])])
    s = scales.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(s - want_scales) <= rel * want_scales), (what, np.max(np.abs(s / want_scales - 1)))


def check_values(y, want, dtype, what):
    d = np.abs(w8_util.f64(y.cpu()) - want)
    # (the smallest subnormal's half: that of the type's exponent range)
    tiny = float(torch.finfo(dtype).smallest_normal) * half_step(dtype)
    bound = np.abs(want) * (half_step(dtype) * (1 + 2.0 ** -10) + 2.0 ** -22) + tiny * (1 + 2.0 ** -10)
    assert np.all(d <= bound), (what, np.max(d / bound))


def guarded(rows, width, dtype, fill, pad=24):
    """A [rows, width] view inside a filled buffer, and the buffer."""
    buf = torch.full((rows + 2, width + 2 * pad), fill, dtype=dtype, device=device())
    return buf[1:-1, pad:pad + width], buf


def outside_kept(view, buf, fill, pad=24):
    keep = buf.clone()
    keep[1:-1, pad:buf.shape[1] - pad] = fill
    return bool((keep == fill).all())


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("R,K", SIZES)
@pytest.mark.parametrize("gate", [False, True])
def test_rows_match_definition(R, K, dt, gate):
    dev = device()
    note(f"quantize_rows R={R} K={K} {dt} gate={gate}")
    packed = randn(R * 1000 + K, R, 2 * K).to(TYPES[dt])
    packed[0, K // 2] = 0.0
    g, x = (packed[:, :K], packed[:, K:]) if gate else (None, packed[:, K:])
    on = packed.to(dev)
    codes, scales = wq.quantize_rows(on[:, K:], on[:, :K] if gate else None)
    check_codes(codes, scales, *w8_util.rows(x, g), 2.0 ** -22, "packed halves")
    # Into strided rows of a guarded buffer, from tensors of their own.
    out, buf = guarded(R, K, torch.int8, 99)
    s = torch.empty(R, dtype=torch.float32, device=dev)
    got = wq.quantize_rows(x.contiguous().to(dev), g.contiguous().to(dev) if gate else None, out=(out, s))
    assert got[0] is out and got[1] is s
    assert torch.equal(out, codes) and torch.equal(s, scales) and outside_kept(out, buf, 99)
    assert torch.equal(bits(on), bits(packed))


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("R,K", SIZES)
@pytest.mark.parametrize("residual", [False, True])
def test_norms_match_definition(R, K, dt, residual):
    dev, dtype = device(), TYPES[dt]
    note(f"rmsnorm R={R} K={K} {dt} residual={residual}")
    x, w = randn(R + K, R, K).to(dtype), (1 + 0.3 * randn(K, K)).to(dtype)
    res = (5 * randn(R + K + 1, R, K)).to(dtype) if residual else None
    y, codes, scales, h = w8_util.norm(x, w, res, 1e-5)
    xd, wd, rd = x.to(dev), w.to(dev), res.to(dev) if residual else None
    c, s, t = wq.rmsnorm_quantize(xd, wd, residual=rd, eps=1e-5)
    check_codes(c, s, codes, scales, 2.0 ** -21, "codes")
    v, t2 = wq.rmsnorm(xd, wd, residual=rd, eps=1e-5)
    check_values(v, y, dtype, "values")
    if not residual:
        assert t is None and t2 is None
        return
    assert torch.equal(bits(t), bits(h)) and torch.equal(bits(t2), bits(h))
    assert torch.equal(bits(xd), bits(x)) and torch.equal(bits(rd), bits(res))
    # total written over the residual, over x, and into strided rows.
    rr, xx = rd.clone(), xd.clone()
    c2, s2, t = wq.rmsnorm_quantize(xd, wd, residual=rr, eps=1e-5, total=rr)
    assert t is rr and torch.equal(bits(rr), bits(h)) and torch.equal(c2, c) and torch.equal(s2, s)
    v2, t = wq.rmsnorm(xx, wd, residual=rd, eps=1e-5, total=xx)
    assert t is xx and torch.equal(bits(xx), bits(h)) and torch.equal(bits(v2), bits(v))
    out, buf = guarded(R, K, dtype, -3.0)
    tot, tbuf = guarded(R, K, dtype, 7.0)
    xs, xbuf = guarded(R, K, dtype, 1.0, pad=9)
    xs.copy_(xd)
    wq.rmsnorm(xs, wd, residual=rd, eps=1e-5, total=tot, out=out)
    assert torch.equal(bits(out), bits(v)) and torch.equal(bits(tot), bits(h))
    assert outside_kept(out, buf, -3.0) and outside_kept(tot, tbuf, 7.0)
    cs, cbuf = guarded(R, K, torch.int8, 99, pad=9)
    wq.rmsnorm_quantize(xs, wd, residual=rd, eps=1e-5, total=tot, out=(cs, s2))
    assert torch.equal(cs, c) and torch.equal(s2, s) and outside_kept(cs, cbuf, 99, pad=9)


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("K", [256, 2048, 8192, 12288, 40000])
def test_ties_and_borders(dt, K):
    """Rows full of values on the border between two codes (odd halves of max /
    127, max = 127 times a power of two) and of the 16-bit values next to them."""
    dev, dtype = device(), TYPES[dt]
    note(f"ties K={K} {dt}")
    span = 64 if dt == "fp16" else 16                     # halves up to here are 16-bit values
    rng = np.random.default_rng(K)
    rows = []
    for e in (-6, 0, 3):
        t = torch.from_numpy(rng.integers(-2 * span, 2 * span, K).astype(np.float32) / 2 * 2.0 ** e).to(dtype)
        near = (bits(t).numpy().view(np.uint16) + rng.integers(-1, 2, K)).astype(np.uint16)
        near = torch.from_numpy(near.view(np.int16)).view(dtype)
        near = torch.where(near.abs() < 127 * 2.0 ** e, near, t)
        t[K // 3] = near[K // 3] = 127 * 2.0 ** e
        rows += [t, near]
    x = torch.stack(rows)
    codes, scales = wq.quantize_rows(x.to(dev))
    check_codes(codes, scales, *w8_util.rows(x, None), 2.0 ** -22, "rows")
    w = torch.ones(K, dtype=dtype)
    w[::3] = 2.0
    w[K // 3] = 4.0 if dt == "bf16" else 2.0
    _, want, ws, _ = w8_util.norm(x, w, None, 1e-6)
    c, s, _ = wq.rmsnorm_quantize(x.to(dev), w.to(dev), eps=1e-6)
    check_codes(c, s, want, ws, 2.0 ** -21, "norm")


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_many_random_codes(dt):
    """Eight million codes of each kind: some hundreds lie within fp32's error of
    a border."""
    dev, dtype = device(), TYPES[dt]
    note(f"many codes {dt}")
    R, K = 1024, 8192
    g, x = randn(1, R, K).to(dtype), randn(2, R, K).to(dtype)
    check_codes(*wq.quantize_rows(x.to(dev)), *w8_util.rows(x, None), 2.0 ** -22, "plain")
    check_codes(*wq.quantize_rows(x.to(dev), gate=(3 * g).to(dev)), *w8_util.rows(x, 3 * g), 2.0 ** -22, "gated")
    w = (1 + 0.3 * randn(3, K)).to(dtype)
    _, codes, scales, h = w8_util.norm(x, w, g, 1e-6)
    c, s, t = wq.rmsnorm_quantize(x.to(dev), w.to(dev), residual=g.to(dev))
    check_codes(c, s, codes, scales, 2.0 ** -21, "norm")
    assert torch.equal(bits(t), bits(h))


@pytest.mark.parametrize("K", [5, 64, 4096, 12288, 33000])
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_special_rows(dt, K):
    """Zeros, a single value, the smallest and largest of the type, infinities and
    NaN, each in a row of its own among ordinary rows."""
    dev, dtype = device(), TYPES[dt]
    note(f"special rows K={K} {dt}")
    big, tiny = torch.finfo(dtype).max, float(torch.finfo(dtype).smallest_normal) * torch.finfo(dtype).eps
    x = randn(K, 12, K).to(dtype)
    x[1] = 0.0
    x[2] = 0.0
    x[2, K - 1] = -0.75
    x[3] = 0.0
    x[3, 0], x[3, K // 2] = tiny, -2 * tiny
    x[4, K // 2] = big
    x[5] = big
    x[6, K - 1] = float("inf")
    x[7, 0] = float("-inf")
    x[8, K // 2] = float("nan")
    x[9] = -0.0
    x[10] *= 2.0 ** -12
    bad = [6, 7, 8]
    good = [i for i in range(12) if i not in bad]
    w = torch.ones(K, dtype=dtype)
    xd = x.to(dev)
    for gate in (None, torch.full((12, K), 3.0, dtype=dtype)):
        codes, scales = wq.quantize_rows(xd, gate=gate.to(dev) if gate is not None else None)
        want, ws = w8_util.rows(x[good], gate[good] if gate is not None else None)
        fine = ws * 127 <= 3.4e38                          # bf16's largest times silu(3) is past fp32
        lost = [good[i] for i in np.flatnonzero(~fine)]
        keep = [good[i] for i in np.flatnonzero(fine)]
        normal = ws[fine] >= 2.0 ** -126                   # a subnormal scale has fewer bits
        assert np.array_equal(codes[keep].cpu().numpy(), want[fine])
        s = scales[keep].cpu().numpy().astype(np.float64)
        assert np.all(np.abs(s - ws[fine]) <= np.where(normal, 2.0 ** -22 * ws[fine], 2.0 ** -149))
        assert torch.isnan(scales[bad + lost]).all() and not codes[bad + lost].any()
    y, codes, scales, _ = w8_util.norm(x[good], w, None, 1e-6)
    c, s, _ = wq.rmsnorm_quantize(xd, w.to(dev))
    assert torch.isnan(s[bad]).all() and not c[bad].any()
    assert np.array_equal(c[good].cpu().numpy(), codes)
    normal = scales >= 2.0 ** -126
    s = s[good].cpu().numpy().astype(np.float64)
    assert np.all(np.abs(s - scales) <= np.where(normal, 2.0 ** -21 * scales, 2.0 ** -148))
    v, _ = wq.rmsnorm(xd, w.to(dev))
    check_values(v[good], y, dtype, "values")
    assert torch.isnan(v[8]).all() and torch.isnan(v[6, K - 1]) and torch.isnan(v[7, 0])
    assert not v[6, :K - 1].any() and not v[7, 1:].any()


def test_residual_past_the_type():
    """A sum past fp16's range is infinite in total, and its row says so."""
    dev = device()
    x = torch.full((2, 64), 60000.0, dtype=torch.float16, device=dev)
    x[1] = 1.0
    c, s, t = wq.rmsnorm_quantize(x, torch.ones(64, dtype=torch.float16, device=dev), residual=x)
    assert torch.isinf(t[0]).all() and torch.isnan(s[0]) and not c[0].any()
    assert (t[1] == 2).all() and (c[1] == 127).all()


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_far_gates(dt):
    """Gates from far below zero (where 1 + exp(-gate) is past fp32) to far above."""
    dev, dtype = device(), TYPES[dt]
    K = 2048
    g = torch.linspace(-110, 110, K).to(dtype).repeat(5, 1)
    x = randn(4, 5, K).to(dtype)
    g[1] = -100.0
    g[2] = -30.0
    g[3, :] = -700.0 if dt == "fp16" else -1e30
    g[4] = randn(5, K).to(dtype) * 12
    note(f"far gates {dt}")
    codes, scales = wq.quantize_rows(x.to(dev), gate=g.to(dev))
    keep = [0, 1, 2, 4]
    want, ws = w8_util.rows(x[keep], g[keep])
    assert np.array_equal(codes[keep].cpu().numpy(), want)
    s = scales[keep].cpu().numpy().astype(np.float64)
    assert np.all(np.abs(s - ws) <= np.maximum(2.0 ** -22 * ws, 2.0 ** -149))
    assert not codes[3].any() and scales[3] == 1.0          # 700 exp(-700) is below fp32


def test_large_norm_sums():
    """bf16 rows whose squares are past fp32."""
    dev = device()
    x = (randn(8, 3, 4096) * torch.tensor([[1e25], [1e-20], [1.0]])).bfloat16()
    w = torch.ones(4096, dtype=torch.bfloat16)
    y, codes, scales, _ = w8_util.norm(x, w, None, 2.0 ** -126)
    c, s, _ = wq.rmsnorm_quantize(x.to(dev), w.to(dev), eps=2.0 ** -126)
    check_codes(c, s, codes, scales, 2.0 ** -21, "codes")
    v, _ = wq.rmsnorm(x.to(dev), w.to(dev), eps=2.0 ** -126)
    check_values(v, y, torch.bfloat16, "values")


@pytest.mark.parametrize("K,pad", [(8, 0), (5, 3), (520, 0)])
def test_more_rows_than_a_launch(K, pad):
    """Rows on both sides of 2^20, where a second launch takes over, 16-byte form
    and not."""
    dev = device()
    R = (1 << 20) + 5
    note(f"many rows K={K}")
    g = torch.Generator(device=dev).manual_seed(K)
    x = torch.randn((R, K + pad), generator=g, device=dev).half()[:, :K]
    gate = torch.randn((R, K), generator=g, device=dev).half()
    w = torch.ones(K, dtype=torch.float16, device=dev)
    codes, scales = wq.quantize_rows(x, gate=gate)
    c, s, total = wq.rmsnorm_quantize(x, w, residual=gate)
    y, _ = wq.rmsnorm(x, w)
    for lo in (0, (1 << 20) - 4):
        part = slice(lo, lo + 9)
        hx, hg = x[part].cpu(), gate[part].cpu()
        check_codes(codes[part], scales[part], *w8_util.rows(hx, hg), 2.0 ** -22, "gated")
        _, want, ws, h = w8_util.norm(hx, w.cpu(), hg, 1e-6)
        check_codes(c[part], s[part], want, ws, 2.0 ** -21, "norm")
        assert torch.equal(bits(total[part]), bits(h))
        check_values(y[part], w8_util.norm(hx, w.cpu(), None, 1e-6)[0], torch.float16, "values")


def test_empty_and_refused():
    dev = device()
    f16 = torch.float16
    c, s = wq.quantize_rows(torch.zeros((0, 64), dtype=f16, device=dev))
    assert c.shape == (0, 64) and s.shape == (0,)
    x = torch.ones((4, 64), dtype=f16, device=dev)
    w = torch.ones(64, dtype=f16, device=dev)
    y, t = wq.rmsnorm(x[:0], w, residual=x[:0])
    assert y.shape == (0, 64) and t.shape == (0, 64)
    codes, scales = torch.empty((4, 64), dtype=torch.int8, device=dev), torch.empty(4, device=dev)
    packed = torch.ones((4, 128), dtype=f16, device=dev)
    for bad in [lambda: wq.quantize_rows(x.float()), lambda: wq.quantize_rows(x.cpu()), lambda: wq.quantize_rows(x[0]),
                lambda: wq.quantize_rows(x.t()), lambda: wq.quantize_rows(x, gate=x.bfloat16()),
                lambda: wq.quantize_rows(x, gate=x[:3]), lambda: wq.quantize_rows(x, out=(codes.view(torch.uint8), scales)),
                lambda: wq.quantize_rows(x, out=(codes[:3], scales)), lambda: wq.quantize_rows(x, out=(codes, scales[:3])),
                lambda: wq.quantize_rows(x, out=(x.view(torch.int8)[:, :64], scales)),
                lambda: wq.quantize_rows(x, out=(codes, codes.view(torch.float32).flatten()[:4])),
                lambda: wq.rmsnorm(x, w.bfloat16()), lambda: wq.rmsnorm(x, w[:63]), lambda: wq.rmsnorm(x, w, total=x),
                lambda: wq.rmsnorm(x, w, residual=x.bfloat16()), lambda: wq.rmsnorm(x, w, out=x),
                lambda: wq.rmsnorm(x, w, residual=packed[:, :64], total=packed[:, 32:96]),
                lambda: wq.rmsnorm(x, w, residual=x[:2].repeat(2, 1), total=w.expand(4, 64)),
                lambda: wq.rmsnorm(packed[:3, :64], w, residual=packed[:3, 64:], total=packed[1:, :64]),
                lambda: wq.rmsnorm_quantize(x, w, residual=x, total=packed[:, :64], out=(packed.view(torch.int8)[:, 64:128], scales))]:
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(wq.WQError):
        wq.rmsnorm(x, w, eps=0.0)
    # Halves of one packed row lie beside each other.
    y, t = wq.rmsnorm(packed[:, :64], w, residual=packed[:, 64:], total=packed[:, 64:])
    assert (packed[:, 64:] == 2).all() and (packed[:, :64] == 1).all() and (y == 1).all()


def test_other_stream_and_graph():
    """Calls on a stream of their own, and captured: every replay follows the
    inputs it finds."""
    dev = device()
    K = 4096
    x, r, w = randn(1, 6, K).half().to(dev), randn(2, 6, K).half().to(dev), torch.ones(K, dtype=torch.float16, device=dev)
    codes, scales = torch.empty((6, K), dtype=torch.int8, device=dev), torch.empty(6, device=dev)
    c2, s2 = torch.empty((6, K), dtype=torch.int8, device=dev), torch.empty(6, device=dev)
    total = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    note("rows on a stream and in a graph")
    with torch.cuda.stream(side):
        wq.rmsnorm_quantize(x, w, residual=r, total=total, out=(codes, scales))
        wq.quantize_rows(total, gate=x, out=(c2, s2))
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wq.rmsnorm_quantize(x, w, residual=r, total=total, out=(codes, scales))
        wq.quantize_rows(total, gate=x, out=(c2, s2))
    for i in range(4):
        x.copy_(randn(10 + i, 6, K))
        want = wq.rmsnorm_quantize(x, w, residual=r)
        want2 = wq.quantize_rows(want[2], gate=x)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for got, ref in ((codes, want[0]), (scales, want[1]), (total, want[2]), (c2, want2[0]), (s2, want2[1])):
            assert torch.equal(got, ref), i
