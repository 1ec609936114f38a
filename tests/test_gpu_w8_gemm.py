"""GPU product of 8-bit activations and weights, bit for bit: the sum is exact in
int32 and each fp32 step after it is rounded by itself, so the oracle's bits are
the only right ones, whatever the kernel, the split of K or the workspace."""

import numpy as np
import pytest

import w8_util
from gpu_util import device, note, to_dev
from w8_util import TYPES, bits

import bit_weight_only_wq_amd as wq

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def inputs(B, K, N, dt, bias, seed=0):
    rng = np.random.default_rng(seed + B * 31 + K * 7 + N)
    a = rng.integers(-128, 128, (B, K)).astype(np.int8)
    w = rng.integers(-128, 128, (N, K)).astype(np.int8)
    sa = rng.uniform(0.005, 0.03, B).astype(np.float32)
    sw = rng.uniform(1e-4, 1e-3, N).astype(np.float32)
    b = torch.from_numpy(rng.standard_normal(N).astype(np.float32)).to(TYPES[dt]) if bias else None
    return a, sa, w, sw, b


def check(B, K, N, dt, bias, **kw):
    a, sa, w, sw, b = inputs(B, K, N, dt, bias)
    want = w8_util.product(a, sa, w, sw, b, TYPES[dt])
    dev = [to_dev(v) for v in (a, sa, w, sw)]
    bd = b.to(device()) if bias else None
    for use in (True, False):
        note(f"gemm_w8a8 B={B} K={K} N={N} {dt} bias={bias} workspace={use}")
        got = wq.gemm_w8a8(*dev, bias=bd, dtype=TYPES[dt], use_workspace=use, **kw)
        bad = (bits(got) != bits(want)).nonzero()
        assert not len(bad), (len(bad), bad[0].tolist(), got.cpu()[tuple(bad[0])], want[tuple(bad[0])])


# Batches from one row up, on both sides of 16, 32, 64, 128 and 256; K from one
# chunk, around steps of 64, 128 and 256; N odd, small, wide.
@pytest.mark.parametrize("B", [1, 2, 3, 8, 15, 16, 17, 31, 32, 33, 48, 64, 65, 100, 128, 129, 255, 256, 257, 300])
@pytest.mark.parametrize("K,N", [(16, 1), (48, 17), (64, 64), (80, 130), (128, 33), (256, 256), (400, 300), (1040, 129)])
def test_small_products(B, K, N):
    device()
    check(B, K, N, "fp16" if (B + N) % 2 else "bf16", (B + K // 16) % 3 == 0)


@pytest.mark.parametrize("B,K,N", [
    (1, 4096, 4096), (1, 11008, 4096), (2, 8192, 1024), (5, 4096, 11008), (16, 8192, 1000), (33, 896, 4864),
    (48, 8192, 777), (64, 4096, 4096), (65, 11008, 512), (128, 8192, 257), (200, 2064, 4096), (333, 11008, 1031),
    (512, 4096, 1024), (700, 1008, 1500), (1025, 512, 1030), (64, 131056, 40), (300, 65536, 129)])
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_models_products(B, K, N, dt):
    device()
    check(B, K, N, dt, N % 2 == 1)


# Sizes past what one workgroup a compute unit covers, for every kind of tile:
# few rows on wide matrices, splits of a long K, workgroups that take several
# tiles (one step of K, an odd number of steps, a last step that is not whole).
@pytest.mark.parametrize("B,K,N", [
    (20, 304, 16500), (32, 512, 16640), (7, 1040, 9000), (60, 304, 16501), (49, 640, 9000), (40, 8192, 5200),
    (700, 8208, 3000), (500, 8208, 2050), (130, 4112, 8200), (1025, 272, 8200), (2300, 272, 8200), (2300, 96, 8200),
    (4300, 272, 8200), (4300, 112, 8195), (4300, 400, 8192), (300, 16, 20000), (20000, 16, 300), (20000, 144, 17),
    (1100, 304, 2050), (2100, 1168, 2052), (600, 28672, 2050),
    # (two groups of waves: parts of K that are not equally long)
    (3, 2064, 3000), (16, 4240, 1030), (25, 2192, 2000), (50, 2320, 2000), (100, 2192, 1500), (200, 2320, 4100), (9, 6032, 700)])
@pytest.mark.parametrize("dt,bias", [("fp16", False), ("bf16", True)])
def test_many_tiles(B, K, N, dt, bias):
    device()
    check(B, K, N, dt, bias)


@pytest.mark.parametrize("B,K,N", [(1, 131056, 33), (20, 131056, 65), (300, 131056, 129)])
def test_largest_sums(B, K, N):
    """All of -128 * -128 (and of 127 * -128) over the longest K: just inside int32."""
    dev = device()
    note(f"largest sums B={B} N={N}")
    a = torch.full((B, K), -128, dtype=torch.int8, device=dev)
    w = torch.full((N, K), -128, dtype=torch.int8, device=dev)
    w[1::2] = 127
    one = torch.full((max(B, N),), 2.0 ** -10, dtype=torch.float32, device=dev)
    y = wq.gemm_w8a8(a, one[:B], w, one[:N], dtype=torch.bfloat16).float().cpu()
    top = torch.tensor([128.0 * 128 * K, -128.0 * 127 * K]) * 2.0 ** -20
    want = top.bfloat16().float().repeat(N)[:N].expand(B, N)
    assert torch.equal(y, want)


@pytest.mark.parametrize("B,K,N", [(1, 256, 100), (20, 512, 65), (70, 144, 200), (300, 1040, 257)])
def test_strided_operands(B, K, N):
    """Rows of a and w inside wider rows whose other bytes are not read, Y inside
    a buffer whose other values stay, at even and odd strides and offsets."""
    dev = device()
    a, sa, w, sw, b = inputs(B, K, N, "fp16", True)
    want = w8_util.product(a, sa, w, sw, b, torch.float16)
    wide_a = torch.full((B, K + 48), 77, dtype=torch.int8, device=dev)
    wide_w = torch.full((N, K + 160), -77, dtype=torch.int8, device=dev)
    wide_a[:, 16:16 + K], wide_w[:, 32:32 + K] = to_dev(a), to_dev(w)
    for pad in (8, 7):
        note(f"strided B={B} K={K} N={N} pad={pad}")
        buf = torch.full((B + 2, N + 2 * pad), 9.0, dtype=torch.float16, device=dev)
        out = buf[1:-1, pad:pad + N]
        got = wq.gemm_w8a8(wide_a[:, 16:16 + K], to_dev(sa), wide_w[:, 32:32 + K], to_dev(sw), bias=b.to(dev), out=out)
        assert got is out and torch.equal(bits(out), bits(want))
        buf[1:-1, pad:pad + N] = 9.0
        assert (buf == 9.0).all()


@pytest.mark.parametrize("B", [1, 40, 300])
def test_scales_that_are_not_finite(B):
    """A row of activations that could not be quantized (scale NaN) makes its own
    row of Y NaN and no other; a sum of zero stays zero; fp16 overflows to infinity."""
    dev = device()
    K, N = 512, 96
    a, sa, w, sw, _ = inputs(B, K, N, "fp16", False)
    a[0], sa[0] = 0, np.nan
    sw[5] = 1e3
    w[7] = 0
    want = w8_util.product(a, sa, w, sw, None, torch.float16)
    note(f"not finite B={B}")
    y = wq.gemm_w8a8(to_dev(a), to_dev(sa), to_dev(w), to_dev(sw)).cpu()
    assert torch.isnan(y[0]).all()
    assert torch.equal(bits(y[1:]), bits(want[1:]))
    assert B == 1 or (torch.isinf(y[1:, 5]).any() and not y[1:, 7].any())


def test_rows_do_not_depend_on_the_batch():
    dev = device()
    B, K, N = 300, 4096, 1024
    a, sa, w, sw, _ = inputs(B, K, N, "bf16", False)
    ad, sd, wd, swd = (to_dev(v) for v in (a, sa, w, sw))
    whole = wq.gemm_w8a8(ad, sd, wd, swd, dtype=torch.bfloat16)
    for lo, n in ((0, 1), (7, 5), (100, 16), (30, 40), (10, 100), (1, 299)):
        note(f"part {lo} {n}")
        part = wq.gemm_w8a8(ad[lo:lo + n], sd[lo:lo + n], wd, swd, dtype=torch.bfloat16)
        assert torch.equal(bits(part), bits(whole[lo:lo + n])), (lo, n)
    assert dev == ad.device


def test_wide_strides():
    """Operands and Y whose rows lie megabytes apart, offsets past 2^31 bytes."""
    dev = device()
    B, K, N = 1100, 64, 1040
    a, sa, w, sw, _ = inputs(B, K, N, "fp16", False)
    want = w8_util.product(a, sa, w, sw, None, torch.float16)
    step = 1 << 21
    buf = torch.zeros(B * step, dtype=torch.int8, device=dev)
    wbuf = torch.zeros(N * step, dtype=torch.int8, device=dev)
    av, wv = buf.view(B, step)[:, :K], wbuf.view(N, step)[:, step - K:]
    av.copy_(to_dev(a))
    wv.copy_(to_dev(w))
    y = torch.zeros((B, step), dtype=torch.float16, device=dev)[:, 5:5 + N]
    note("wide strides")
    got = wq.gemm_w8a8(av, to_dev(sa), wv, to_dev(sw), out=y)
    assert torch.equal(bits(got), bits(want))


def test_codes_of_the_symmetric_packer():
    """8-bit codes of quantize_pack (scheme sym, one group a row) serve as weights:
    top bit flipped, scales widened."""
    dev = device()
    g = torch.Generator().manual_seed(3)
    W = (torch.randn((96, 512), generator=g) * 0.02).half().to(dev)
    X = torch.randn((5, 512), generator=g).half().to(dev)
    codes, scales, _ = wq.quantize_pack(W, group=512, bits=8, scheme="sym")
    w, sw = (codes ^ 128).view(torch.int8), scales.float()[:, 0]
    a, sa = wq.quantize_rows(X)
    note("packer's codes")
    y = wq.gemm_w8a8(a, sa, w, sw.contiguous())
    want = w8_util.product(a.cpu().numpy(), sa.cpu().numpy(), w.cpu().numpy(), sw.cpu().numpy(), None, torch.float16)
    assert torch.equal(bits(y), bits(want))


def test_empty_and_refused():
    dev = device()
    i8 = torch.int8
    a, w = torch.zeros((4, 64), dtype=i8, device=dev), torch.zeros((32, 64), dtype=i8, device=dev)
    sa, sw = torch.ones(4, device=dev), torch.ones(32, device=dev)
    assert wq.gemm_w8a8(a[:0], sa[:0], w, sw).shape == (0, 32)
    assert wq.gemm_w8a8(a, sa, w[:0], sw[:0]).shape == (4, 0)
    buf = torch.zeros((4, 128), dtype=torch.float16, device=dev)
    for bad in [lambda: wq.gemm_w8a8(a.view(torch.uint8), sa, w, sw), lambda: wq.gemm_w8a8(a, sa, w[:, :32], sw),
                lambda: wq.gemm_w8a8(a, sa[:3], w, sw), lambda: wq.gemm_w8a8(a, sa, w, sw.half()),
                lambda: wq.gemm_w8a8(a, sa, w, sw, dtype=torch.float32), lambda: wq.gemm_w8a8(a.t(), sa, w, sw),
                lambda: wq.gemm_w8a8(a, sa, w, sw, bias=sw), lambda: wq.gemm_w8a8(a, sa, w, sw, out=buf),
                lambda: wq.gemm_w8a8(a, sa, w, sw, bias=sw.half(), dtype=torch.bfloat16),
                lambda: wq.gemm_w8a8(a, sa, w, sw, workspace=torch.zeros(64, device=dev)),
                lambda: wq.gemm_w8a8(buf.view(i8)[:, :64], sa, w, sw, out=buf[:, :32]),
                lambda: wq.gemm_w8a8(a, sa.cpu(), w, sw), lambda: wq.gemm_w8a8(a.cpu(), sa.cpu(), w.cpu(), sw.cpu())]:
        with pytest.raises(ValueError):
            bad()
    for bad in [lambda: wq.gemm_w8a8(a[:, :40], sa, w[:, :40], sw),              # K no multiple of 16
                lambda: wq.gemm_w8a8(a[:, 8:56], sa, w[:, 8:56], sw)]:           # rows not aligned
        with pytest.raises(wq.WQError):
            bad()


def test_streams_and_graph():
    """Two calls at once on two streams, each with a workspace of its own, and
    captured calls replayed over changed inputs."""
    dev = device()
    shapes = [(20, 8192, 512), (1, 4096, 1024), (300, 4096, 512)]
    data = []
    for B, K, N in shapes:
        a, sa, w, sw, _ = inputs(B, K, N, "fp16", False)
        data.append([to_dev(v) for v in (a, sa, w, sw)] + [torch.empty((B, N), dtype=torch.float16, device=dev),
                                                          wq.gemm_w8a8_workspace(B, N, K)])
    streams = [torch.cuda.Stream() for _ in data]
    torch.cuda.synchronize()
    note("gemm on three streams")
    for _ in range(3):
        for s, (a, sa, w, sw, y, ws) in zip(streams, data):
            with torch.cuda.stream(s):
                wq.gemm_w8a8(a, sa, w, sw, out=y, workspace=ws)
    torch.cuda.synchronize()
    for a, sa, w, sw, y, ws in data:
        assert torch.equal(y, wq.gemm_w8a8(a, sa, w, sw))
    graph = torch.cuda.CUDAGraph()
    note("gemm captured")
    with torch.cuda.graph(graph):
        for a, sa, w, sw, y, ws in data:
            wq.gemm_w8a8(a, sa, w, sw, out=y, workspace=ws)
    for i in range(4):
        for a, sa, w, sw, y, ws in data:
            a.copy_(torch.randint(-128, 128, a.shape, dtype=torch.int8, device=dev))
        want = [wq.gemm_w8a8(a, sa, w, sw) for a, sa, w, sw, y, ws in data]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for (a, sa, w, sw, y, ws), ref in zip(data, want):
            assert torch.equal(y, ref), i
