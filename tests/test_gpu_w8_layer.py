"""A decoder layer's 8-bit path as it is used, in one run: norm to codes, q/k/v
product, rotary positions, paged cache and its attention, codes of the
attention's output, output product, norm with the residual, gate and up product,
gated codes, down product, last norm.

Each step is held against its definition applied to what the step before it gave
(the codes exactly, products bit for bit), so no tolerance piles up."""

import numpy as np
import pytest

import w8_util
from gpu_util import device, note
from w8_util import TYPES, bits

import bit_weight_only_wq_amd as wq

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def weights(N, K, seed):
    g = torch.Generator().manual_seed(seed)
    return wq.quantize_rows((torch.randn((N, K), generator=g) * 0.05).half().to("cuda"))


def host(t):
    return t.detach().cpu()


def check_product(y, a, sa, w, bias=None):
    want = w8_util.product(host(a).numpy(), host(sa).numpy(), host(w[0]).numpy(), host(w[1]).numpy(),
                           host(bias) if bias is not None else None, y.dtype)
    assert torch.equal(bits(y), bits(want))


def check_rows(codes, scales, x, gate=None):
    c, s = w8_util.rows(host(x), host(gate) if gate is not None else None)
    assert np.array_equal(host(codes).numpy(), c)
    assert np.allclose(host(scales).numpy(), s, rtol=2.0 ** -22, atol=0)


def check_norm(codes, scales, total, x, weight, residual):
    _, c, s, h = w8_util.norm(host(x), host(weight), host(residual) if residual is not None else None, 1e-6)
    assert np.array_equal(host(codes).numpy(), c) and np.allclose(host(scales).numpy(), s, rtol=2.0 ** -21, atol=0)
    assert residual is None or torch.equal(bits(total), bits(h))


@pytest.mark.parametrize("B", [1, 5, 70])
def test_layer(B):
    dev = device()
    note(f"8-bit layer B={B}")
    heads, q_heads, width, ffn, vocab = 2, 4, 512, 1408, 1000
    f16 = torch.float16
    gen = torch.Generator().manual_seed(B)
    x = (torch.randn((B, width), generator=gen)).half().to(dev)
    n1, n2, n3 = (torch.ones(width, dtype=f16, device=dev) + 0.1 * i for i in range(3))
    wqkv, wo = weights((q_heads + 2 * heads) * 128, width, 1), weights(width, q_heads * 128, 2)
    wgu, wd, wv = weights(2 * ffn, width, 3), weights(width, ffn, 4), weights(vocab, width, 5)
    bias = torch.randn((q_heads + 2 * heads) * 128, generator=gen).half().to(dev)
    cache = wq.PagedKV(heads=heads, num_pages=2 * B, slots=B, max_pages=2)
    cache.table.copy_(torch.arange(2 * B, dtype=torch.int32).view(B, 2))
    lens = torch.zeros(B, dtype=torch.int32, device=dev)
    freqs = wq.rope_frequencies(128)

    a, sa, none = wq.rmsnorm_quantize(x, n1)
    assert none is None
    check_norm(a, sa, None, x, n1, None)
    qkv = wq.gemm_w8a8(a, sa, *wqkv, bias=bias)
    check_product(qkv, a, sa, wqkv, bias)
    heads_rows = qkv.view(B, q_heads + 2 * heads, 128)
    turned = wq.rope(heads_rows[:, :q_heads + heads], lens, freqs)
    lens += 1
    wq.kv_paged_append(turned[:, q_heads:], heads_rows[:, q_heads + heads:], cache, lens)
    o = wq.kv_paged_attention(turned[:, :q_heads], cache, lens)
    # One token: the attention gives its v, each KV head's for the two query heads on it.
    assert torch.equal(o.view(B, heads, 2, 128), heads_rows[:, q_heads + heads:, None].expand(B, heads, 2, 128))
    a, sa = wq.quantize_rows(o.view(B, -1))
    check_rows(a, sa, o.view(B, -1))
    y = wq.gemm_w8a8(a, sa, *wo)
    check_product(y, a, sa, wo)
    stream = x.clone()
    before = stream.clone()
    a, sa, total = wq.rmsnorm_quantize(y, n2, residual=stream, total=stream)
    assert total is stream
    check_norm(a, sa, total, y, n2, before)
    gu = wq.gemm_w8a8(a, sa, *wgu)
    check_product(gu, a, sa, wgu)
    a, sa = wq.quantize_rows(gu[:, ffn:], gate=gu[:, :ffn])
    check_rows(a, sa, gu[:, ffn:], gu[:, :ffn])
    y = wq.gemm_w8a8(a, sa, *wd, dtype=TYPES["fp16"])
    check_product(y, a, sa, wd)
    v, total = wq.rmsnorm(y, n3, residual=stream)
    want, _, _, h = w8_util.norm(host(y), host(n3), host(stream), 1e-6)
    assert torch.equal(bits(total), bits(h))
    assert np.all(np.abs(w8_util.f64(host(v)) - want) <= np.abs(want) * 2.0 ** -10.9 + 2.0 ** -24)
    # The last product as a weight-only one: the norm's values are its activations.
    codes, scales, zeros = wq.quantize_pack(torch.randn((vocab, width), generator=gen).half().to(dev), group=128, bits=4)
    logits = wq.gemm(v, codes, scales, zeros, N=vocab, K=width)
    assert logits.shape == (B, vocab) and torch.isfinite(logits).all()
    a, sa, _ = wq.rmsnorm_quantize(y, n3, residual=stream)
    check_product(wq.gemm_w8a8(a, sa, *wv), a, sa, wv)


def test_bench_line():
    """bench.py's 8-bit table on a small layer."""
    import types

    import bench
    device()
    note("8-bit bench lines")
    rows = bench.run_w8a8(types.SimpleNamespace(batches="1,33", steps=3, warmup=1), shape=(512, 1408), layers=2)
    assert [r["config"]["tokens"] for r in rows] == [1, 33]
    for r in rows:
        assert r["value"] > 0 and r["roofline"]["bytes_per_step"] > 0 and len(r["kernels"]) == 8
