"""GPU rotary positions against the definition in float64: both layouts, parts
of a head, strided and in-place tensors, sizes of the 16-byte and the
one-channel form, far and negative positions.

Tolerance: the angle is off by at most 2^-25 of a turn and fp32's sine and
cosine by some steps of 2^-24, together under 2^-21; the two products and their
sum add 3 * 2^-24; so a value is off by at most 2^-20 (|u| + |w|) scale before
it is rounded to fp16, which adds half a step: 2^-11 of it, or 2^-25 if it is
subnormal."""

import numpy as np
import pytest

from gpu_util import bits16, device, note, to_dev

import bit_weight_only_wq_amd as wq

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def reference(x, pos, freqs, layout, scale):
    """(y, bound) float64."""
    x = x.astype(np.float64)
    rot = 2 * len(freqs)
    a = (pos.astype(np.float64)[:, None] * freqs)[:, None, :]
    c, s = np.cos(a) * scale, np.sin(a) * scale
    i0 = np.arange(rot // 2) if layout == "half" else 2 * np.arange(rot // 2)
    i1 = i0 + rot // 2 if layout == "half" else i0 + 1
    y, m = x.copy(), np.zeros_like(x)
    u, w = x[..., i0], x[..., i1]
    y[..., i0], y[..., i1] = u * c - w * s, u * s + w * c
    m[..., i0] = m[..., i1] = (np.abs(u) + np.abs(w)) * scale * 2.0 ** -20
    return y, m + 2.0 ** -11 * np.abs(y) + 2.0 ** -25


def check(got, x, pos, freqs, layout, scale, what):
    y, bound = reference(x, pos, freqs, layout, scale)
    d = np.abs(got.cpu().numpy().astype(np.float64) - y)
    assert np.all(d <= bound), (what, np.max(d / bound))
    rot = 2 * len(freqs)
    if rot < x.shape[2]:
        assert np.array_equal(bits16(got[..., rot:].cpu().numpy()), bits16(x[..., rot:])), what


CASES = [  # tokens, heads, dim, rot, layout
    (1, 64, 128, 128, "half"), (1, 1, 2, 2, "half"), (5, 3, 128, 64, "half"), (33, 40, 128, 64, "interleaved"),
    (7, 5, 80, 80, "half"), (7, 5, 80, 80, "interleaved"), (9, 2, 96, 40, "half"), (3, 7, 13, 10, "interleaved"),
    (3, 7, 13, 10, "half"), (2, 3, 256, 256, "half"), (2, 3, 1024, 1024, "half"), (4, 3, 1024, 16, "interleaved"),
    (2, 2, 1023, 1022, "interleaved"), (700, 72, 128, 128, "half"), (300, 9, 64, 64, "interleaved"),
    (3, 700, 64, 64, "half"), (2, 300, 1024, 1024, "half"), (4, 2, 128, 0, "half"),
]


@pytest.mark.parametrize("T,H,dim,rot,layout", CASES)
@pytest.mark.parametrize("form", ["new", "in place", "strided"])
def test_rope_matches_definition(T, H, dim, rot, layout, form):
    device()
    note(f"rope T={T} H={H} dim={dim} rot={rot} {layout} {form}")
    rng = np.random.default_rng(T * 1000 + dim + rot)
    x = rng.standard_normal((T, H, dim)).astype(np.float16)
    pos = rng.integers(0, 1 << 20, T).astype(np.int32)
    f = wq.rope_frequencies(rot, kind="parts", factor=4.0)
    freqs, scale = f.cpu().numpy(), 1.25
    p = to_dev(pos)
    if form == "new":
        xd = to_dev(x)
        got = wq.rope(xd, p, f, layout=layout, scale=scale)
        assert np.array_equal(bits16(xd.cpu().numpy()), bits16(x))
    elif form == "in place":
        xd = to_dev(x)
        got = wq.rope(xd, p, f, layout=layout, scale=scale, out=xd)
        assert got is xd
    else:                                      # heads of a packed row, into a [heads, tokens, dim] buffer
        row = to_dev(np.concatenate([np.full((T, 2, dim), 9.0, np.float16), x], 1))
        buf = torch.full((H + 2, T, dim), -3.0, dtype=torch.float16, device="cuda")
        got = wq.rope(row[:, 2:], p, f, layout=layout, scale=scale, out=buf[1:-1].transpose(0, 1))
        assert torch.all(buf[0] == -3.0) and torch.all(buf[-1] == -3.0)
    check(got, x, pos, freqs, layout, scale, form)


def test_far_and_negative_positions():
    device()
    rng = np.random.default_rng(5)
    pos = np.array([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 10 ** 6, 123456789], np.int32)
    x = rng.standard_normal((len(pos), 4, 128)).astype(np.float16)
    f = wq.rope_frequencies(128, base=500000.0)
    note("rope far positions")
    # The last bits of the frequencies matter here: the reference takes the
    # product p f in 80-bit numbers, mod one turn (p f / (2 pi) is off by
    # 2^31 * 2^-52 turns, 2^-21, in 64 bits; its sine by 2^-18.4).
    y, bound = reference(x, pos, f.cpu().numpy(), "half", 1.0)
    turns = pos.astype(np.longdouble)[:, None] * f.cpu().numpy().astype(np.longdouble) / (2 * np.longdouble(np.pi))
    a = ((turns - np.rint(turns)) * 2 * np.pi).astype(np.float64)[:, None, :]
    xd = x.astype(np.float64)
    u, w = xd[..., :64], xd[..., 64:]
    y = np.concatenate([u * np.cos(a) - w * np.sin(a), u * np.sin(a) + w * np.cos(a)], -1)
    bound = bound + 2.0 ** -18 * (np.abs(u) + np.abs(w)).max()
    got = wq.rope(to_dev(x), to_dev(pos), f).cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - y) <= bound)
    assert np.array_equal(bits16(got[0].astype(np.float16)), bits16(x[0]))       # position 0: as it was


def test_turning_back_undoes():
    """Position -p after p gives x again, within two roundings."""
    device()
    rng = np.random.default_rng(6)
    x = rng.standard_normal((17, 6, 128)).astype(np.float16)
    pos = to_dev(rng.integers(0, 100000, 17).astype(np.int32))
    f = wq.rope_frequencies(128)
    note("rope there and back")
    back = wq.rope(wq.rope(to_dev(x), pos, f), -pos, f).cpu().numpy().astype(np.float64)
    # Each rotation rounds a pair by at most 2^-11 of its length per channel; a
    # rotation keeps lengths, so the pair ends within 2 sqrt(2) 2^-11 of it.
    u, w = x[..., :64].astype(np.float64), x[..., 64:].astype(np.float64)
    length = np.hypot(u, w)
    off = np.hypot(back[..., :64] - u, back[..., 64:] - w)
    assert np.all(off <= 2 * np.sqrt(2) * 2.0 ** -11 * length * (1 + 2.0 ** -8) + 2.0 ** -20)


def test_empty_and_refused():
    dev = device()
    f = wq.rope_frequencies(128)
    x = torch.zeros((0, 4, 128), dtype=torch.float16, device=dev)
    assert wq.rope(x, torch.zeros(0, dtype=torch.int32, device=dev), f).shape == (0, 4, 128)
    x = torch.zeros((4, 4, 128), dtype=torch.float16, device=dev)
    p = torch.zeros(4, dtype=torch.int32, device=dev)
    for bad in [lambda: wq.rope(x.float(), p, f), lambda: wq.rope(x, p.long(), f), lambda: wq.rope(x, p[:3], f),
                lambda: wq.rope(x, p, f.float()), lambda: wq.rope(x, p, f, layout="third"),
                lambda: wq.rope(x.transpose(1, 2), p, f), lambda: wq.rope(x[0], p, f),
                lambda: wq.rope(x, p, f, out=x.transpose(0, 1)),                # x's memory in another order
                lambda: wq.rope(x, p, f, out=x[:2]),
                lambda: wq.rope(x[:, :2], p, f, out=x[:, 1:3]),                 # heads that overlap
                lambda: wq.rope(x, p.cpu(), f)]:
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(wq.WQError):                                             # rot past the head
        wq.rope(x, p, wq.rope_frequencies(256))
    with pytest.raises(wq.WQError):                                             # every head the same memory
        wq.rope(x, p, f, out=torch.zeros((1, 1, 128), dtype=torch.float16, device=dev).expand(4, 4, 128))
    # Heads side by side in one packed row are apart.
    row = torch.randn((4, 6, 128), device=dev).half()
    want = wq.rope(row[:, :2], p, f)
    assert torch.equal(wq.rope(row[:, :2], p, f, out=row[:, 2:4]), want)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_out_beside_x_in_every_head(layout):
    """x and out as the two halves of each head's row, and as alternating heads."""
    dev = device()
    rng = np.random.default_rng(8)
    T, H, dim = 5, 6, 64
    x = rng.standard_normal((T, H, dim)).astype(np.float16)
    pos = to_dev(np.arange(T, dtype=np.int32) * 1000)
    freqs = wq.rope_frequencies(dim)
    want = wq.rope(to_dev(x), pos, freqs, layout)
    for buf, a, b in ((torch.full((T, H, 2 * dim), 9.0, dtype=torch.float16, device=dev), np.s_[..., :dim], np.s_[..., dim:]),
                      (torch.full((T, 2 * H, dim), 9.0, dtype=torch.float16, device=dev), np.s_[:, ::2], np.s_[:, 1::2])):
        buf[a] = to_dev(x)
        note(f"rope out beside x {layout}")
        got = wq.rope(buf[a], pos, freqs, layout, out=buf[b])
        assert torch.equal(got, want) and torch.equal(buf[a], to_dev(x))
