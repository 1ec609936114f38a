"""Checks of the paged KV cache's and the rotary positions' C entry points that
need no GPU: bad arguments are refused synchronously, before any launch, with a
status and a message; empty calls are no-ops; the frequency tables."""

import ctypes
import math

import numpy as np
import pytest

wq = pytest.importorskip("bit_weight_only_wq_amd")
from bit_weight_only_wq_amd import _lib  # noqa: E402

FAKE = 0x100000  # 16-byte aligned, never dereferenced (validation fails first)
OK, BAD, UNSUP, MIS = _lib.WQ_OK, _lib.WQ_ERR_INVALID_ARG, _lib.WQ_ERR_UNSUPPORTED, _lib.WQ_ERR_MISALIGNED


def rope(T=3, H=2, D=128, rot=128, layout=0, xt=256, xh=128, ot=256, oh=128, x=FAKE, p=FAKE, f=FAKE, o=FAKE + 0x10000):
    return wq.load().wq_rope(x, T, H, D, xt, xh, p, f, rot, layout, 1.0, o, ot, oh, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), BAD), (dict(H=-1), BAD), (dict(D=0), BAD), (dict(rot=-2), BAD), (dict(rot=3), BAD), (dict(rot=130), BAD),
    (dict(layout=2), BAD), (dict(layout=-1), BAD), (dict(D=1026, xh=1026, oh=1026, xt=2052, ot=2052), UNSUP),
    (dict(T=1 << 24), UNSUP), (dict(H=65536), UNSUP), (dict(xt=-1), BAD), (dict(ot=-256), BAD), (dict(xh=1 << 38), BAD),
    (dict(oh=127), BAD), (dict(ot=255), BAD), (dict(ot=0), BAD), (dict(oh=0), BAD),
    (dict(ot=128, oh=383), BAD), (dict(o=FAKE, xt=512), BAD), (dict(o=FAKE, xh=256, oh=128), BAD),
    (dict(x=0), BAD), (dict(o=0), BAD), (dict(p=0), BAD), (dict(f=0), BAD),
    (dict(x=FAKE + 1), MIS), (dict(o=FAKE + 0x10001), MIS), (dict(p=FAKE + 2), MIS), (dict(f=FAKE + 4), MIS),
    (dict(T=0, x=0, o=0), OK), (dict(H=0, x=0, o=0), OK)])
def test_rope_refusals(kw, want):
    assert rope(**kw) == want
    assert (want == OK) == (wq.load().wq_last_error() == b"")


def paged(pages=FAKE, windows=FAKE, table=FAKE, heads=4, num_pages=16, slots=8, max_pages=5):
    return _lib.KvPaged(pages, windows, table, heads, num_pages, slots, max_pages)


BAD_CACHES = [(dict(heads=0), BAD), (dict(heads=32768), BAD), (dict(num_pages=0), BAD), (dict(num_pages=1 << 31), BAD),
              (dict(slots=0), BAD), (dict(slots=1 << 31), BAD), (dict(max_pages=0), BAD), (dict(max_pages=1 << 24), BAD)]
BAD_BUFFERS = [(dict(pages=0), BAD, 1), (dict(windows=0), BAD, 2), (dict(table=0), BAD, 4), (dict(pages=FAKE + 8), MIS, 1),
               (dict(windows=FAKE + 8), MIS, 2), (dict(table=FAKE + 2), MIS, 4)]


def append(c=None, T=3, ks=512, vs=512, k=FAKE, v=FAKE, lens=FAKE, seqs=FAKE, cu=0, n=3):
    c = ctypes.byref(paged()) if c is None else c
    return wq.load().wq_kv_paged_append(k, v, T, ks, vs, c, lens, seqs, cu, n, None)


def attend(c=None, qs=2048, qh=16, q=FAKE, lens=FAKE, seqs=FAKE, n=3, window=0, scale=0.1, out=FAKE, os_=2048, ws=0, wn=0):
    c = ctypes.byref(paged()) if c is None else c
    return wq.load().wq_kv_paged_attention(q, qs, qh, c, lens, seqs, n, window, scale, out, os_, ws, wn, None)


def pairs(*p):
    return np.array(p, np.int32).reshape(-1, 2)


def copy(c=None, p=None, n=None):
    c = ctypes.byref(paged()) if c is None else c
    p = pairs((0, 1)) if p is None else p
    return wq.load().wq_kv_paged_copy(c, p.ctypes.data, len(p) if n is None else n, None)


def fork(c=None, p=None, n=None, lens=FAKE):
    c = ctypes.byref(paged()) if c is None else c
    p = pairs((0, 1)) if p is None else p
    return wq.load().wq_kv_paged_fork(c, lens, p.ctypes.data, len(p) if n is None else n, None)


def compact(c=None, lens=FAKE, out=FAKE + 0x1000, used=FAKE, ws=FAKE, wn=1 << 20):
    c = ctypes.byref(paged()) if c is None else c
    return wq.load().wq_kv_paged_compact(c, lens, out, used, ws, wn, None)


@pytest.mark.parametrize("call,needs", [(append, 7), (attend, 7), (copy, 1), (fork, 6), (compact, 5)])
def test_cache_refusals(call, needs):
    assert call(ctypes.POINTER(_lib.KvPaged)()) == BAD
    for kw, want in BAD_CACHES:
        assert call(ctypes.byref(paged(**kw))) == want, kw
    for kw, want, bit in BAD_BUFFERS:
        if needs & bit:
            assert call(ctypes.byref(paged(**kw))) == want, kw
            assert wq.load().wq_last_error()


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), BAD), (dict(n=65536, T=65536), BAD), (dict(n=9, T=9, seqs=0), BAD), (dict(T=-1), BAD), (dict(T=4), BAD),
    (dict(T=(1 << 30) + 1, cu=FAKE), BAD), (dict(ks=511), BAD), (dict(vs=504), BAD), (dict(vs=1 << 32), BAD),
    (dict(ks=516), MIS), (dict(vs=513), MIS), (dict(k=0), BAD), (dict(v=0), BAD), (dict(k=FAKE + 8), MIS),
    (dict(v=FAKE + 2), MIS), (dict(lens=0), BAD), (dict(lens=FAKE + 2), MIS), (dict(seqs=FAKE + 1), MIS),
    (dict(cu=FAKE + 2), MIS), (dict(n=0, T=0, k=0, v=0, lens=0), OK), (dict(T=0, cu=FAKE, k=0, v=0), OK)])
def test_append_refusals(kw, want):
    assert append(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), BAD), (dict(n=65536), BAD), (dict(n=9, seqs=0), BAD), (dict(qh=0), BAD), (dict(qh=3), BAD),
    (dict(qh=18, qs=4096, os_=4096), BAD), (dict(n=256, qh=65536, qs=1 << 23, os_=1 << 23), UNSUP), (dict(qs=2047), BAD),
    (dict(os_=2040), BAD), (dict(qs=2052), MIS), (dict(os_=2050), MIS), (dict(q=FAKE + 8), MIS), (dict(out=FAKE + 4), MIS),
    (dict(q=0), BAD), (dict(out=0), BAD), (dict(lens=0), BAD), (dict(lens=FAKE + 1), MIS), (dict(window=-1), BAD),
    (dict(scale=math.inf), BAD), (dict(scale=math.nan), BAD), (dict(wn=64), BAD), (dict(ws=FAKE + 4, wn=1 << 30), MIS),
    (dict(n=0, q=0, out=0, lens=0), OK)])
def test_attention_refusals(kw, want):
    assert attend(**kw) == want


def test_attention_workspace_size():
    lib, n = wq.load(), ctypes.c_size_t(7)
    c = paged(pages=0, windows=0, table=0)
    assert lib.wq_kv_paged_workspace_size(ctypes.byref(c), 3, 16, None) == BAD
    assert lib.wq_kv_paged_workspace_size(ctypes.byref(c), 0, 16, ctypes.byref(n)) == OK and n.value == 0
    assert lib.wq_kv_paged_workspace_size(ctypes.byref(c), 3, 17, ctypes.byref(n)) == BAD and n.value == 0
    assert lib.wq_kv_paged_workspace_size(ctypes.byref(c), 3, 16, ctypes.byref(n)) == OK
    if n.value:                                    # one byte too few is refused before any launch
        assert attend(ws=FAKE, wn=n.value - 1) == BAD
    big = paged(max_pages=(1 << 24) - 1)
    assert lib.wq_kv_paged_workspace_size(ctypes.byref(big), 1000, 16, ctypes.byref(n)) == UNSUP


def test_pairs_refusals():
    for call, top in ((copy, 16), (fork, 8)):
        assert call(p=pairs((0, top))) == BAD
        assert call(p=pairs((top, 0))) == BAD
        assert call(p=pairs((-1, 0))) == BAD
        assert call(p=pairs((0, -1))) == BAD
        assert call(p=pairs((1, 1))) == BAD
        assert call(p=pairs((0, 3), (1, 3))) == BAD and b"twice" in wq.load().wq_last_error()
        assert call(p=pairs((0, 3), (3, 4))) == BAD and b"source" in wq.load().wq_last_error()
        assert call(n=-1) == BAD
        assert call(p=pairs(), n=0) == OK
        assert call(p=np.array([], np.int32).reshape(0, 2)) == OK
    assert wq.load().wq_kv_paged_copy(ctypes.byref(paged()), None, 1, None) == BAD
    assert fork(lens=0) == BAD
    assert fork(lens=FAKE + 2) == MIS


def test_compact_refusals():
    need = ctypes.c_size_t(0)
    assert wq.load().wq_kv_paged_compact_workspace_size(ctypes.byref(paged()), ctypes.byref(need)) == OK
    assert need.value > 0
    assert compact(wn=need.value - 1) == BAD
    assert compact(ws=0, wn=0) == BAD
    assert compact(ws=0, wn=1 << 20) == BAD
    assert compact(ws=FAKE + 4) == MIS
    assert compact(lens=0) == BAD
    assert compact(out=0) == BAD
    assert compact(used=0) == BAD
    assert compact(out=FAKE) == BAD                # the cache's own table
    assert compact(out=FAKE + 2) == MIS
    assert compact(used=FAKE + 2) == MIS
    assert wq.load().wq_kv_paged_compact_workspace_size(ctypes.byref(paged()), None) == BAD


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros((2, 2, 128), dtype=torch.float16)
    with pytest.raises(ValueError):
        wq.rope(x, torch.zeros(2, dtype=torch.int32), torch.zeros(64, dtype=torch.float64))
    with pytest.raises(ValueError):
        wq.PagedKV(2, 2, 2, 2, device="cpu")


def test_rope_frequencies():
    f = wq.rope_frequencies(128, base=10000.0, device="cpu").numpy()
    want = np.array([10000.0 ** (-2 * j / 128) for j in range(64)])
    assert np.allclose(f, want, rtol=1e-14, atol=0)
    assert np.array_equal(wq.rope_frequencies(128, kind="linear", factor=4.0, device="cpu").numpy(), f / 4)
    b = wq.rope_frequencies(128, kind="base", factor=8.0, device="cpu").numpy()
    assert b[0] == 1.0 and np.isclose(b[-1], f[-1] / 8, rtol=1e-12)
    p = wq.rope_frequencies(128, kind="parts", factor=8.0, context=4096, low=1.0, high=32.0, device="cpu").numpy()
    turns = 4096 * f / (2 * np.pi)
    assert np.array_equal(p[turns >= 32], f[turns >= 32])
    assert np.allclose(p[turns <= 1], f[turns <= 1] / 8, rtol=1e-14)
    mid = (turns > 1) & (turns < 32)
    k = (turns[mid] - 1) / 31
    assert mid.any() and np.allclose(p[mid], f[mid] * k + f[mid] / 8 * (1 - k), rtol=1e-14)
    assert wq.rope_frequencies(0, device="cpu").shape == (0,)
    for kw in (dict(rot=3), dict(rot=-2), dict(rot=4, kind="x"), dict(rot=4, base=0.0), dict(rot=4, factor=-1.0)):
        with pytest.raises(ValueError):
            wq.rope_frequencies(**kw, device="cpu")


@pytest.mark.parametrize("kw", [dict(low=4.0, high=4.0), dict(low=5.0, high=4.0), dict(context=0)])
def test_rope_frequencies_parts_refused(kw):
    pytest.importorskip("torch")
    with pytest.raises(ValueError):
        wq.rope_frequencies(64, kind="parts", factor=2.0, device="cpu", **kw)


@pytest.mark.parametrize("heads,group,n", [(129, 1, 65535), (8192, 1, 1024), (4096, 1, 2048), (32767, 1, 512)])
def test_attention_rows_past_a_grid(heads, group, n):
    """Without a workspace a row is a workgroup of 512 threads, and a grid takes
    fewer than 2^32 threads: refused before any launch."""
    c = ctypes.byref(paged(heads=heads, slots=65535, max_pages=1))
    qh, need = heads * group, ctypes.c_size_t(0)
    assert n * heads * -(-group // 16) >= 1 << 23 and n * qh < 1 << 24
    assert attend(c=c, n=n, qh=qh, qs=qh * 128, os_=qh * 128) == UNSUP
    assert b"workspace" in wq.load().wq_last_error()
    assert wq.load().wq_kv_paged_workspace_size(c, n, qh, ctypes.byref(need)) == OK


def test_rows_meet_against_the_addresses():
    """Whether two strided [tokens, heads, channels] views share an element, by
    their addresses: never denied where they do, and not claimed for rows or heads
    that lie side by side."""
    torch = pytest.importorskip("torch")
    meet = wq._rows_meet
    base = torch.zeros(4096, dtype=torch.float16)

    def cells(t):
        at = t.storage_offset()
        return {at + i * t.stride(0) + h * t.stride(1) + c for i in range(t.shape[0]) for h in range(t.shape[1])
                for c in range(t.shape[2])}

    rng = np.random.default_rng(1)
    for _ in range(3000):
        T, H, D = (int(rng.integers(1, n)) for n in (5, 5, 9))
        views = [base.as_strided((T, H, D), (int(rng.integers(0, 60)), int(rng.integers(0, 30)), 1),
                                 int(rng.integers(0, 100))) for _ in range(2)]
        if cells(views[0]) & cells(views[1]):
            assert meet(*views) and meet(*views[::-1])
    x = base[:3 * 4 * 32].view(3, 4, 32)
    for a, b in ((x[..., :16], x[..., 16:]), (x[:, :2], x[:, 2:]), (x[:, ::2], x[:, 1::2]), (x[..., 4:12], x[..., 20:28]),
                 (x[:1], x[1:2])):
        assert not cells(a) & cells(b)
        assert not meet(a, b) and not meet(b, a)
    for a, b in ((x, x), (x[..., :17], x[..., 15:]), (x[:, :2], x[:, 1:3]), (x[:2], x[1:])):
        assert cells(a) & cells(b) and meet(a, b)


def test_compact_table_over_the_cache_s_refused():
    for off in (4, -4, 156, -156):                 # 8 slots of 5 entries: 160 bytes
        assert compact(out=FAKE + off) == BAD, off
        assert b"overlap" in wq.load().wq_last_error()
    assert compact(out=FAKE + 156, ws=0, wn=0) == BAD
    wide = paged(slots=(1 << 31) - 1, max_pages=(1 << 24) - 1)
    assert compact(c=ctypes.byref(wide), out=FAKE + (1 << 40)) == BAD and b"overlap" in wq.load().wq_last_error()
