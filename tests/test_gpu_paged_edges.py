"""The paged int4 KV cache at the sizes its kernels change their form: decode
appends of more entries than one workgroup's list, repeated and padding slots
among single tokens, pools past 4 GB, and the paged decode step of bench.py."""

import sys
from types import SimpleNamespace

import numpy as np
import pytest

from conftest import ROOT
from gpu_util import device, note, to_dev
from paged_util import D, G, Host, append, draw_tokens, gpu_cache
from test_gpu_paged import check_attention, filled, i32

import bit_weight_only_wq_amd as wq

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("count", [1, 63, 64, 65, 1024, 1025, 1500])
def test_append_single_tokens_of_many_slots(count):
    """One token each, a third of the slots completing a block."""
    device()
    rng = np.random.default_rng(count)
    host = Host(1, count + 2, count, 1)
    cache = gpu_cache(wq, host)
    note(f"paged append {count} slots to near a block")
    append(wq, cache, host, [(s, *draw_tokens(rng, 127 if s % 3 == 0 else 1, 1)) for s in range(count)])
    note(f"paged append one token to each of {count} slots")
    append(wq, cache, host, [(int(s), *draw_tokens(rng, 1, 1)) for s in rng.permutation(count)], cu=False)
    host.check_buffers(cache, count)


@pytest.mark.parametrize("count", [40, 1100])
def test_append_single_tokens_left_out(count):
    """Of single tokens: padding, a slot's second entry, an empty slot, a length
    past the table and a whole block without a page leave all buffers alone."""
    device()
    rng = np.random.default_rng(77)
    heads, S = 2, 8
    host = Host(heads, 9, S, 2)
    cache = gpu_cache(wq, host)
    append(wq, cache, host, [(s, *draw_tokens(rng, 127, heads)) for s in range(6)])
    K, V = draw_tokens(rng, count, heads)
    seqs = np.full(count, -1, np.int32)
    seqs[:9] = [3, 3, S, 0, 5, 6, 7, 0, 2 ** 31 - 1]
    seqs[-1] = 4
    lens = host.lens
    lens[[0, 3, 4, 5]] += 1
    lens[6], lens[7] = 0, 2 * G + 200
    host.give_pages(0, 1)
    host.give_pages(3, 1)
    host.table[4, 0], host.table[5, 0] = 9, -1          # no such pages
    cache.table.copy_(to_dev(host.table))
    before_w, before_p = cache.windows.clone(), cache.pages.clone()
    note(f"paged append single tokens left out, {count} entries")
    wq.kv_paged_append(to_dev(K), to_dev(V), cache, to_dev(lens), seqs=to_dev(seqs))
    host.add(3, K[:1], V[:1])
    host.add(0, K[3:4], V[3:4])
    want_p = before_p.clone()
    for s in (0, 3):
        want_p[host.table[s, 0]] = cache.pages[host.table[s, 0]]
    assert torch.equal(cache.pages, want_p)
    for s in (1, 2, 6, 7):
        assert torch.equal(cache.windows[s], before_w[s]), s
    host.K[4], host.V[4] = host.K[4][:0], host.V[4][:0]  # their blocks have no page to compare
    host.K[5], host.V[5] = host.K[5][:0], host.V[5][:0]
    host.check_buffers(cache, "left out")


def test_pages_past_4_gb():
    """Page ids whose byte offsets pass 2^31 and 2^32, in every operator."""
    device()
    heads, pages = 8, 31500                              # 139264 bytes a page, 4.39 GB
    rng = np.random.default_rng(5)
    host = Host(heads, pages, 3, 4)
    ids = [pages - 1, 15421, 30841, 15420, 30840, 7, pages - 2, 2]     # about 2^31 and 2^32 bytes
    host.free = ids[::-1]
    cache = wq.PagedKV(heads, pages, 3, 4)
    note("paged pool of 4.39 GB")
    append(wq, cache, host, [(0, *draw_tokens(rng, 3 * G + 9, heads)), (1, *draw_tokens(rng, 2 * G, heads))])
    q = rng.standard_normal((3, 2 * heads, D)).astype(np.float16)
    for use_ws in (True, False):
        out = wq.kv_paged_attention(to_dev(q), cache, to_dev(host.lens), use_workspace=use_ws)
        check_attention(out, host, q, [0, 1, 2], what="past 4 GB")
    wq.kv_paged_copy(cache, [[ids[0], pages - 3], [ids[2], 4]])
    assert torch.equal(cache.pages[pages - 3], cache.pages[ids[0]])
    assert torch.equal(cache.pages[4], cache.pages[ids[2]])
    held = [cache.pages[int(p)].clone() for p in host.table[0, :3]]
    table, used = wq.kv_paged_compact(cache, to_dev(host.lens))
    assert int(used) == 5 and int(table.max()) == 4
    for p, want in zip(table[0, :3].tolist(), held):
        assert torch.equal(cache.pages[p], want)
    cache.table = table
    out = wq.kv_paged_attention(to_dev(q), cache, to_dev(host.lens))
    check_attention(out, host, q, [0, 1, 2], what="compacted")


def test_bench_paged_decode_step(capsys):
    """The command's step at a small shape: every kernel timed, lengths within
    the table, bytes counted."""
    device()
    sys.path.insert(0, ROOT)
    import bench
    note("bench paged decode step")
    row = bench.run_kv_paged(SimpleNamespace(steps=130, warmup=2), shape=(3, 2, 4, 256), layers=2)
    assert sorted(row["kernels"]) == ["kv_paged_append", "kv_paged_attention", "rope"]
    assert row["roofline"]["bytes_per_step"] > 0 and row["config"]["tokens"] == 256
    assert "kv_paged_decode" in capsys.readouterr().out


def test_attention_most_rows_without_a_workspace():
    """65535 entries of 128 heads, 128 rows below what a grid takes: three hold
    tokens, the others are padding and give zeros."""
    dev = device()
    heads = 128
    rng = np.random.default_rng(6)
    host = Host(heads, 2, 3, 1)
    cache = gpu_cache(wq, host)
    append(wq, cache, host, [(s, *draw_tokens(rng, n, heads)) for s, n in enumerate((3, 130, 40))])
    seqs = np.full(65535, -1, np.int32)
    at = [0, 40000, 65534]
    seqs[at] = [2, 0, 1]
    q = rng.standard_normal((3, heads, D)).astype(np.float16)
    big = torch.zeros((65535, heads, D), dtype=torch.float16, device=dev)
    big[at] = to_dev(q)
    out = torch.full_like(big, 3.0)
    note("paged attention with 8388480 rows")
    wq.kv_paged_attention(big, cache, to_dev(host.lens), seqs=to_dev(seqs), out=out, use_workspace=False)
    check_attention(out[at], host, q, [2, 0, 1], what="most rows")
    out[at] = 0
    assert not out.any()


def test_attention_out_over_q_refused():
    """q itself, a shifted view of its packed row, rows one entry on: refused.
    Beside q in the row: taken."""
    dev = device()
    host, cache, rng = filled(2, [77, 300, 128], 31)
    q = rng.standard_normal((3, 4, D)).astype(np.float16)
    row = torch.zeros((4, 12, D), dtype=torch.float16, device=dev)
    row[:3, :4] = to_dev(q)
    args = dict(cache=cache, lens=to_dev(host.lens), seqs=i32([1, 2, 3]))
    for out in (row[:3, :4], row[:3, 1:5], row[:3, 3:7], row[1:, :4], row.view(-1, 4, D)[1:4]):
        before = row.clone()
        with pytest.raises(ValueError):
            wq.kv_paged_attention(row[:3, :4], out=out, **args)
        assert torch.equal(row, before)
    note("paged attention beside its q")
    for out in (row[:3, 4:8], row[:3, 8:]):
        got = wq.kv_paged_attention(row[:3, :4], out=out, **args)
        check_attention(got, host, q, [1, 2, 3], what="beside q")


def test_replaced_buffers_are_the_ones_used():
    """pages, windows and table set anew (a packed pool cut to what is in use):
    every call follows; what does not fit, and the sizes themselves, cannot be
    set."""
    dev = device()
    host, cache, rng = filled(2, [300, 700, 40], 33, max_pages=7, extra_pages=20)
    q = rng.standard_normal((3, 4, D)).astype(np.float16)
    slots, lens = [1, 2, 3], to_dev(host.lens)
    old = cache.pages
    note("paged cache with its buffers replaced")
    table, used = wq.kv_paged_compact(cache, lens)
    n = int(used.item())
    cache.table = table
    cache.pages = cache.pages[:n + 2].clone()
    cache.windows = cache.windows.clone()
    old.fill_(0x5A)                                   # nobody's any more
    assert (cache.num_pages, cache.descriptor().num_pages) == (n + 2, n + 2)
    check_attention(wq.kv_paged_attention(to_dev(q), cache, lens, seqs=i32(slots)), host, q, slots, what="cut")
    host.table, host.free = table.cpu().numpy(), [n + 1, n]
    append(wq, cache, host, [(1, *draw_tokens(rng, 100, 2)), (3, *draw_tokens(rng, 90, 2))])
    host.check_buffers(cache, "cut")
    assert torch.all(old == 0x5A)
    cache.table[1, 0] = n + 2                         # an id of the old pool only
    lens = to_dev(host.lens)
    out = wq.kv_paged_attention(to_dev(q), cache, lens, seqs=i32(slots))
    assert torch.isnan(out[0]).all()
    check_attention(out[1:], host, q[1:], slots[1:], what="beside a page past the pool")
    held = cache.pages, cache.windows, cache.table
    for name, bad in [("pages", cache.pages[:, :1].contiguous()), ("pages", cache.pages[:, :, :100]),
                      ("pages", cache.pages.cpu()), ("pages", cache.pages.view(torch.int8)),
                      ("windows", cache.windows[:1]), ("windows", cache.windows[:, :1].contiguous()),
                      ("windows", cache.windows.float()), ("table", cache.table[:2]), ("table", cache.table.long())]:
        with pytest.raises(ValueError):
            setattr(cache, name, bad)
    for name in ("num_pages", "heads", "slots", "max_pages", "device"):
        with pytest.raises(AttributeError):
            setattr(cache, name, getattr(cache, name))
    assert all(a is b for a, b in zip(held, (cache.pages, cache.windows, cache.table)))


def test_compact_at_the_border_of_a_range():
    """The plan marks 131072 pages at a time: pages in use and free on both sides
    of that border, the first and the last of either range, fewer and more of
    them in use than a range holds."""
    dev = device()
    R = 131072
    P = R + 200                                       # 2.3 GB of one head
    cache = wq.PagedKV(1, P, 2, R + 100)
    rng = np.random.default_rng(3)
    for rows in ([[R - 1, R, 0, P - 1], [R + 1, R - 2, 5]], [[R], [R - 1]],
                 [np.delete(np.arange(R + 90), [3, R - 1, R, R + 7])[rng.permutation(R + 86)], [P - 1, R + 150]]):
        lens, table = np.zeros(2, np.int32), np.full((2, R + 100), -1, np.int32)
        for s, r in enumerate(rows):
            table[s, :len(r)], lens[s] = r, len(r) * G
        held = np.unique(np.concatenate([np.asarray(r) for r in rows]))
        cache.pages.view(torch.int32)[:, 0, 17] = torch.arange(P, dtype=torch.int32, device=dev)
        cache.table.copy_(to_dev(table))
        note(f"paged compact of {len(held)} pages about {R}")
        new, used = wq.kv_paged_compact(cache, to_dev(lens))
        n = int(used.item())
        assert n == len(held)
        new, got = new.cpu().numpy(), cache.pages.view(torch.int32)[:, 0, 17].cpu().numpy()
        for s, r in enumerate(rows):
            ids = new[s, :len(r)]
            assert np.all((ids >= 0) & (ids < n)) and np.array_equal(got[ids], r), s
            assert np.all(new[s, len(r):] == -1)
            assert np.array_equal(ids[np.asarray(r) < n], np.asarray(r)[np.asarray(r) < n])      # these stay
        assert len(np.unique(np.concatenate([new[s, :len(r)] for s, r in enumerate(rows)]))) == n
