"""GPU parity of the paged int4 KV cache with the CPU oracle: append bit for
bit, decode attention within a derived bound (paged_util.Host.attend) and the
product tolerance, copies, forks and compactions byte for byte; ragged batches,
padding, empty sequences, wrong ids; and all of them together as a server
would run them, eager and as a replayed graph."""

import numpy as np
import pytest

from edge_groups import crafted_groups
from gpu_util import L2_REL, bits16, device, note, to_dev
from paged_util import D, G, REC, Host, append, draw_tokens, gpu_cache

import bit_weight_only_wq_amd as wq

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def i32(a):
    return to_dev(np.array(a, np.int32))


def check_attention(got, host, q, slots, window=0, scale=None, what=""):
    ref, bound = host.attend(q, slots, window, scale)
    got = got.cpu().numpy().astype(np.float64)
    d = np.abs(got - ref)
    assert np.all(np.isfinite(got)), what
    assert np.all(d <= bound), (what, np.max(d / bound))
    norm = np.linalg.norm(ref)
    assert np.linalg.norm(got - ref) <= L2_REL * norm, (what, np.linalg.norm(got - ref) / max(norm, 1e-300))
    for i, s in enumerate(slots):
        if not 0 <= s < host.slots or len(host.K[s]) == 0:
            assert not got[i].any(), (what, i)


# ---- append ---------------------------------------------------------------------

@pytest.mark.parametrize("heads,packed", [(1, False), (3, True), (8, False)])
def test_append_ragged_bit_exact(heads, packed):
    """Batches of unlike entries: inside the window, ending on a block's border,
    across one and several borders, none at all; then chunks on top."""
    device()
    rng = np.random.default_rng(heads)
    host = Host(heads, 64, 9, 8)
    cache = gpu_cache(wq, host)
    for step, counts in enumerate([{0: 1, 3: 127, 1: 128, 7: 129, 4: 700, 8: 0, 5: 300},
                                   {5: 84, 0: 126, 3: 1, 8: 55, 1: 200, 4: 37}, {0: 1, 5: 1, 4: 260, 8: 72, 3: 5}]):
        note(f"paged append ragged heads={heads} step={step} {counts}")
        append(wq, cache, host, [(s, *draw_tokens(rng, n, heads)) for s, n in counts.items()], packed=packed)
        host.check_buffers(cache, step)
    # Nothing else was written: free pages, window rows never reached, unused slots.
    pages, windows = cache.pages.cpu().numpy(), cache.windows.cpu().numpy()
    assert np.all(pages[[p for p in range(64) if p in host.free]] == 0xA5)
    assert np.all(windows[[2, 6]] == -7.0)
    assert np.all(windows[8, :, :, 127:] == -7.0)


def test_append_one_by_one_equals_at_once():
    """300 tokens of three sequences, one call per token (with and without cu,
    slots in changing order), against one call with all of them."""
    device()
    rng = np.random.default_rng(11)
    n, heads = 300, 2
    data = [draw_tokens(rng, n, heads) for _ in range(3)]
    one, many = Host(heads, 8, 3, 3, seed=1), Host(heads, 8, 3, 3, seed=1)
    c1, c2 = gpu_cache(wq, one), gpu_cache(wq, many)
    note("paged append token by token")
    for t in range(n):
        order = [(t + j) % 3 for j in range(3)]
        append(wq, c1, one, [(s, data[s][0][t:t + 1], data[s][1][t:t + 1]) for s in order], cu=t % 2 == 0)
    append(wq, c2, many, [(s, *data[s]) for s in range(3)])
    one.check_buffers(c1, "one by one")
    many.check_buffers(c2, "at once")


def test_append_edge_groups():
    """Ties, constant, subnormal and +-65504 groups along both axes."""
    device()
    cols = crafted_groups(G, 4, seed=5)
    n = min(G, cols.shape[0])
    rng = np.random.default_rng(3)
    K, V = draw_tokens(rng, G, 4)
    for h in range(3):
        K[:, h, :n] = cols[(np.arange(n) + 7 * h) % cols.shape[0]].T
        V[:n, h, :] = cols[(np.arange(n) + 5 * h) % cols.shape[0]]
    host = Host(4, 2, 1, 1)
    cache = gpu_cache(wq, host)
    note("paged append crafted groups")
    append(wq, cache, host, [(0, K, V)])
    host.check_buffers(cache, "crafted")


def test_append_matches_flat_cache():
    """The record holds what wq_kv_quantize_block writes for the same block."""
    device()
    rng = np.random.default_rng(4)
    H = 5
    K, V = draw_tokens(rng, G, H)
    host = Host(H, 3, 1, 1)
    cache = gpu_cache(wq, host)
    flat = wq.KVCache(H, 1)
    note("paged append against the flat cache")
    append(wq, cache, host, [(0, K, V)])
    wq.kv_quantize_block(to_dev(K.transpose(1, 0, 2)), to_dev(V.transpose(1, 0, 2)), flat, 0)
    rec = cache.pages[int(host.table[0, 0])]
    parts = [flat.kcodes[:, 0], flat.vcodes[:, 0], flat.kscales[:, 0], flat.kzeros[:, 0], flat.vscales, flat.vzeros]
    want = torch.cat([p.contiguous().view(H, -1).view(torch.uint8) for p in parts], 1)
    assert torch.equal(rec, want)


def test_append_leaves_out():
    """Padding, a slot named twice (its first entry counts), a cu outside the
    tokens, lengths that do not fit, pages that do not exist: nothing of those
    entries is written, and the others' work is done."""
    dev = device()
    rng = np.random.default_rng(8)
    heads, S = 2, 12
    host = Host(heads, 16, S, 2)
    cache = gpu_cache(wq, host)
    K, V = draw_tokens(rng, 3 * G, heads)
    before_w, before_p = cache.windows.clone(), cache.pages.clone()
    # Each entry brings tokens 5 .. 132, a whole block, unless said otherwise.
    rows = [(3, 5, 133, 128), (-1, 5, 133, 128), (S, 5, 133, 128), (2 ** 31 - 1, 5, 133, 128), (3, 200, 328, 128),
            (4, 5, 133, 127), (5, 5, 133, 2 * G + 128), (6, -1, 127, 128), (7, 300, 385, 128), (8, 133, 5, 128),
            (9, 5, 133, -5), (10, 5, 133, 128), (11, 5, 133, 128)]
    host.table[3, 0], host.table[10, 0], host.table[11, 0] = 7, 16, -1
    for s in (4, 5, 6, 7, 8, 9):
        host.table[s] = [1, 2]
    cache.table.copy_(to_dev(host.table))
    lens = np.zeros(S, np.int32)
    for s, _, _, n in rows:
        if 0 <= s < S:
            lens[s] = n
    for s, a, b, n in rows:                   # one call per entry: a cu of two values
        note(f"paged append left out {s} {a} {b} {n}")
        wq.kv_paged_append(to_dev(K), to_dev(V), cache, to_dev(lens), seqs=i32([s]), cu=i32([a, b]))
        if s == 3:
            host.K[3], host.V[3] = K[a:b], V[a:b]       # (both rows of slot 3 are good on their own)
            host.check_buffers(cache, "alone")
    want_p = before_p.clone()
    want_p[7] = cache.pages[7]
    assert torch.equal(cache.pages, want_p) and torch.equal(cache.windows, before_w)
    # In one call: the first entry of slot 3 counts, the second is left out.
    cache.pages.copy_(before_p)
    note("paged append one batch with padding and a repeated slot")
    seqs, lens[4] = [-1, 3, 4, S, 3, 3], 10
    wq.kv_paged_append(to_dev(K), to_dev(V), cache, to_dev(lens), seqs=i32(seqs),
                       cu=i32([0, 5, 133, 143, 200, 328, 384]))
    host.K[3], host.V[3], host.K[4], host.V[4] = K[5:133], V[5:133], K[133:143], V[133:143]
    host.check_buffers(cache, "batch")
    assert torch.equal(cache.windows[:4], before_w[:4]) and torch.equal(cache.windows[5:], before_w[5:])
    # No entries, no tokens.
    empty = torch.zeros((0, heads, D), dtype=torch.float16, device=dev)
    wq.kv_paged_append(empty, empty, cache, to_dev(lens), seqs=i32([]))
    wq.kv_paged_append(empty, empty, cache, to_dev(lens), seqs=i32([3]), cu=i32([0, 0]))
    host.check_buffers(cache, "empty")


def test_append_many_entries():
    """More entries than a workgroup has threads, in shuffled slots."""
    device()
    rng = np.random.default_rng(9)
    S = 600
    host = Host(1, 900, S, 2)
    cache = gpu_cache(wq, host)
    note("paged append 600 entries")
    order = rng.permutation(S)
    append(wq, cache, host, [(int(s), *draw_tokens(rng, int(rng.integers(0, 200)), 1)) for s in order])
    host.check_buffers(cache, "600")
    append(wq, cache, host, [(int(s), *draw_tokens(rng, 1, 1)) for s in rng.permutation(S)], cu=False)
    host.check_buffers(cache, "600 + 1")


# ---- attention ------------------------------------------------------------------

def filled(heads, lens, seed, extra_slots=2, max_pages=None, extra_pages=3):
    """Host and GPU cache whose slot i + 1 holds lens[i] tokens."""
    rng = np.random.default_rng(seed)
    slots = len(lens) + extra_slots
    pages = sum(n // G for n in lens) + extra_pages
    host = Host(heads, pages, slots, max_pages or max(max(lens) // G, 1), seed)
    cache = gpu_cache(wq, host)
    append(wq, cache, host, [(i + 1, *draw_tokens(rng, n, heads)) for i, n in enumerate(lens)])
    return host, cache, rng


LENS = [0, 1, 31, 32, 33, 127, 128, 129, 160, 255, 256, 300, 1000, 2049]


@pytest.mark.parametrize("use_ws", [True, False])
@pytest.mark.parametrize("heads,group", [(1, 1), (2, 3), (2, 8), (1, 7), (1, 16), (1, 17), (1, 40), (3, 5)])
def test_attention_ragged(heads, group, use_ws):
    device()
    host, cache, rng = filled(heads, LENS, 100 + group)
    slots = [int(s) for s in rng.permutation(len(LENS)) + 1] + [-1, 0, host.slots, 5]
    q = rng.standard_normal((len(slots), heads * group, D)).astype(np.float16)
    note(f"paged attention heads={heads} group={group} workspace={use_ws}")
    lens = to_dev(host.lens)
    out = wq.kv_paged_attention(to_dev(q), cache, lens, seqs=i32(slots), use_workspace=use_ws)
    check_attention(out, host, q, slots, what="ragged")
    again = wq.kv_paged_attention(to_dev(q), cache, lens, seqs=i32(slots), use_workspace=use_ws)
    assert torch.equal(out, again)


@pytest.mark.parametrize("window", [1, 2, 31, 33, 100, 128, 129, 200, 257, 5000, 2 ** 40])
def test_attention_window(window):
    device()
    host, cache, rng = filled(2, LENS, 7)
    slots = list(range(1, len(LENS) + 1))
    q = rng.standard_normal((len(slots), 8, D)).astype(np.float16)
    note(f"paged attention window={window}")
    for use_ws in (True, False):
        out = wq.kv_paged_attention(to_dev(q), cache, to_dev(host.lens), seqs=i32(slots), window=window,
                                    use_workspace=use_ws)
        check_attention(out, host, q, slots, window=window, what=window)


@pytest.mark.parametrize("lens", [[1], [128], [20000], [3, 9000], [5] * 200, [130] * 70 + [0] * 10 + [4000]])
def test_attention_batch_shapes(lens):
    """One token, one long sequence, many short ones, many entries."""
    device()
    host, cache, rng = filled(2, lens, len(lens), extra_slots=1)
    slots = list(range(1, len(lens) + 1))
    q = rng.standard_normal((len(slots), 8, D)).astype(np.float16)
    note(f"paged attention entries={len(lens)} longest={max(lens)}")
    for use_ws in (True, False):
        out = wq.kv_paged_attention(to_dev(q), cache, to_dev(host.lens), seqs=i32(slots), use_workspace=use_ws)
        check_attention(out, host, q, slots, what="shapes")


def test_attention_values_of_unlike_size():
    """Scales from 2^-20 to 2^10: a token that takes nearly all of the weight but
    has tiny values, far and tiny queries; sharp and flat softmaxes."""
    device()
    rng = np.random.default_rng(21)
    n, heads = 700, 3
    K, V = draw_tokens(rng, n, heads)
    V[5] = (V[5].astype(np.float64) * 2.0 ** -12).astype(np.float16)
    V[:, 1] = (V[:, 1].astype(np.float64) * 2.0 ** -14).astype(np.float16)
    V[:, 2] = (V[:, 2].astype(np.float64) * 2.0 ** 9).astype(np.float16)
    K[:, 1] = (K[:, 1].astype(np.float64) * 2.0 ** -12).astype(np.float16)
    K[:, 2] = (K[:, 2].astype(np.float64) * 2.0 ** 5).astype(np.float16)
    host = Host(heads, 6, 1, 5)
    cache = gpu_cache(wq, host)
    append(wq, cache, host, [(0, K, V)])
    q = rng.standard_normal((1, heads * 4, D))
    q[:, 0] = 2.0 * K[5, 0]                    # points at the token of tiny values
    q[:, 1] *= 2.0 ** -13
    q[:, 5] *= 2.0 ** 10
    q[:, 6] = 0.0
    q[:, 9] *= 2.0 ** -6
    q = q.astype(np.float16)
    note("paged attention values of unlike size")
    for scale in (None, 0.01, -0.125, 0.0):
        got = wq.kv_paged_attention(to_dev(q), cache, to_dev(host.lens), scale=scale)
        ref, bound = host.attend(q, [0], scale=scale)
        d = np.abs(got.cpu().numpy().astype(np.float64) - ref)
        assert np.all(d <= bound), (scale, np.max(d / bound))


def test_attention_strides_and_untouched_rows():
    """q a part of a packed row, out a part of a larger buffer: the rows behind
    the last entry and the columns beside it stay as they were."""
    dev = device()
    host, cache, rng = filled(2, [77, 500, 128], 31)
    q = rng.standard_normal((3, 6, D)).astype(np.float16)
    row = torch.full((5, 11, D), 8.0, dtype=torch.float16, device=dev)
    row[:3, 2:8] = to_dev(q)
    buf = torch.full((5, 9, D), -2.0, dtype=torch.float16, device=dev)
    note("paged attention strided")
    out = wq.kv_paged_attention(row[:3, 2:8], cache, to_dev(host.lens), seqs=i32([1, 2, 3]), out=buf[:3, 1:7])
    check_attention(out, host, q, [1, 2, 3], what="strided")
    assert torch.all(buf[3:] == -2.0) and torch.all(buf[:, 0] == -2.0) and torch.all(buf[:, 7:] == -2.0)


def test_attention_masked_values_do_not_count():
    """Infinities and NaN in window rows past the sequence, in pages that belong
    to nobody and in another entry's blocks change nothing."""
    device()
    host, cache, rng = filled(2, [300, 40, 256], 41)
    q = rng.standard_normal((3, 4, D)).astype(np.float16)
    args = (to_dev(q), cache, to_dev(host.lens))
    note("paged attention with NaN around it")
    want = wq.kv_paged_attention(*args, seqs=i32([1, 2, 3]))
    for s, n in ((1, 300 % G), (2, 40), (3, 0)):
        cache.windows[s, :, :, n:] = float("nan")
        cache.windows[s, :, 1, n + 1:] = float("inf")
    used = {int(p) for s in (1, 2, 3) for p in host.table[s, :len(host.K[s]) // G]}
    for p in range(host.num_pages):
        if p not in used:
            cache.pages[p] = 0xFF              # NaN scales
    got = wq.kv_paged_attention(*args, seqs=i32([1, 2, 3]))
    assert torch.equal(got, want)
    check_attention(got, host, q, [1, 2, 3], what="nan around")
    cache.pages[int(host.table[1, 0])] = 0xFF  # a block that a window leaves out
    for use_ws in (True, False):
        got = wq.kv_paged_attention(*args, seqs=i32([1, 2, 3]), window=60, use_workspace=use_ws)
        check_attention(got, host, q, [1, 2, 3], window=60, what="window")


@pytest.mark.parametrize("use_ws", [True, False])
def test_attention_wrong_pages_give_nan(use_ws):
    """A page id that does not exist among the blocks that are read: NaN in that
    entry's rows only; past the blocks that are read it does not matter."""
    device()
    host, cache, rng = filled(2, [300, 700, 256, 2000], 51)
    q = rng.standard_normal((4, 4, D)).astype(np.float16)
    table = host.table.copy()
    table[1, 1], table[2, 0], table[4, 15:] = host.num_pages, -1, 10 ** 9
    cache.table.copy_(to_dev(table))
    note(f"paged attention wrong pages workspace={use_ws}")
    out = wq.kv_paged_attention(to_dev(q), cache, to_dev(host.lens), seqs=i32([1, 2, 3, 4]), use_workspace=use_ws)
    assert torch.isnan(out[:2]).all()
    check_attention(out[2:], host, q[2:], [3, 4], what="beside wrong pages")
    # Outside the window they are not read.
    out = wq.kv_paged_attention(to_dev(q), cache, to_dev(host.lens), seqs=i32([1, 2, 3, 4]), window=44,
                                use_workspace=use_ws)
    check_attention(out, host, q, [1, 2, 3, 4], window=44, what="window past wrong pages")


def test_attention_lengths_are_clamped():
    device()
    host, cache, rng = filled(1, [2 * G + 127], 61, max_pages=2)
    q = rng.standard_normal((2, 3, D)).astype(np.float16)
    note("paged attention clamped lengths")
    lens = i32([-4, 2 ** 31 - 1, 0])
    out = wq.kv_paged_attention(to_dev(q), cache, lens, seqs=i32([1, 0]))
    check_attention(out, host, q, [1, 0], what="clamped")


def test_attention_no_entries():
    dev = device()
    cache = wq.PagedKV(2, 1, 1, 1)
    out = wq.kv_paged_attention(torch.zeros((0, 4, D), dtype=torch.float16, device=dev), cache, i32([0]), seqs=i32([]))
    assert out.shape == (0, 4, D)


# ---- pages ----------------------------------------------------------------------

@pytest.mark.parametrize("heads,count", [(1, 1), (3, 7), (2, 500), (5, 900)])
def test_copy_pages(heads, count):
    device()
    rng = np.random.default_rng(count)
    P = 2 * count + 5
    cache = wq.PagedKV(heads, P, 1, 1)
    before = rng.integers(0, 256, (P, heads, REC)).astype(np.uint8)
    cache.pages.copy_(to_dev(before))
    ids = rng.permutation(P)
    src, dst = rng.choice(ids[:count], count), ids[count:2 * count]     # a source may stand twice
    note(f"paged copy heads={heads} count={count}")
    wq.kv_paged_copy(cache, np.stack([src, dst], 1))
    want = before.copy()
    want[dst] = before[src]
    assert np.array_equal(cache.pages.cpu().numpy(), want)
    wq.kv_paged_copy(cache, [])
    assert np.array_equal(cache.pages.cpu().numpy(), want)


def test_fork_shares_pages_and_goes_apart():
    device()
    host, cache, rng = filled(2, [300, 128, 50, 0], 71, extra_slots=6, max_pages=5)
    lens = to_dev(host.lens)
    windows, table = cache.windows.clone(), host.table.copy()
    pairs = [(1, 6), (1, 7), (2, 8), (3, 9), (4, 5)]
    note("paged fork")
    wq.kv_paged_fork(cache, lens, pairs)
    for a, b in pairs:
        n = len(host.K[a])
        windows[b, :, :, :n % G] = windows[a, :, :, :n % G]
        table[b, :n // G] = table[a, :n // G]
        host.K[b], host.V[b] = host.K[a], host.V[a]
    assert torch.equal(cache.windows, windows) and np.array_equal(cache.table.cpu().numpy(), table)
    assert np.array_equal(lens.cpu().numpy(), host.lens)
    host.table = table
    slots = [6, 1, 7, 8, 9, 5]
    q = rng.standard_normal((len(slots), 4, D)).astype(np.float16)
    check_attention(wq.kv_paged_attention(to_dev(q), cache, lens, seqs=i32(slots)), host, q, slots, what="forked")
    # The copies grow apart; their shared blocks stay.
    append(wq, cache, host, [(s, *draw_tokens(rng, n, 2)) for s, n in ((1, 90), (6, 85), (7, 3), (8, 1))])
    host.check_buffers(cache, "apart")


@pytest.mark.parametrize("pages,slots,blocks,live", [(1, 1, 1, 1), (40, 5, 12, 30), (40, 5, 12, 0), (300, 40, 20, 300),
                                                     (5000, 70, 100, 2500), (64, 3, 30, 5)])
def test_compact(pages, slots, blocks, live):
    dev = device()
    rng = np.random.default_rng(pages + live)
    cache = wq.PagedKV(1, pages, slots, blocks)
    before = rng.integers(0, 256, (pages, 1, REC)).astype(np.uint8)
    cache.pages.copy_(to_dev(before))
    ids = list(rng.permutation(pages)[:live])
    table = rng.integers(-3, pages + 3, (slots, blocks)).astype(np.int32)     # entries past a row's blocks: anything
    lens, use = np.zeros(slots, np.int32), []
    for s in range(slots):
        row = [ids.pop() for _ in range(min(len(ids), int(rng.integers(0, blocks + 1))))]
        if use and rng.random() < 0.3:                                         # shared blocks
            row = (use[:2] + row)[:blocks]
        if len(row) > 2 and rng.random() < 0.3:
            row[1] = -5                                                        # no page
        table[s, :len(row)] = row
        lens[s] = len(row) * G + int(rng.integers(0, G))
        use += [p for p in row if p >= 0]
    if slots > 2:
        lens[1] = -7                                                           # freed
    held = {int(table[s, b]) for s in range(slots) for b in range(max(lens[s], 0) // G)} - {-5}
    cache.table.copy_(to_dev(table))
    note(f"paged compact pages={pages} slots={slots} held={len(held)}")
    new, used = wq.kv_paged_compact(cache, to_dev(lens))
    n = int(used.item())
    assert n == len(held)
    new, after = new.cpu().numpy(), cache.pages.cpu().numpy()
    holes = [p for p in range(n) if p not in held]
    to = dict(zip(sorted(p for p in held if p >= n), holes))
    for s in range(slots):
        for b in range(blocks):
            p = int(table[s, b])
            want = -1 if b >= max(lens[s], 0) // G or p < 0 else to.get(p, p)
            assert new[s, b] == want, (s, b)
    want = before.copy()
    for p, h in to.items():
        want[h] = before[p]
    assert np.array_equal(after, want)
    assert np.array_equal(cache.table.cpu().numpy(), table)
    # Packed already: nothing moves.
    cache.table = to_dev(new)
    again, used = wq.kv_paged_compact(cache, to_dev(lens))
    assert int(used.item()) == n and np.array_equal(again.cpu().numpy(), new)
    assert np.array_equal(cache.pages.cpu().numpy(), want)


def test_compact_more_pages_than_a_range():
    """Past 262144 pages the plan works in ranges.  (One head: 4.6 GB of pages.)"""
    dev = device()
    P = 262144 + 5000
    cache = wq.PagedKV(1, P, 3, 400)
    rng = np.random.default_rng(1)
    rows = [rng.choice(100, 60, replace=False), 262144 + rng.choice(4900, 300, replace=False),
            np.array([262143, P - 1, 250000, 7])]
    lens, table = np.zeros(3, np.int32), np.full((3, 400), -1, np.int32)
    for s, r in enumerate(rows):
        table[s, :len(r)], lens[s] = r, len(r) * G
    held = sorted({int(p) for r in rows for p in r})
    mark = to_dev(np.arange(len(held), dtype=np.int32))
    cache.pages.view(torch.int32)[torch.tensor(held, device=dev), 0, 17] = mark
    cache.table.copy_(to_dev(table))
    note("paged compact past one range")
    new, used = wq.kv_paged_compact(cache, to_dev(lens))
    n = int(used.item())
    assert n == len(held)
    new = new.cpu().numpy()
    got = cache.pages.view(torch.int32)[:n, 0, 17].cpu().numpy()
    for s, r in enumerate(rows):
        for b, p in enumerate(r):
            assert 0 <= new[s, b] < n and got[new[s, b]] == held.index(int(p)), (s, b)
    assert np.all(new[0, 60:] == -1)


# ---- together -------------------------------------------------------------------

def _rope_ref(x, pos, freqs):
    a = (np.asarray(pos, np.float64)[:, None] * freqs)[:, None, :]
    u, w = x[..., :64].astype(np.float64), x[..., 64:].astype(np.float64)
    return np.concatenate([u * np.cos(a) - w * np.sin(a), u * np.sin(a) + w * np.cos(a)], -1)


class Server:
    """Decode steps over a packed q/k/v row, as a program runs them: rope on the
    row's q and k in place, append, attention; the host follows with what the
    GPU's rope gave (checked against float64 on the way)."""

    def __init__(self, heads, group, host, cache, seed):
        self.heads, self.group, self.host, self.cache = heads, group, host, cache
        self.rng = np.random.default_rng(seed)
        self.freqs = wq.rope_frequencies(D, base=10000.0)
        self.ws = wq.kv_paged_workspace(cache, host.slots, heads * group)

    def rows(self, n):
        H, q = self.heads, self.heads * self.group
        x = self.rng.standard_normal((n, q + 2 * H, D))
        x[:, q:q + H, 3] *= 8.0
        return x.astype(np.float16)

    def step(self, row, lens, seqs, pos, cu=None, attend=True):
        """The GPU calls of one layer's step; row [tokens, q_heads + 2 heads, 128]."""
        H, q = self.heads, self.heads * self.group
        wq.rope(row[:, :q + H], pos, self.freqs, out=row[:, :q + H])
        wq.kv_paged_append(row[:, q:q + H], row[:, q + H:], self.cache, lens, seqs=seqs, cu=cu)
        if attend:
            return wq.kv_paged_attention(row[:, :q], self.cache, lens, seqs=seqs, workspace=self.ws)

    def follow(self, raw, row, slots, counts, pos):
        """Takes the step into the host model; returns the rotated q."""
        H, q = self.heads, self.heads * self.group
        got = row.cpu().numpy()
        want = _rope_ref(raw[:, :q + H], pos, self.freqs.cpu().numpy())
        assert np.all(np.abs(got[:, :q + H].astype(np.float64) - want) <= 2.0 ** -10 * np.abs(raw[:, :q + H]).max())
        assert np.array_equal(bits16(got[:, q + H:]), bits16(raw[:, q + H:]))
        at = 0
        for s, n in zip(slots, counts):
            self.host.add(s, got[at:at + n, q:q + H], got[at:at + n, q + H:])
            at += n
        return got[:, :q]


@pytest.mark.parametrize("heads,group", [(2, 4), (3, 1)])
def test_server_run(heads, group):
    """Prompts, decode steps across block borders, a fork, more steps, a
    sequence that ends, a compaction, more steps."""
    device()
    host = Host(heads, 40, 6, 6, seed=3)
    cache = gpu_cache(wq, host)
    srv = Server(heads, group, host, cache, 5)

    def run(slots, counts, what):
        raw = srv.rows(sum(counts))
        start = host.lens.copy()
        pos = np.concatenate([start[s] + np.arange(n) for s, n in zip(slots, counts)]).astype(np.int32)
        row = to_dev(raw)
        lens = start.copy()
        lens[slots] += counts
        for s, n in zip(slots, counts):
            host.give_pages(s, n)
        cache.table.copy_(to_dev(host.table))
        prompt = max(counts) > 1
        cu = i32(np.concatenate([[0], np.cumsum(counts)])) if prompt else None
        out = srv.step(row, to_dev(lens), i32(slots), to_dev(pos), cu=cu, attend=not prompt)
        q = srv.follow(raw, row, slots, counts, pos)
        host.check_buffers(cache, what)
        if out is not None:
            check_attention(out, host, q, slots, what=what)

    note(f"server run heads={heads} group={group}")
    run([0, 2, 4], [200, 1, 381], "prompts")
    for i in range(4):
        run([2, 0, 4], [1, 1, 1], f"step {i}")               # slot 4 crosses a border
    lens = to_dev(host.lens)
    wq.kv_paged_fork(cache, lens, [(0, 1), (4, 5)])
    host.table = cache.table.cpu().numpy()
    for a, b in ((0, 1), (4, 5)):
        host.K[b], host.V[b] = host.K[a], host.V[a]
    run([0, 1, 2, 4, 5], [1] * 5, "forked")
    run([1, 5], [60, 127], "chunks")
    host.K[4], host.V[4] = host.K[4][:0], host.V[4][:0]      # ends
    table, used = wq.kv_paged_compact(cache, to_dev(host.lens))
    cache.table = table
    host.table, n = table.cpu().numpy(), int(used.item())
    host.free = list(range(host.num_pages - 1, n - 1, -1))
    host.check_buffers(cache, "compacted")
    run([0, 1, 2, 5], [1] * 4, "after")
    run([4], [140], "the freed slot again")
    run([5, 4, 0], [1, 1, 1], "last")


def test_replayed_graph_equals_eager_steps():
    """One captured decode step (lengths, positions and pages follow through
    device memory, a padded entry among them) replayed over a block border,
    with eager work between the replays, against the same steps run eagerly."""
    dev = device()
    heads, group, S = 2, 4, 4
    slots = [2, 0, -1, 3]
    states = []
    for _ in range(2):
        host, cache, _ = filled(heads, [125, 381, 60], 81, max_pages=4, extra_pages=12)
        states.append((host, cache, Server(heads, group, host, cache, 9)))
    host = states[0][0]
    table = host.table.copy()
    for s in (0, 2, 3):
        for b in range(len(host.K[s]) // G, 4):
            table[s, b] = host.free.pop()
    for _, cache, _ in states:
        cache.table.copy_(to_dev(table))
    steps, lens0 = 6, host.lens
    raws = [states[0][2].rows(S) for _ in range(steps)]
    seqs = i32(slots)

    def buffers():
        return dict(row=torch.zeros((S, heads * group + 2 * heads, D), dtype=torch.float16, device=dev),
                    lens=to_dev(lens0), pos=torch.zeros(S, dtype=torch.int32, device=dev),
                    real=i32([max(s, 0) for s in slots]).long())

    def step(srv, b):
        b["lens"].add_(1)
        b["pos"].copy_(b["lens"][b["real"]] - 1)
        return srv.step(b["row"], b["lens"], seqs, b["pos"])

    note("graph: eager steps")
    eager, b = [], buffers()
    for r in raws:
        b["row"].copy_(to_dev(r))
        eager.append(step(states[1][2], b).clone())
    note("graph: capture")
    b = buffers()
    cache, srv = states[0][1], states[0][2]
    windows, pages = cache.windows.clone(), cache.pages.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(srv, b)                                       # warm-up
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(srv, b)
    cache.windows.copy_(windows)
    cache.pages.copy_(pages)
    b["lens"].copy_(to_dev(lens0))
    for i, r in enumerate(raws):
        note(f"graph: replay {i}")
        b["row"].copy_(to_dev(r))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager[i]), i
        wq.kv_paged_attention(b["row"][:, :heads * group], cache, b["lens"], seqs=seqs)     # eager work between
        assert not out[2].any()
    assert torch.equal(cache.windows, states[1][1].windows) and torch.equal(cache.pages, states[1][1].pages)


def test_other_stream_and_two_graphs():
    """Calls on another stream than the default one; two graphs with workspaces
    of their own replayed at the same time."""
    dev = device()
    host, cache, rng = filled(2, [900, 2000, 64, 3000], 91)
    qs = [rng.standard_normal((4, 16, D)).astype(np.float16) for _ in range(2)]
    lens, seqs = to_dev(host.lens), i32([4, 3, 2, 1])
    want = [wq.kv_paged_attention(to_dev(q), cache, lens, seqs=seqs) for q in qs]
    torch.cuda.synchronize()
    note("paged attention on side streams")
    streams, graphs, outs = [torch.cuda.Stream() for _ in qs], [], []
    ins = [to_dev(q) for q in qs]
    torch.cuda.synchronize()
    for st, q in zip(streams, ins):
        ws = wq.kv_paged_workspace(cache, 4, 16)
        with torch.cuda.stream(st):
            got = wq.kv_paged_attention(q, cache, lens, seqs=seqs, workspace=ws)
        torch.cuda.synchronize()
        assert any(torch.equal(got, w) for w in want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            outs.append(wq.kv_paged_attention(q, cache, lens, seqs=seqs, workspace=ws))
        graphs.append((g, ws))
    for i in range(5):
        for st, (g, _) in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want)), i
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()


def test_refused_tensors():
    """What the binding refuses before any call."""
    dev = device()
    cache = wq.PagedKV(2, 4, 3, 2)
    f16 = torch.float16
    k = torch.zeros((3, 2, D), dtype=f16, device=dev)
    q = torch.zeros((3, 4, D), dtype=f16, device=dev)
    lens = torch.zeros(3, dtype=torch.int32, device=dev)
    app, att = wq.kv_paged_append, wq.kv_paged_attention
    for bad in [lambda: app(k.float(), k, cache, lens), lambda: app(k[:2], k, cache, lens),
                lambda: app(k[:, :1], k[:, :1], cache, lens), lambda: app(k.transpose(0, 1)[:, :2], k, cache, lens),
                lambda: app(k, k, cache, lens.long()), lambda: app(k, k, cache, lens[:2]),
                lambda: app(k, k, cache, lens, seqs=lens[:2]), lambda: app(k, k, cache, lens, cu=lens[:0]),
                lambda: app(k, k, cache, lens.cpu()), lambda: att(q[..., :64], cache, lens),
                lambda: att(q, cache, lens, out=q[:2]), lambda: att(q, cache, lens, workspace=q),
                lambda: att(q.transpose(0, 1), cache, lens), lambda: wq.kv_paged_copy(cache, [(0, 1, 2)]),
                lambda: wq.kv_paged_copy(cache, [(0.5, 1)]), lambda: wq.kv_paged_copy(cache, [(0, 2 ** 32 + 1)]),
                lambda: wq.PagedKV(pages=cache.pages[:, :, :100], windows=cache.windows, table=cache.table),
                lambda: wq.PagedKV(pages=cache.pages, windows=cache.windows[:, :1], table=cache.table),
                lambda: setattr(cache, "table", cache.table[:2])]:
        with pytest.raises(ValueError):
            bad()
    for bad in [lambda: att(q[:, :3], cache, lens), lambda: att(q, cache, lens, window=-1),
                lambda: att(q, cache, lens, scale=float("inf")),
                lambda: wq.kv_paged_copy(cache, [(0, 1), (2, 1)]), lambda: wq.kv_paged_copy(cache, [(0, 1), (1, 2)]),
                lambda: wq.kv_paged_copy(cache, [(0, 4)]), lambda: wq.kv_paged_copy(cache, [(-1, 0)]),
                lambda: wq.kv_paged_copy(cache, [(1, 1)]), lambda: wq.kv_paged_fork(cache, lens, [(0, 3)]),
                lambda: wq.kv_paged_compact(cache, lens, out=(cache.table, torch.zeros(1, dtype=torch.int32, device=dev))),
                lambda: app(torch.zeros((4, 2, D), dtype=f16, device=dev), torch.zeros((4, 2, D), dtype=f16, device=dev),
                            cache, lens),                       # more entries than slots
                lambda: wq.kv_paged_compact(cache, lens, workspace=torch.zeros(16, dtype=torch.uint8, device=dev))]:
        with pytest.raises(wq.WQError):
            bad()
