"""Cases of the paged KV cache's operators: rotary positions, append, decode
attention, and copying, forking and compacting pages.

A case is measured through the library's entry points (own = True) or in the
plain form below (own = False).

The cache of one layer: `pages` u8 [pages, heads, 17408], one record per page
and KV head holding 128 tokens of 128 channels:
    K codes u8 [128 tokens][64]    two channels a byte, even channel low
    V codes u8 [128 channels][64]  two tokens a byte, even token low
    K scales, K zeros fp16 [128]   one per channel
    V scales, V zeros fp16 [128]   one per token
`windows` fp16 [slots, heads, 2, 128, 128] (0 = K, 1 = V): the newest len % 128
tokens of the sequence in a slot; `table` int32 [slots, max_pages]: the page of
each whole block; `lens` int32 [slots]: tokens held by a slot.
"""

import math
import random

import numpy as np
import torch

own = False

G = 128                    # tokens of a block
D = 128                    # channels of a head
REC = 17408                # bytes of a page's record of one head
DEV = "cuda"


# ---- the cases ---------------------------------------------------------------

def listed():
    return [
        # Rotary positions.  One token of one sequence: 32 query and 32 key
        # heads (the 7B decode set's), the smallest call there is.
        dict(name="rope_one_token", op="rope", tokens=1, heads=64, dim=128, rot=128, layout="half",
             start=4095, factor=1.0),
        # A long prompt's chunk far into a stretched context, grouped heads
        # (64 query, 8 key).
        dict(name="rope_long_prompt", op="rope", tokens=8192, heads=72, dim=128, rot=128, layout="half",
             start=100000, factor=8.0),
        # An odd number of packed tokens, interleaved pairs on half of the head.
        dict(name="rope_part_of_head", op="rope", tokens=1777, heads=40, dim=128, rot=64, layout="interleaved",
             start=0, factor=1.0),
        # Append.  A decode step of 64 sequences, one of which fills its block.
        dict(name="append_decode", op="append", seqs=64, heads=8, new=1, longest=8192, whole=1, lengths=1),
        # Prompts and chunks of prompts of 16 sequences in one ragged batch.
        dict(name="append_prompts", op="append", seqs=16, heads=8, new=4096, longest=4096, whole=0, lengths=2),
        # Attention.  One short chat, 32 heads of their own (the 7B set's):
        # latency counts.
        dict(name="attention_one_short", op="attention", seqs=1, heads=32, group=1, longest=500, spread="equal",
             window=0, lengths=3),
        # A full batch at one length (the KV benchmark's 1024 heads of 4096 tokens).
        dict(name="attention_batch", op="attention", seqs=32, heads=32, group=1, longest=4096, spread="equal",
             window=0, lengths=4),
        # A serving batch of very unlike lengths, empty sequences among them,
        # grouped heads (64 query heads on 8).
        dict(name="attention_ragged", op="attention", seqs=64, heads=8, group=8, longest=16384, spread="log",
             window=0, lengths=5),
        # One long document, grouped heads.
        dict(name="attention_long", op="attention", seqs=1, heads=8, group=8, longest=131149, spread="equal",
             window=0, lengths=6),
        # Pages.  Eight sequences sampled four more times each.
        dict(name="fork_samples", op="fork", seqs=8, copies=4, heads=8, longest=4096, lengths=7),
        # A preempted batch's pages brought back to other places.
        dict(name="copy_pages", op="copy", pages=1024, count=400, heads=8),
        # A pool half empty after many sequences ended, packed for its resize.
        dict(name="compact_pool", op="compact", pages=4096, heads=8, slots=96, longest=8192, live=0.5, lengths=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "append", "attention", "attention", "attention", "fork", "copy", "compact"])
    heads = rng.choice([1, 2, 4, 5, 8, 8, 16, 32])
    seed = rng.randrange(1 << 30)
    if op == "rope":
        dim = rng.choice([64, 80, 96, 128, 128, 128, 256])
        n = rng.choice([1, 5, 12, 40, 64, 72])
        most = max(1, min(16384, 8192 * 72 * 128 // (n * dim)))
        return dict(op=op, tokens=_log(rng, 1, most), heads=n, dim=dim, rot=rng.choice([dim, dim, dim // 2]),
                    layout=rng.choice(["half", "interleaved"]), start=_log(rng, 1, 1 << 20) - 1,
                    factor=rng.choice([1.0, 4.0, 32.0]))
    if op == "append":
        if rng.random() < 0.5:
            seqs = _log(rng, 1, 256)
            return dict(op=op, seqs=seqs, heads=heads, new=1, longest=_log(rng, 1, 16384),
                        whole=min(seqs, rng.choice([0, 0, 1, 3])), lengths=seed)
        seqs = _log(rng, 1, 32)
        most = max(2, min(8192, 16 * 4096 * 8 // (seqs * heads)))
        return dict(op=op, seqs=seqs, heads=heads, new=_log(rng, 2, most), longest=_log(rng, 1, 8192), whole=0,
                    lengths=seed)
    if op == "attention":
        group = rng.choice([1, 1, 2, 4, 7, 8, 16, 24])
        seqs = _log(rng, 1, 128)
        most = max(2, min(131072, 32 * 32 * 4096 // (seqs * heads * max(1, group // 4))))
        return dict(op=op, seqs=seqs, heads=heads, group=group, longest=_log(rng, 1, most),
                    spread=rng.choice(["equal", "log", "log"]), window=rng.choice([0, 0, 0, 1, 1000, 4096]),
                    lengths=seed)
    if op == "fork":
        seqs = _log(rng, 1, 32)
        return dict(op=op, seqs=seqs, copies=rng.choice([1, 2, 4, 7]), heads=heads, longest=_log(rng, 1, 16384),
                    lengths=seed)
    if op == "copy":
        pages = _log(rng, 4, 8192 // heads)
        return dict(op=op, pages=pages, count=_log(rng, 1, pages // 2), heads=heads)
    pages = _log(rng, 4, 32768 // heads)
    return dict(op=op, pages=pages, heads=heads, slots=_log(rng, 1, 256), longest=_log(rng, 1, 16384),
                live=rng.choice([0.1, 0.5, 0.9, 1.0]), lengths=seed)


def _lengths(case):
    """Tokens held by each of the case's sequences."""
    rng = random.Random(case["lengths"])
    n, top = case["seqs"], case["longest"]
    if case.get("spread") == "equal":
        return [top] * n
    got = [0 if rng.random() < 1 / 16 else _log(rng, 1, top) for _ in range(n)]
    got[rng.randrange(n)] = top
    return got


def _append_plan(case):
    """(tokens before, new tokens) of each sequence.  A sequence begins at a
    block's border, ends at one, or stays inside its last block, as prompts,
    their chunks and single tokens do; so a pass writes nothing that a second
    pass over the same state would read."""
    rng = random.Random(case["lengths"])
    plan = []
    for i in range(case["seqs"]):
        old = _log(rng, 1, case["longest"])
        if case["new"] == 1:
            plan.append((old // G * G + G - 1 if i < case["whole"] else old - (old % G == G - 1), 1))
            continue
        n, kind = _log(rng, 1, case["new"]), i % 4
        if kind == 0:
            plan.append((0, n))
        elif kind == 1:
            plan.append((old // G * G, n))
        elif kind == 2:
            plan.append((old, n + (-(old + n)) % G))
        else:
            plan.append((old, min(n, max(0, G - 1 - old % G))))
    return plan


def _compact_plan(case):
    """Page ids [slots][blocks] of the live blocks; a slot may share the first
    blocks of the one before it."""
    rng = random.Random(case["lengths"])
    free = list(range(case["pages"]))
    rng.shuffle(free)
    free = free[:max(1, int(case["pages"] * case["live"]))]
    rows, lens = [], []
    most = max(1, case["longest"] // G)
    for s in range(case["slots"]):
        row = []
        if rng.random() < 0.9:
            if rows and rng.random() < 0.25:
                row = rows[-1][:rng.randrange(len(rows[-1]) + 1)]
            row = row + [free.pop() for _ in range(min(len(free), max(0, _log(rng, 1, most) - len(row))))]
        rows.append(row)
        lens.append(len(row) * G + rng.randrange(G))
    return rows, lens


def _moves(rows):
    live = sorted({p for row in rows for p in row})
    return sum(p >= len(live) for p in live)


def work(case):
    """Bytes and operations that one pass cannot do without."""
    op = case["op"]
    if op == "rope":
        n = case["tokens"] * case["heads"]
        return {"bytes": 4 * n * case["dim"] + 4 * case["tokens"] + 4 * case["rot"], "flops": 3 * n * case["rot"]}
    heads = case["heads"]
    if op == "append":
        total = 0
        for old, n in _append_plan(case):
            total += 512 * n                                            # the new tokens
            whole = (old + n) // G - old // G
            total += whole * REC + (512 * (old % G) if whole else 0)    # pages, and the rows their first block held
            total += 512 * min(n, (old + n) % G)                        # rows of the window
        return {"bytes": heads * total + 20 * case["seqs"], "flops": 0}
    if op == "attention":
        byte, seen = 0, 0
        for n in _lengths(case):
            left = max(0, n - case["window"]) if case["window"] else 0
            inside = max(0, n // G * G - left)
            byte += 136 * inside + 512 * (n - left - inside)
            seen += n - left
        rows = case["seqs"] * heads * case["group"]
        return {"bytes": heads * byte + 4 * D * rows + 8 * case["seqs"],
                "flops": 4 * D * heads * case["group"] * seen}
    if op == "fork":
        byte = sum(2 * 512 * heads * (n % G) + 8 * (n // G) + 8 for n in _lengths(case))
        return {"bytes": byte * case["copies"], "flops": 0}
    if op == "copy":
        return {"bytes": 2 * REC * heads * case["count"], "flops": 0}
    rows, _ = _compact_plan(case)
    return {"bytes": 2 * REC * heads * _moves(rows) + 8 * case["slots"] * max(1, case["longest"] // G + 1) + 4 * case["slots"],
            "flops": 0}


# ---- the codec ---------------------------------------------------------------

def _to_half(v):
    """v >= 0 (64 bits) rounded once to the nearest fp16 value, ties to even."""
    e = torch.frexp(v).exponent.clamp(min=-13) - 11
    step = (e.long() + 1023 << 52).view(torch.float64)      # 2^e from its bits: a device's pow(2, e) may be off
    return torch.round(v / step) * step


def _codec(x, dim):
    """4-bit codes, scales and zeros of fp16 x, a group being a line along dim.
    64 bits: every rounding decides as the exact quotient does."""
    x = x.double()
    lo, hi = x.amin(dim, keepdim=True), x.amax(dim, keepdim=True)
    s = _to_half((hi - lo) / 15)
    s = torch.where(s == 0, torch.ones_like(s), s)
    z = (torch.round(-lo / s) + 0.0).clamp(-65504, 65504).half()
    q = (torch.round(x / s) + z.double()).clamp(0, 15).to(torch.uint8)
    return q, s.half(), z


def _pack(q):
    return q[..., 0::2] | (q[..., 1::2] << 4)


def _unpack(c):
    return torch.stack((c & 15, c >> 4), -1).flatten(-2)


def _records(K, V):
    """Records u8 [..., 17408] of blocks K, V fp16 [..., 128 tokens, 128 channels]."""
    kq, ks, kz = _codec(K, -2)
    vq, vs, vz = _codec(V, -1)
    parts = [_pack(kq).flatten(-2), _pack(vq.transpose(-1, -2)).flatten(-2)]
    parts += [h.reshape(*K.shape[:-2], G).contiguous().view(torch.uint8) for h in (ks, kz, vs, vz)]
    return torch.cat(parts, -1)


def _halves(rec, at):
    """The fp16 [..., 128] at byte `at` of records, in 32 bits."""
    return rec[..., at:at + 256].contiguous().view(torch.float16).float()


# ---- the inputs --------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _noise(g, *shape):
    """u8 of any value."""
    n = math.prod(shape)
    return torch.randint(-(1 << 63), (1 << 63) - 1, (-(-n // 8),), generator=g, device=DEV,
                         dtype=torch.int64).view(torch.uint8)[:n].view(shape)


def _draw_kv(g, n):
    """K, V fp16 [n, 128, 128]: normal, with one hot key channel."""
    K, V = _randn(g, n, G, D), _randn(g, n, G, D)
    K[..., 3] *= 8.0
    return K.half(), V.half()


def _int(a):
    return torch.tensor(a, dtype=torch.int32, device=DEV)


def _frequencies(rot, factor):
    """Radians per token of each pair, 64 bits.  For a context stretched by
    `factor`, pairs that turn less than once within 4096 tokens are slowed by
    it, those of over 32 turns are left, and those between go over linearly."""
    f = 10000.0 ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    keep = np.clip((4096 * f / (2 * np.pi) - 1.0) / 31.0, 0.0, 1.0)
    return torch.from_numpy(f * keep + f / factor * (1 - keep)).to(DEV)


def prepare(case, seed):
    g, host, op = _gen(seed), np.random.default_rng(seed), case["op"]
    st = dict(op=op)
    if op == "rope":
        T, H, dim = case["tokens"], case["heads"], case["dim"]
        rows = _randn(g, T, H + max(1, H // 8), dim).half()     # q and k heads, then v heads
        factor = case["factor"]
        st.update(x=rows[:, :H], pos=torch.arange(case["start"], case["start"] + T, dtype=torch.int32, device=DEV),
                  freqs=_frequencies(case["rot"], factor), layout=case["layout"], rot=case["rot"],
                  scale=0.1 * math.log(factor) + 1.0)
        return st
    H = case["heads"]
    if op == "append":
        plan = _append_plan(case)
        S = len(plan)
        slots = S + S // 4 + 1
        blocks = max((old + n) // G for old, n in plan) + 1
        where = host.permutation(slots)[:S]
        lens = np.zeros(slots, np.int64)
        lens[where] = [old + n for old, n in plan]
        pages = slots * 2 + sum((old + n) // G - old // G for old, n in plan)
        table = host.integers(0, pages, (slots, blocks))        # old blocks: any page
        fresh = host.permutation(pages)
        for s, (old, n) in zip(where, plan):
            count = (old + n) // G - old // G
            table[s, old // G:old // G + count], fresh = fresh[:count], fresh[count:]
        T = sum(n for _, n in plan)
        qkv = _randn(g, T, 6 * H, D)                            # 4 query heads to a KV head
        qkv[:, 4 * H:5 * H, 3] *= 8.0
        qkv = qkv.half()
        cu = np.concatenate([[0], np.cumsum([n for _, n in plan])])
        st.update(k=qkv[:, 4 * H:5 * H], v=qkv[:, 5 * H:], pages=torch.zeros((pages, H, REC), dtype=torch.uint8, device=DEV),
                  windows=_randn(g, slots, H, 2, G, D).half(), table=_int(table), lens=_int(lens), seqs=_int(where),
                  cu=_int(cu) if case["new"] > 1 else None)
        return st
    if op == "attention":
        held = _lengths(case)
        S = len(held)
        slots = S + S // 4 + 1
        where = host.permutation(slots)[:S]
        lens = np.zeros(slots, np.int64)
        lens[where] = held
        pages = max(1, sum(n // G for n in held))
        ids, table = host.permutation(pages), np.zeros((slots, max(held) // G + 1), np.int64)
        for s, n in zip(where, held):
            table[s, :n // G], ids = ids[:n // G], ids[n // G:]
        rec = torch.empty((pages * H, REC), dtype=torch.uint8, device=DEV)
        for at in range(0, pages * H, 4096):
            K, V = _draw_kv(g, min(4096, pages * H - at))
            rec[at:at + 4096] = _records(K, V)
        K, V = _draw_kv(g, slots * H)
        windows = torch.stack((K, V), 1).view(slots, H, 2, G, D)
        Hq = H * case["group"]
        st.update(q=_randn(g, S, Hq + 2 * H, D).half()[:, :Hq], pages=rec.view(pages, H, REC), windows=windows,
                  table=_int(table), lens=_int(lens), seqs=_int(where), window=case["window"])
        return st
    if op == "fork":
        held = _lengths(case)
        S, n = len(held), case["copies"]
        slots = S * (n + 1)
        order = host.permutation(slots)
        pairs = np.stack([np.repeat(order[:S], n), order[S:]], 1).astype(np.int32)
        blocks = max(held) // G + 1
        lens = np.zeros(slots, np.int64)
        lens[order[:S]] = held
        pages = max(1, sum(n // G for n in held))
        ids, table = host.permutation(pages), np.full((slots, blocks), -1)
        for s, h in zip(order, held):
            table[s, :h // G], ids = ids[:h // G], ids[h // G:]
        st.update(pairs=pairs, pages=_noise(g, 1, H, REC).expand(pages, H, REC), windows=_randn(g, slots, H, 2, G, D).half(),
                  table=_int(table), lens=_int(lens))
        st["pages"] = st["pages"].contiguous()
        return st
    P = case["pages"]
    st["pages"] = _noise(g, P, H, REC)
    if op == "copy":
        ids = host.permutation(P)[:2 * case["count"]].astype(np.int32)
        st["pairs"] = np.ascontiguousarray(ids.reshape(2, -1).T)
        st.update(windows=torch.zeros((1, H, 2, G, D), dtype=torch.float16, device=DEV), table=_int([[0]]))
        return st
    rows, lens = _compact_plan(case)
    blocks = max(1, case["longest"] // G + 1, *(len(r) for r in rows))
    table = host.integers(0, P, (len(rows), blocks))            # what lies past a row's blocks is not in use
    for s, r in enumerate(rows):
        table[s, :len(r)] = r
    st.update(windows=torch.zeros((len(rows), H, 2, G, D), dtype=torch.float16, device=DEV), table=_int(table),
              lens=_int(lens))
    return st


# ---- one pass ----------------------------------------------------------------

def run(st):
    return _kernels(st) if own else _PLAIN[st["op"]](st)


def _handle(st):
    """The library's view of the state's cache, which a program keeps."""
    import bit_weight_only_wq_amd as wq
    if "cache" not in st:
        st["cache"] = wq.PagedKV(pages=st["pages"], windows=st["windows"], table=st["table"])
    return wq, st["cache"]


def _kernels(st):
    op = st["op"]
    if op == "rope":
        import bit_weight_only_wq_amd as wq
        return wq.rope(st["x"], st["pos"], st["freqs"], layout=st["layout"], scale=st["scale"])
    wq, cache = _handle(st)
    if op == "append":
        wq.kv_paged_append(st["k"], st["v"], cache, st["lens"], seqs=st["seqs"], cu=st["cu"])
        return {"pages": st["pages"], "windows": st["windows"]}
    if op == "attention":
        if "workspace" not in st:
            st["workspace"] = wq.kv_paged_workspace(cache, st["q"].shape[0], st["q"].shape[1])
        return wq.kv_paged_attention(st["q"], cache, st["lens"], seqs=st["seqs"], window=st["window"],
                                     workspace=st["workspace"])
    if op == "fork":
        wq.kv_paged_fork(cache, st["lens"], st["pairs"])
        return {"windows": st["windows"], "table": st["table"], "lens": st["lens"]}
    if op == "copy":
        wq.kv_paged_copy(cache, st["pairs"])
        return {"pages": st["pages"]}
    if "workspace" not in st:
        st["workspace"] = wq.kv_paged_compact_workspace(cache)
    table, used = wq.kv_paged_compact(cache, st["lens"], workspace=st["workspace"])
    return {"pages": st["pages"], "table": table, "used": used}


def _plain_rope(st):
    # Angles of far positions need 64 bits; the rotation itself 32.
    x, rot = st["x"].float(), st["rot"]
    angle = st["pos"].double()[:, None, None] * st["freqs"]
    c, s = (angle.cos() * st["scale"]).float(), (angle.sin() * st["scale"]).float()
    y = x.clone()
    if st["layout"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, a * s + b * c
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, a * s + b * c
    return y.half()


def _plain_append(st):
    k, v, windows, table = st["k"], st["v"], st["windows"], st["table"]
    T, S = k.shape[0], st["seqs"].shape[0]
    slot = st["seqs"].long()
    cu = st["cu"].long() if st["cu"] is not None else torch.arange(S + 1, device=DEV)
    new = cu[1:] - cu[:-1]
    after = st["lens"].long()[slot]
    start = after - new
    kv = torch.stack((k, v), 2)                                      # [T, H, 2, D]
    # Blocks that become whole: their tokens from the window and from the call.
    whole = after // G - start // G
    count = int(whole.sum())
    e = torch.repeat_interleave(torch.arange(S, device=DEV), whole, output_size=count)
    block = (start // G)[e] + torch.arange(count, device=DEV) - (whole.cumsum(0) - whole)[e]
    at = block[:, None] * G + torch.arange(G, device=DEV)            # positions [count, 128]
    old = windows[slot[e][:, None], :, :, at % G]                    # [count, 128, H, 2, D]
    fresh = kv[(cu[e][:, None] + at - start[e][:, None]).clamp(0, max(0, T - 1))]
    rows = torch.where((at < start[e][:, None])[..., None, None, None], old, fresh)
    rows = rows.permute(3, 0, 2, 1, 4)                               # [2, count, H, 128, D]
    st["pages"][table.long()[slot[e], block]] = _records(rows[0], rows[1])
    # Tokens of the last, unfinished block go to the window.
    te = torch.repeat_interleave(torch.arange(S, device=DEV), new, output_size=T)
    pos = start[te] + torch.arange(T, device=DEV) - cu[te]
    keep = pos >= (after // G * G)[te]
    windows[slot[te][keep], :, :, pos[keep] % G] = kv[keep]
    return {"pages": st["pages"], "windows": windows}


def _plain_attention(st):
    pages, windows = st["pages"], st["windows"]
    slot = st["seqs"].long()
    S, H = slot.shape[0], pages.shape[1]
    held = st["lens"].long()[slot]
    blocks = st["table"].shape[1] - 1
    rec = pages[st["table"].long()[slot, :blocks].clamp(min=0)]      # [S, blocks, H, 17408]
    K = _unpack(rec[..., :8192].reshape(S, blocks, H, G, D // 2)).float()
    K = (K - _halves(rec, 16640)[..., None, :]) * _halves(rec, 16384)[..., None, :]
    V = _unpack(rec[..., 8192:16384].reshape(S, blocks, H, D, G // 2)).float().transpose(-1, -2)
    V = (V - _halves(rec, 17152)[..., None]) * _halves(rec, 16896)[..., None]
    # Whole blocks, then the window, as one line of tokens.
    win = windows[slot].float()
    K = torch.cat((K.transpose(1, 2).reshape(S, H, blocks * G, D), win[:, :, 0]), 2)
    V = torch.cat((V.transpose(1, 2).reshape(S, H, blocks * G, D), win[:, :, 1]), 2)
    place = torch.arange(blocks * G + G, device=DEV)
    pos = torch.where(place < blocks * G, place, held[:, None] // G * G + place - blocks * G)
    seen = torch.where(place < blocks * G, pos < held[:, None] // G * G, pos < held[:, None])
    if st["window"]:
        seen = seen & (pos >= held[:, None] - st["window"])
    seen = seen[:, None, :, None]
    q = st["q"].float().view(S, H, -1, D).transpose(-1, -2).contiguous()
    s = torch.where(seen, torch.matmul(K, q) / math.sqrt(D), -math.inf)    # [S, H, tokens, group]
    top = s.amax(2, keepdim=True)
    p = torch.where(seen, torch.exp(s - torch.where(top.isfinite(), top, 0.0)), 0.0)
    o = torch.matmul(p.transpose(-1, -2).contiguous(), V)
    total = p.sum(2)[..., None]
    o = torch.where(total > 0, o / total, 0.0)
    return o.reshape(S, -1, D).half()


def _plain_fork(st):
    windows, table, lens = st["windows"], st["table"], st["lens"]
    pairs = torch.from_numpy(st["pairs"]).to(DEV).long()
    src, dst = pairs[:, 0], pairs[:, 1]
    held = lens[src].long()
    row = torch.arange(G, device=DEV) < held[:, None] % G
    windows[dst] = torch.where(row[:, None, None, :, None], windows[src], windows[dst])
    block = torch.arange(table.shape[1], device=DEV) < held[:, None] // G
    table[dst] = torch.where(block, table[src], table[dst])
    lens[dst] = lens[src]
    return {"windows": windows, "table": table, "lens": lens}


def _plain_copy(st):
    pairs = torch.from_numpy(st["pairs"]).to(DEV).long()
    st["pages"][pairs[:, 1]] = st["pages"][pairs[:, 0]]
    return {"pages": st["pages"]}


def _plain_compact(st):
    pages, table = st["pages"], st["table"].long()
    used = torch.arange(table.shape[1], device=DEV) < st["lens"].long()[:, None] // G
    live = torch.zeros(pages.shape[0], dtype=torch.bool, device=DEV)
    live[table[used]] = True
    n = int(live.sum())
    holes, movers = (~live[:n]).nonzero()[:, 0], live[n:].nonzero()[:, 0] + n
    to = torch.arange(pages.shape[0], device=DEV)
    to[movers] = holes
    pages[holes] = pages[movers]
    table = torch.where(used, to[table.clamp(min=0)], -1).int()
    return {"pages": pages, "table": table, "used": torch.full((1,), n, dtype=torch.int32, device=DEV)}


_PLAIN = {"rope": _plain_rope, "append": _plain_append, "attention": _plain_attention, "fork": _plain_fork,
          "copy": _plain_copy, "compact": _plain_compact}


# ---- the definitions in 64 bits ------------------------------------------------

def exact(case, seed):
    """From the definitions, in 64 bits or whole numbers.  Copies and
    compactions only move bytes."""
    op = case["op"]
    if op in ("copy", "compact"):
        return None
    st = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "attention": _exact_attention, "fork": _exact_fork}[op](st)


def _exact_fork(st):
    windows, table, lens = st["windows"].double(), st["table"].clone(), st["lens"].clone()
    for a, b in st["pairs"].tolist():
        n = int(lens[a])
        windows[b, :, :, :n % G] = windows[a, :, :, :n % G]
        table[b, :n // G] = table[a, :n // G]
        lens[b] = n
    return {"windows": windows, "table": table, "lens": lens}


def _exact_rope(st):
    """Each pair as a complex number times scale * exp(i position frequency)."""
    x, rot = st["x"].double(), st["rot"]
    turn = torch.polar(torch.full_like(st["freqs"], st["scale"]).expand(x.shape[0], -1),
                       st["pos"].double()[:, None] * st["freqs"])[:, None]
    if st["layout"] == "half":
        y = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * turn
        return torch.cat((y.real, y.imag, x[..., rot:]), -1)
    y = torch.view_as_real(torch.view_as_complex(x[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * turn)
    return torch.cat((y.flatten(-2), x[..., rot:]), -1)


def _nearest(a, b):
    """a / b in whole numbers, b > 0, to the nearest, ties to even."""
    q = torch.div(a, b, rounding_mode="floor")
    r = 2 * (a - q * b)
    return q + ((r > b) | ((r == b) & (q % 2 == 1))).long()


def _whole_codec(x, dim):
    """The codec in whole multiples of 2^-24, which every fp16 value is."""
    u = (x.double() * 2.0 ** 24).long()
    lo, hi = u.amin(dim, keepdim=True), u.amax(dim, keepdim=True)
    span = hi - lo
    size = sum((span >= 15 << k).long() for k in range(11, 42))    # bits of span / 15 past the 11 that are kept
    s = _nearest(span, 15 << size) << size
    s = torch.where(s == 0, 1 << 24, s)
    z = _nearest(-lo, s).clamp(-65504, 65504)
    more = sum((z.abs() >= 1 << k).long() for k in range(11, 17))
    z = _nearest(z, 1 << more) << more
    q = (_nearest(u, s) + z).clamp(0, 15)
    half = lambda w: w.half().flatten(1).contiguous().view(torch.uint8)  # noqa: E731
    return q, half(s.double() * 2.0 ** -24), half(z.double())


def _exact_append(st):
    slots, cu, lens = st["seqs"].tolist(), st["cu"], st["lens"].tolist()
    cu = cu.tolist() if cu is not None else list(range(len(slots) + 1))
    windows = st["windows"].double()
    for i, s in enumerate(slots):
        n = cu[i + 1] - cu[i]
        start = lens[s] - n
        held = start % G
        for side, new in enumerate((st["k"], st["v"])):
            line = torch.cat((st["windows"][s, :, side, :held], new[cu[i]:cu[i + 1]].transpose(0, 1)), 1)   # [H, tokens, D]
            for b in range(line.shape[1] // G):
                page = st["pages"][int(st["table"][s, start // G + b])]
                q, sc, ze = _whole_codec(line[:, b * G:(b + 1) * G], 1 if side == 0 else 2)
                if side:
                    q = q.transpose(1, 2)
                page[:, side * 8192:side * 8192 + 8192] = (q[..., 0::2] + 16 * q[..., 1::2]).flatten(1).to(torch.uint8)
                page[:, 16384 + 512 * side:16640 + 512 * side] = sc
                page[:, 16640 + 512 * side:16896 + 512 * side] = ze
            if (start + n) // G > start // G:
                held_now, rest = 0, line[:, line.shape[1] // G * G:]
            else:
                held_now, rest = held, line[:, held:]
            windows[s, :, side, held_now:held_now + rest.shape[1]] = rest.double()
    return {"pages": st["pages"], "windows": windows}


def _exact_attention(st):
    slots, lens, H = st["seqs"].tolist(), st["lens"].tolist(), st["pages"].shape[1]
    q = st["q"].double()
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    for i, s in enumerate(slots):
        n = lens[s]
        first = max(0, n - st["window"]) if st["window"] else 0
        if n == first:
            continue
        b0, b1 = first // G, n // G
        rec = st["pages"][st["table"][s, b0:b1].long()].transpose(0, 1)             # [H, blocks, 17408]
        head = lambda at: rec[..., at:at + 256].contiguous().view(torch.float16).double()  # noqa: E731
        codes = rec[..., :16384].reshape(H, -1, 2, 128, 64)
        codes = torch.stack((codes % 16, codes // 16), -1).reshape(H, -1, 2, 128, 128).double()
        K = ((codes[:, :, 0] - head(16640).unsqueeze(2)) * head(16384).unsqueeze(2)).flatten(1, 2)
        V = ((codes[:, :, 1] - head(17152).unsqueeze(2)) * head(16896).unsqueeze(2)).transpose(2, 3).flatten(1, 2)
        win = st["windows"][s].double()
        K = torch.cat((K, win[:, 0, :n % G]), 1)[:, first - b0 * G if b0 < b1 else first - b1 * G:]
        V = torch.cat((V, win[:, 1, :n % G]), 1)[:, first - b0 * G if b0 < b1 else first - b1 * G:]
        p = torch.softmax(torch.matmul(q[i].view(H, -1, D), K.transpose(1, 2).contiguous()) * D ** -0.5, -1)
        out[i] = torch.matmul(p, V).view(-1, D)
    return out
