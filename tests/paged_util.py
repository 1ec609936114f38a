"""Host model of the paged KV cache for the GPU tests: what every slot holds as
fp16 tokens, a page allocator, and what the buffers must contain.  The codec
and the attention come from the CPU oracle."""

import numpy as np

import oracle.kv as okv
from gpu_util import to_dev

G = D = 128
REC = 17408


def draw_tokens(rng, n, heads):
    """fp16 K, V [n, heads, 128]: normal, with one hot key channel."""
    K, V = rng.standard_normal((2, n, heads, D))
    K[..., 3] *= 8.0
    return K.astype(np.float16), V.astype(np.float16)


def record(K, V):
    """u8 [17408]: the record of one block, K, V fp16 [128, 128]."""
    b = okv.quantize_block(K, V)
    parts = [b["kcodes"], b["vcodes"], b["ks"], b["kz"], b["vs"], b["vz"]]
    return np.concatenate([np.ascontiguousarray(p).reshape(-1).view(np.uint8) for p in parts])


class Host:
    """What each slot should hold."""

    def __init__(self, heads, num_pages, slots, max_pages, seed=0):
        self.heads, self.num_pages, self.slots, self.max_pages = heads, num_pages, slots, max_pages
        self.K = [np.zeros((0, heads, D), np.float16) for _ in range(slots)]
        self.V = [np.zeros((0, heads, D), np.float16) for _ in range(slots)]
        self.free = list(np.random.default_rng(seed).permutation(num_pages))
        self.table = np.full((slots, max_pages), -1, np.int32)

    @property
    def lens(self):
        return np.array([len(k) for k in self.K], np.int32)

    def give_pages(self, slot, n):
        """Pages for the blocks that n more tokens of a slot complete."""
        old = len(self.K[slot])
        for b in range(old // G, (old + n) // G):
            self.table[slot, b] = self.free.pop()

    def add(self, slot, K, V):
        self.K[slot] = np.concatenate([self.K[slot], K])
        self.V[slot] = np.concatenate([self.V[slot], V])

    def cached(self, slot, h):
        """K, V float64 [tokens, 128] as the cache gives them back."""
        n = len(self.K[slot])
        Ks, Vs = [], []
        for b in range(n // G):
            k, v = okv.dequantize_block(okv.quantize_block(self.K[slot][b * G:(b + 1) * G, h],
                                                           self.V[slot][b * G:(b + 1) * G, h]))
            Ks.append(k)
            Vs.append(v)
        Ks.append(self.K[slot][n // G * G:, h].astype(np.float64))
        Vs.append(self.V[slot][n // G * G:, h].astype(np.float64))
        return np.concatenate(Ks), np.concatenate(Vs)

    def attend(self, q, slots, window=0, scale=None):
        """(reference, bound on the error) float64 of q [entries, q_heads, 128].

        The bound: with sums in fp32 a score is off by at most
        d = 2^-17 * scale * sum_c |q_c| m_c, m_c the largest magnitude that
        channel's term (c and z apart) reaches (128 terms of relative error
        2^-24 each, and operands split into two halves of 11 bits, 2^-22); the
        weights then by a factor within exp(+-2d), the values' sum by 2^-16 of
        its largest term; the fp16 result by half a step, 2^-11 relative, or
        2^-25 for a subnormal one."""
        S, Hq, _ = q.shape
        R = Hq // self.heads
        ref, bound = np.zeros((S, Hq, D)), np.zeros((S, Hq, D))
        scale = D ** -0.5 if scale is None else scale
        for i, s in enumerate(slots):
            if s < 0 or s >= self.slots or len(self.K[s]) == 0:
                continue
            for h in range(self.heads):
                K, V = self.cached(s, h)
                first = max(0, len(K) - window) if window else 0
                qh = q[i, h * R:(h + 1) * R].astype(np.float64)
                # |c s| and |z s| apart reach at most 3 times a block's largest |x|
                # for data whose range includes zero (range <= 2 max).
                mk = 3.0 * np.abs(K).max(0)
                d = 2.0 ** -17 * abs(scale) * (np.abs(qh) @ mk)
                for r in range(R):
                    ref[i, h * R + r] = okv.attend(qh[r], K[first:], V[first:], scale)
                b = 3.0 * np.abs(V[first:]).max() * (np.expm1(2 * d) + 2.0 ** -16)
                bound[i, h * R:(h + 1) * R] = b[:, None]
        return ref, bound + 2.0 ** -11 * np.abs(ref) + 2.0 ** -25

    def check_buffers(self, cache, what=""):
        """Every page a slot holds, and every window row in use, bit for bit."""
        pages, windows = cache.pages.cpu().numpy(), cache.windows.cpu().numpy()
        table = cache.table.cpu().numpy()
        for s in range(self.slots):
            n = len(self.K[s])
            for b in range(n // G):
                for h in range(self.heads):
                    want = record(self.K[s][b * G:(b + 1) * G, h], self.V[s][b * G:(b + 1) * G, h])
                    assert np.array_equal(pages[table[s, b], h], want), (what, s, b, h)
            r = n % G
            for side, X in enumerate((self.K[s], self.V[s])):
                want = X[n - r:].transpose(1, 0, 2)
                got = windows[s, :, side, :r]
                assert np.array_equal(got.view(np.uint16), np.ascontiguousarray(want).view(np.uint16)), (what, s, side)


def gpu_cache(wq, host):
    """A cache of the host's sizes, its pages and windows filled with a marker."""
    cache = wq.PagedKV(host.heads, host.num_pages, host.slots, host.max_pages)
    cache.pages.fill_(0xA5)
    cache.windows.fill_(-7.0)
    cache.table.copy_(to_dev(host.table))
    return cache


def append(wq, cache, host, items, seqs=None, cu=True, packed=False):
    """Append (slot, K, V) items to the GPU cache, in one call, and to the host."""
    slots = [s for s, _, _ in items]
    for s, K, V in items:
        host.give_pages(s, len(K))
        host.add(s, K, V)
    cache.table.copy_(to_dev(host.table))
    K = np.concatenate([k for _, k, _ in items])
    V = np.concatenate([v for _, _, v in items])
    if packed:                                   # parts of one q/k/v row
        H = host.heads
        row = np.zeros((len(K), 4 * H, D), np.float16)
        row[:, 2 * H:3 * H], row[:, 3 * H:] = K, V
        row = to_dev(row)
        k, v = row[:, 2 * H:3 * H], row[:, 3 * H:]
    else:
        k, v = to_dev(K), to_dev(V)
    counts = [len(k_) for _, k_, _ in items]
    cu_t = to_dev(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)) if cu else None
    wq.kv_paged_append(k, v, cache, to_dev(host.lens), seqs=to_dev(np.array(slots, np.int32)), cu=cu_t)
