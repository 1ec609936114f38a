"""Accuracy of the paged decode attention where its factors are far from 1: keys
with small or unlike scales, values of unlike size in one block, headers that no
quantizer writes, and scores so far out that their fp32 steps are whole powers
of two.  Every check is against 64 bits, head by head."""

import numpy as np
import pytest

import oracle.kv as okv
from gpu_util import L2_REL, device, note, to_dev
from paged_util import D, G, REC, Host, append, gpu_cache

import bit_weight_only_wq_amd as wq

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

GROUPS = [1, 4, 8, 16]          # the kernel's forms: up to 4, 8 and 16 heads of a row


def head_errors(got, ref):
    """Relative L2 error of every query head [entries, heads]."""
    got = got.cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(got))
    return np.linalg.norm(got - ref, axis=-1) / np.linalg.norm(ref, axis=-1)


def held(K, V, pages=16):
    """Host and GPU cache of one slot that holds fp16 K, V [n, heads, 128]."""
    host = Host(K.shape[1], pages, 1, max(len(K) // G, 1))
    cache = gpu_cache(wq, host)
    append(wq, cache, host, [(0, K, V)])
    return host, cache


# Every head's relative L2 error is held to L2_REL = 1e-3.  Of that the fp16
# result takes at most 2^-11 = 4.9e-4.  A score is a sum of 128 products |q_c|
# |c s| and as many with z, in natural units 0.088 * 128 * 0.8 * (3.3 + 3.3) = 60
# here for keys about zero and 0.088 * 128 * 0.8 * (13 + 6.6) = 177 for keys ten
# deviations off it; sums in fp32 leave sqrt(256) * 2^-24 of that at random,
# 6e-5 and 1.7e-4, and factors of 22 bits 2^-22 / sqrt(128) of it, 4e-6.  Errors of
# unlike tokens average as the values do, so the output takes them over about
# once: below 5e-4 with a factor of three to spare.
@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("down,up,mean,scale", [(7, 7, 10.0, None), (10, 10, 0.0, None), (10, 10, 10.0, None),
                                                (13, 13, 0.0, None), (16, 13, 0.0, 8 * 128 ** -0.5)])
def test_small_key_scales(group, down, up, mean, scale):
    """K at 2^-down and q at 2^up: the same scores as of K and q about 1."""
    device()
    rng = np.random.default_rng(100 * group + down)
    n, heads = 8 * G + 41, 2
    K, V = rng.standard_normal((2, n, heads, D))
    K = ((K + mean * rng.choice([-1.0, 1.0], (1, heads, D))) * 2.0 ** -down).astype(np.float16)
    q = (rng.standard_normal((1, heads * group, D)) * 2.0 ** up).astype(np.float16)
    host, cache = held(K, V.astype(np.float16))
    note(f"paged attention small key scales group={group} 2^-{down} mean {mean}")
    for use_ws in (True, False):
        got = wq.kv_paged_attention(to_dev(q), cache, to_dev(host.lens), scale=scale, use_workspace=use_ws)
        assert head_errors(got, host.attend(q, [0], scale=scale)[0]).max() <= L2_REL


@pytest.mark.parametrize("group", GROUPS)
def test_unlike_key_scales(group):
    """Channels of K from 2^-13 to 1 and of q from 2^13 to 1, block by block other
    ones, so that every channel has its part in the scores."""
    device()
    rng = np.random.default_rng(group)
    n, heads = 6 * G, 2
    K, V = rng.standard_normal((2, n, heads, D))
    x = rng.integers(0, 14, (heads, D))
    K = (K * 2.0 ** -x).astype(np.float16)
    K[2 * G:4 * G] *= np.float16(0.25)
    q = (rng.standard_normal((1, heads, group, D)) * 2.0 ** x[:, None]).astype(np.float16).reshape(1, -1, D)
    host, cache = held(K, V.astype(np.float16))
    note(f"paged attention unlike key scales group={group}")
    for use_ws in (True, False):
        got = wq.kv_paged_attention(to_dev(q), cache, to_dev(host.lens), use_workspace=use_ws)
        assert head_errors(got, host.attend(q, [0])[0]).max() <= L2_REL


# The bound below: a weight keeps 22 bits down to 2^-10 of the largest weight
# times scale among the tokens it stands with, the values' sums 2^-16 of their
# largest term; the result is rounded to fp16, by at most 2^-11 or, subnormal,
# 2^-25.
@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("winner,loud", [(5, 2), (64, 71), (127, 120), (100, 30)])
def test_small_values_beside_large(group, winner, loud):
    """Two tokens share all of the weight, 1 to 3 to 1 to 1, and have values of 2^-14;
    another of their block, far below them in score, has the largest values there
    are."""
    device()
    rng = np.random.default_rng(winner)
    heads, n = 2, G + 7
    K = rng.standard_normal((n, heads, D)).astype(np.float16)
    second = winner ^ 3
    K[second] = K[winner]
    V = rng.standard_normal((n, heads, D)) * 2.0 ** -14
    V[loud] = rng.choice([-60000.0, 60000.0], (heads, D))
    V = V.astype(np.float16)
    q = np.repeat(8.0 * K[winner].astype(np.float64), group, 0)[None]
    q = (q * (1 + rng.random(q.shape) / 4)).astype(np.float16)
    K[second] *= np.float16(1 - 2.0 ** -7)
    host, cache = held(K, V)
    note(f"paged attention small values beside large group={group} {winner} {loud}")
    ref, _ = host.attend(q, [0])
    for h in range(heads):
        k, v = host.cached(0, h)
        for r in range(group):
            s = k @ q[0, h * group + r].astype(np.float64) * D ** -0.5
            assert s[winner] - np.delete(s, [winner, second]).max() > 40          # (60000 e^-40 is below 2^-41)
        top = np.abs(v[winner]).max()
        for use_ws in (True, False):
            got = wq.kv_paged_attention(to_dev(q), cache, to_dev(host.lens), use_workspace=use_ws)
            d = np.abs(got.cpu().numpy().astype(np.float64) - ref)[0, h * group:(h + 1) * group]
            assert np.all(d <= 2.0 ** -16 * top + 2.0 ** -11 * np.abs(ref[0, h * group:(h + 1) * group]) + 2.0 ** -25)


def test_sizes_apart_head_by_head():
    """Keys of 2^-12, 1 and 2^5 and values of 2^-10, 1 and 2^9, queries that bring
    each head's scores to a few units; in one head a token with values 2^-6 of the
    others' takes more than 0.99 of the weight."""
    device()
    rng = np.random.default_rng(21)
    n, heads, group = 700, 3, 4
    K, V = rng.standard_normal((2, n, heads, D))
    size = 2.0 ** np.array([0, -12, 5])[:, None]
    K = (K * size).astype(np.float16)
    V[5, 0] *= 2.0 ** -6
    V = (V * 2.0 ** np.array([0, -10, 9])[:, None]).astype(np.float16)
    q = rng.standard_normal((heads, group, D)) * 4 / size[..., None]
    q[0, 0] = 1.5 * K[5, 0]
    q[0, 1] = 1.75 * K[5, 0]
    q = q.astype(np.float16).reshape(1, -1, D)
    host, cache = held(K, V)
    k, _ = host.cached(0, 0)
    for r in range(2):
        s = k @ q[0, r].astype(np.float64) * D ** -0.5
        assert np.exp(s[5] - s.max()) / np.exp(s - s.max()).sum() > 0.99
    note("paged attention sizes apart")
    for use_ws in (True, False):
        got = wq.kv_paged_attention(to_dev(q), cache, to_dev(host.lens), use_workspace=use_ws)
        assert head_errors(got, host.attend(q, [0])[0]).max() <= L2_REL


@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("window", [0, 200])
def test_any_headers(group, window):
    """Headers that the append does not write: zeros with fractions, scales of
    either sign.  A value is (c - z) s all the same."""
    device()
    rng = np.random.default_rng(7 * group + window)
    heads, blocks = 2, 5
    codes = rng.integers(0, 256, (blocks, heads, 16384)).astype(np.uint8)
    sign = lambda: rng.choice([-1.0, 1.0], (blocks, heads, 1, 128))  # noqa: E731
    head = np.concatenate([sign() * rng.uniform(0.1, 0.4, (blocks, heads, 1, 128)),
                           rng.uniform(4, 11, (blocks, heads, 1, 128)),
                           sign() * rng.uniform(0.01, 0.4, (blocks, heads, 1, 128)),
                           rng.uniform(4, 11, (blocks, heads, 1, 128))], 2).astype(np.float16)
    rec = np.concatenate([codes, head.reshape(blocks, heads, 512).view(np.uint8)], 2)
    assert rec.shape[2] == REC
    cache = wq.PagedKV(heads, blocks, 1, blocks)
    cache.pages.copy_(to_dev(rec))
    cache.table.copy_(to_dev(np.arange(blocks, dtype=np.int32)[None]))
    q = rng.standard_normal((1, heads * group, D)).astype(np.float16)
    ref = np.zeros((1, heads * group, D))
    for h in range(heads):
        K, V = [np.concatenate(x) for x in zip(*[okv.dequantize_block(dict(
            kcodes=rec[b, h, :8192].reshape(G, 64), vcodes=rec[b, h, 8192:16384].reshape(D, 64), ks=head[b, h, 0],
            kz=head[b, h, 1], vs=head[b, h, 2], vz=head[b, h, 3])) for b in range(blocks)])]
        first = max(0, len(K) - window) if window else 0
        for r in range(h * group, (h + 1) * group):
            ref[0, r] = okv.attend(q[0, r], K[first:], V[first:], D ** -0.5)
    lens = to_dev(np.array([blocks * G], np.int32))
    note(f"paged attention any headers group={group} window={window}")
    for use_ws in (True, False):
        got = wq.kv_paged_attention(to_dev(q), cache, lens, window=window, use_workspace=use_ws)
        assert head_errors(got, ref).max() <= L2_REL


@pytest.mark.parametrize("vsize", [2.0 ** -8, 1.0, 2.0 ** 8])
@pytest.mark.parametrize("group", GROUPS)
def test_far_scores(group, vsize):
    """Scores from 2^20 to 2^34 units of the exponent, of either sign: past 2^24
    neighbouring fp32 numbers are whole powers of two apart.  One token wins by
    far, in a block or in the window; its values come back.  (Its weight is rounded to
    2^-14 at worst: 2^-25 of what is left of 2^13 after two steps of 16, 2^-11.)"""
    device()
    rng = np.random.default_rng(group)
    heads, n = 2, 2 * G + 50
    u = rng.choice([-1.0, 1.0], (heads, D))
    V = (rng.standard_normal((n, heads, D)) * vsize).astype(np.float16)
    for best, least in ((77, 200), (2 * G + 33, 2 * G + 5), (200, 2 * G + 49)):
        level = rng.integers(1, 15, n).astype(np.float64)
        level[best], level[least] = 15.0, 0.0
        for half in range(18, 32):                        # the largest |K| and |q| are 2^(half / 2)
            size = min(2.0 ** (half / 2), 60000.0)
            K = ((level[:, None, None] / 15 - 0.5) * u * size).astype(np.float16)
            q = np.repeat(u, group, 0) * size
            q[group // 2:group] *= -1.0                   # these point at `least`
            q = q[None].astype(np.float16)
            host, cache = held(K, V)
            note(f"paged attention far scores group={group} {best} 2^{half / 2}")
            with np.errstate(over="ignore"):              # (attend's own bound is not used)
                ref, _ = host.attend(q, [0])
            bound = 2.0 ** -11 * np.abs(ref) + 2.0 ** -13 * np.abs(V).max() + 2.0 ** -25
            for use_ws in (True, False):
                got = wq.kv_paged_attention(to_dev(q), cache, to_dev(host.lens), use_workspace=use_ws)
                assert np.all(np.abs(got.cpu().numpy().astype(np.float64) - ref) <= bound), half
