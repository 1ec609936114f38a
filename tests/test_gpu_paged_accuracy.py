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
