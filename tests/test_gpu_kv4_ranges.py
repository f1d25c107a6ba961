"""Attention over the 4-bit cache where scores, or the scales of K and V, lie far apart: the softmax's
reference, its denominator and the weights' fp16 range, against 64 bits.
"""
import numpy as np
import pytest
import torch

import kv4_reference as R
import kv_cache_offload_nosa_b200 as nosa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def dev(a):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t.view(torch.int16) if t.dtype == torch.uint16 else t).cuda()


def bf16(x):
    return R.syn.round_bf16(np.ascontiguousarray(x)).reshape(x.shape)


def run(q, k, v, bs, split=0, call="decode_attn"):
    """Attention of q [G, d] over every block of one sequence of rows k, v [n, 1, d] (bf16 bits): the
    output [G, d] and the values that the cache holds for k and v."""
    n, _, d = k.shape
    G, nb = len(q), -(-n // bs)
    cache = nosa.NosaCache(nosa.make_config(1, G, 1, d, bs, 32, nb, 0, nb, attn_split=split, kv_bits=4))
    for name in ("k_pool", "v_pool"):
        cache.pool_view(name).fill_(0xFF)      # NaN scales past the context
    cache.write(dev(k), dev(v), dev(np.array([0, n], np.int32)))
    cache.init(dev(np.array([n], np.int32)))
    out, sel = torch.full((G, d), float("nan"), device="cuda"), dev(np.arange(nb, dtype=np.int32)[None])
    for _ in range(2):      # the second call meets the counters that the first one left
        cache.decode_attn(dev(q[None]), sel, out)
    assert cache.check() == (nosa.NOSA_OK, 0)
    return (out.cpu().numpy().astype(np.float64), R.dequantise(*R.quantise(k))[:, 0], R.dequantise(*R.quantise(v))[:, 0])


def check_row(got, q, K, V, scale):
    """One query row against 64 bits.

    An fp32 score is off by at most off_t = (d + 4) 2^-23 scale sum |q||k_t| (kv4_reference.attend_bound).
    Tokens that stay 100 below the largest score whatever these errors have no weight (e^-100 of at most
    2^12 tokens, times 2^80 between their values and the others', is below 2^-50). Where the others'
    scores are known to 2^-8, the ordinary bound over them holds; a token alone takes all the weight, and
    its two fp16 parts and the three divisions that follow are within 2^-20 of it; else any weighted mean
    of the rest is right, within the same 2^-20.
    """
    x, off = K @ q * scale, (K.shape[1] + 4) * 2.0**-23 * scale * (np.abs(K) @ np.abs(q))
    at = x + off > (x - off).max() - 100
    if off[at].max() < 2.0**-8:
        want = R.attend(q[None], K[at], V[at], scale)[0]
        tol = R.attend_bound(q[None], K[at], V[at], scale)[0]
        assert np.abs(got - want).max() <= tol, (float(np.abs(got - want).max()), float(tol))
    else:
        tol = 2.0**-20 * np.abs(V[at]).max()
        lo, hi = V[at].min(0), V[at].max(0)
        assert ((got >= lo - tol) & (got <= hi + tol)).all()
    return int(at.sum())


def check(got, q, K, V, heads=None):
    scale = float(np.float32(K.shape[1] ** -0.5))
    return [check_row(got[h], R.values(q[h]), K, V, scale) for h in (range(len(q)) if heads is None else heads)]


# ------------------------------------------------------------------ the denominator
@pytest.mark.parametrize("order", ["small first", "large first", "by turns"])
@pytest.mark.parametrize("split", [1, 3, 40])
@pytest.mark.parametrize("large", [1e13, 1e30])
def test_tokens_of_unlike_value_scales_all_count(order, split, large):
    """V of zeros beside V of 1e13 and 1e30, all scores alike or ordinary: the denominator counts both, in
    one warp's units, between the warps and between the CTAs' parts of a group."""
    rng = np.random.default_rng(91)
    n, bs, d = 1250, 32, 64
    k = bf16(rng.standard_normal((n, 1, d)))
    q = bf16(rng.standard_normal((4, d)) * np.array([[0.0], [1.0], [3.0], [0.1]]))
    block = np.arange(n) // bs
    is_large = {"small first": block >= 20, "large first": block < 20, "by turns": (block // 3) % 2 == 1}[order]
    v = bf16(rng.standard_normal((n, 1, d)) * np.where(is_large, large, 0.0)[:, None, None])
    got, K, V = run(q, k, v, bs, split)
    check(got, q, K, V)
