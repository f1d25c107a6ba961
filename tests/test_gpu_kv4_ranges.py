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


# ------------------------------------------------------------------ scores beyond any softmax
@pytest.mark.parametrize("vs", [1e6, 1e-6, 1e-12, 1e25, 1e-25])
@pytest.mark.parametrize("d,bs,G,split", [(128, 64, 4, 0), (64, 32, 8, 40), (64, 128, 1, 2)])
def test_scores_beyond_any_softmax_with_values_far_from_one(vs, d, bs, G, split):
    rng = np.random.default_rng(92)
    n = 700
    k, v = bf16(rng.standard_normal((n, 1, d)) * 1e4), bf16(rng.standard_normal((n, 1, d)) * vs)
    q = bf16(rng.standard_normal((G, d)) * 1e5)
    got, K, V = run(q, k, v, bs, split)
    assert np.abs(R.values(q) @ K.T).max() * d**-0.5 > 1e8
    check(got, q, K, V)


@pytest.mark.parametrize("vs", [1e6, 1e-6, 1e-12])
@pytest.mark.parametrize("what", [3e38, 1e8, "inf", "nan"])
@pytest.mark.parametrize("G,split", [(4, 0), (8, 40)])
def test_one_head_beyond_any_softmax_leaves_the_others_alone(vs, what, G, split):
    """One head of a group with scores of 10^8 and more, or that is not finite; the others are ordinary."""
    rng = np.random.default_rng(93)
    n, d = 700, 64
    k, v = bf16(rng.standard_normal((n, 1, d))), bf16(rng.standard_normal((n, 1, d)) * vs)
    q = bf16(rng.standard_normal((G, d)))
    if isinstance(what, str):
        q[2, 5] = {"inf": 0x7F80, "nan": 0x7FC0}[what]
    else:
        q[2] = bf16(rng.uniform(-1, 1, d) * what)
    got, K, V = run(q, k, v, 32, split)
    check(got, q, K, V, [h for h in range(G) if h != 2])
    if what == 1e8:
        check(got, q, K, V, [2])
    elif what == "nan":
        assert np.isnan(got[2]).all()


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("split", [4, 100])
@pytest.mark.parametrize("vs", [1.0, 1e-9, 1e9])
def test_scores_grow_beyond_any_softmax_on_the_way(sign, split, vs):
    """A sequence whose later keys score 10^8 for the first head (or minus that), with values of unlike
    scales: what was summed before, in registers and in shared memory, goes over to the new reference."""
    rng = np.random.default_rng(94)
    n, d, bs = 4900, 64, 64
    k = rng.standard_normal((n, 1, d))
    q = rng.standard_normal((4, d))
    q[0] = np.abs(q[0])
    late = rng.permutation(n - 3200)[:800] + 3200
    k[late] = sign * np.abs(k[late]) * rng.uniform(0.5, 1, (800, 1, 1)) * 1e8
    q[1:, :] -= (q[1:] @ np.ones(d))[:, None] / d
    v = rng.standard_normal((n, 1, d)) * vs * 10.0 ** rng.uniform(-5, 5, (n, 1, 1))
    q, k, v = bf16(q), bf16(k), bf16(v)
    got, K, V = run(q, k, v, bs, split)
    check(got, q, K, V)


# ------------------------------------------------------------------ keys at the ends of the range
@pytest.mark.parametrize("qs,ks", [(1e-36, 1e36), (1e-33, 1e37), (1e-30, 3e32), (1e-37, 1.0), (3e-39, 1e38), (1e33, 1e-33),
                                   (1e37, 1e-37)])
def test_keys_and_queries_at_the_ends_of_the_range(qs, ks):
    """Ordinary scores of very large and very small keys and queries."""
    rng = np.random.default_rng(95)
    n, d = 500, 128
    k, v = bf16(rng.uniform(-3, 3, (n, 1, d)) * ks), bf16(rng.standard_normal((n, 1, d)))
    q = bf16(rng.standard_normal((4, d)) * qs)
    got, K, V = run(q, k, v, 64)
    check(got, q, K, V)


@pytest.mark.parametrize("other", [1e-38, 1e-30, 1.0, "zero", "nan", "inf"])
def test_large_keys_with_unlike_heads(other):
    """Keys of 10^36 with ordinary scores for one head, beside a head that is far smaller, far larger
    (scores of 10^37, finite in fp32), zero or not finite."""
    rng = np.random.default_rng(96)
    n, d = 500, 64
    k, v = bf16(rng.standard_normal((n, 1, d)) * 1e36), bf16(rng.standard_normal((n, 1, d)))
    q = bf16(rng.standard_normal((2, d)) * 1e-36)
    if isinstance(other, str):
        q[1] = {"zero": 0, "inf": 0x7F80, "nan": 0x7FC0}[other]
    else:
        q[1] = bf16(rng.standard_normal(d) * other)
    got, K, V = run(q, k, v, 32)
    check(got, q, K, V, [0] if other in ("nan", "inf") else [0, 1])
    if other == "nan":
        assert np.isnan(got[1]).all()


@pytest.mark.parametrize("n", [6, 13, 20])
def test_groups_of_unlike_scales_within_a_row(n):
    """A group of 32 values 2^n times smaller than the others of its rows. The largest weight p s is at
    least 2^10 for the largest scale, and each of N weights is off by the ordinary bound and by half the
    last place of fp16, 2^-25: N 2^-35 of the row's largest value."""
    rng = np.random.default_rng(98)
    N, d = 300, 128
    k, q = bf16(rng.standard_normal((N, 1, d))), bf16(rng.standard_normal((4, d)))
    v = rng.standard_normal((N, 1, d))
    v[..., 32:64] *= 2.0**-n
    got, K, V = run(q, k, bf16(v), 64)
    scale = float(np.float32(d**-0.5))
    want = R.attend(R.values(q), K, V, scale)
    tol = R.attend_bound(R.values(q), K, V[:, 32:64], scale) + N * 2.0**-35 * np.abs(V).max()
    assert (np.abs(got - want)[:, 32:64].max(-1) <= tol).all()
    check(got, q, K, V)


# ------------------------------------------------------------------ without a workspace
@pytest.mark.parametrize("B,G,Hkv,d,bs,k", [(1, 4, 1, 128, 64, 300), (1, 8, 2, 64, 32, 500), (5, 4, 8, 128, 32, 70),
                                            (73, 1, 1, 64, 64, 40)])
def test_noalloc_attention_is_the_same_bit_for_bit(B, G, Hkv, d, bs, k):
    rng = np.random.default_rng(97)
    n = k * bs - 5
    cache = nosa.NosaCache(nosa.make_config(B, G * Hkv, Hkv, d, bs, 32, k, 0, k, kv_bits=4))
    gen = torch.Generator(device="cuda").manual_seed(97)
    k_, v_ = (torch.randn(B * n, Hkv, d, device="cuda", generator=gen).bfloat16() for _ in range(2))
    cache.write(k_, v_, torch.arange(B + 1, dtype=torch.int32, device="cuda") * n)
    cache.init(torch.full((B,), n, dtype=torch.int32, device="cuda"))
    q = dev(bf16(rng.standard_normal((B, G * Hkv, d))))
    sel = torch.arange(k, dtype=torch.int32, device="cuda").repeat(B * Hkv, 1)
    out, same = (torch.full((B, G * Hkv, d), float("nan"), device="cuda") for _ in range(2))
    for _ in range(2):
        cache.decode_attn(q, sel, out)
        nosa.decode_attn_noalloc(cache.cfg, cache.state, q, sel, same)
        assert torch.equal(out, same)
    assert cache.check() == (nosa.NOSA_OK, 0)
