"""The 4-bit cache on a B200: pages byte for byte against the format, attention against 64 bits, and
whole steps against the oracle.

Step parity uses prefills and tokens moved to values that the format holds exactly
(kv4_reference.snap), so that the oracle, which keeps bf16 pages, sees the same keys and values.
"""
import types

import numpy as np
import pytest
import torch

import kv4_reference as R
import kv_cache_offload_nosa_b200 as nosa
import nosa_synth as syn
import oracle as O

pytestmark = pytest.mark.gpu

CS = syn.configs()


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def dev(a):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t.view(torch.int16) if t.dtype == torch.uint16 else t).cuda()


def bf16_rows(rng, *shape):
    return R.syn.round_bf16(rng.standard_normal(shape)).reshape(shape)


def hard_rows(rng, n, Hkv, d):
    """Normal rows, and in some groups what can go wrong: zeros, ties, a lone outlier, subnormals, the
    largest finite values, an infinity, a NaN."""
    x = bf16_rows(rng, n, Hkv, d).reshape(-1, 32)
    for i in range(1, len(x), 4):     # halves of the scale: ties in every code
        s = 2.0 ** rng.integers(-20, 20)
        c = rng.integers(-13, 14, 32) / 2
        c[rng.integers(32)] = 7
        x[i] = R.syn.round_bf16(np.ascontiguousarray(c * s))
    for i, put in enumerate([0x0000, 0x8000, 0x0001, 0x7F7F, 0x7F80, 0x7FC1, 0x0380]):
        if len(x) > 2 * i:
            x[-1 - 2 * i][i % 3::3] = put
            if i < 3:
                x[-1 - 2 * i] = put
    return x.reshape(n, Hkv, d)


def make_cache(B, Hq, Hkv, d, bs, max_blocks, k, offload=False, slots=None, **kw):
    c = nosa.make_config(B, Hq, Hkv, d, bs, min(bs, 32), k, 0, max_blocks, slots=slots, kv_bits=4, **kw)
    return nosa.NosaCache(c, offload=offload)


def pools(cache):
    names = ("host_k", "host_v") if cache.offload else ("k_pool", "v_pool")
    return [cache.pool_view(n) for n in names]


def expected_pages(cache, k, v, cu, start, fill):
    """The pools after a write of k, v (numpy) into pages that held `fill` everywhere."""
    c = cache.cfg
    out = []
    for bits, keys in ((k, True), (v, False)):
        codes, scales = R.quantise(bits)
        page = np.full((c.B * c.Hkv, c.max_blocks, c.block_size * c.d * 9 // 16), fill, np.uint8)
        C, S = R.unpack(page, c.block_size, c.d, keys)
        C, S = (z.reshape(c.B * c.Hkv, -1, *z.shape[3:]) for z in (C, S))
        nan = np.zeros(C.shape[:3], bool)
        for b in range(c.B):
            n = cu[b + 1] - cu[b]
            for h in range(c.Hkv):
                at = slice(start[b], start[b] + n)
                C[b * c.Hkv + h, at] = codes[cu[b]:cu[b + 1], h]
                S[b * c.Hkv + h, at] = scales[cu[b]:cu[b + 1], h]
                nan[b * c.Hkv + h, at] = scales[cu[b]:cu[b + 1], h] == R.NAN_SCALE
        out.append((C, S, nan))
    return out


def held(cache, i, keys):
    c = cache.cfg
    C, S = R.unpack(pools(cache)[i].cpu().numpy(), c.block_size, c.d, keys)
    return tuple(z.reshape(c.B * c.Hkv, -1, *z.shape[3:]) for z in (C, S))


def check_pages(cache, want):
    for i, keys in enumerate((True, False)):
        C, S = held(cache, i, keys)
        Cw, Sw, nan = want[i]
        assert np.array_equal(S, Sw)
        assert np.array_equal(C[~nan], Cw[~nan])   # the codes of a group that is NaN say nothing


RUNS = [  # d, bs, Hq, Hkv, lengths, start
    (128, 64, 8, 2, [1], [0]), (64, 32, 1, 1, [1, 1, 1], [31, 32, 63]), (128, 128, 8, 8, [130, 0, 7], [0, 5, 121]),
    (64, 128, 4, 4, [37, 300], [0, 90]), (128, 32, 3, 3, [65, 1, 33, 0], [1, 0, 62, 9]), (64, 64, 5, 5, [129], [64]),
]


@pytest.mark.parametrize("d,bs,Hq,Hkv,lens,start", RUNS)
@pytest.mark.parametrize("layout", ["contiguous", "fused", "heads first"])
def test_write_and_read(d, bs, Hq, Hkv, lens, start, layout):
    rng = np.random.default_rng(d + bs + len(lens))
    B, n, pad = len(lens), sum(lens), 3
    cu = np.concatenate([[0], np.cumsum(lens)])
    nb = max(-(-(l + s) // bs) for l, s in zip(lens, start)) + 1
    cache = make_cache(B, Hq, Hkv, d, bs, nb, 1)
    # `pad` rows behind the last sequence, in a larger buffer that must stay as it is
    k, v = hard_rows(rng, n + pad, Hkv, d), hard_rows(rng, n + pad, Hkv, d)
    if layout == "contiguous":
        kt, vt = dev(k), dev(v)
    elif layout == "fused":
        both = torch.full((n + pad, 3 * Hkv + 1, d), 77, dtype=torch.int16, device="cuda")
        kt, vt = both[:, Hkv:2 * Hkv], both[:, 2 * Hkv:3 * Hkv]
    else:
        kt, vt = (torch.empty(Hkv, n + pad, d, dtype=torch.int16, device="cuda").transpose(0, 1) for _ in range(2))
    kt.copy_(dev(k))
    vt.copy_(dev(v))
    for p in pools(cache):
        p.fill_(0xA5)
    cut = dev(cu.astype(np.int32))
    st = dev(np.array(start, np.int32)) if any(start) else None
    cache.write(kt, vt, cut, st)
    want = expected_pages(cache, k[:n], v[:n], cu, start, 0xA5)
    check_pages(cache, want)
    assert cache.check() == (nosa.NOSA_OK, 0)
    # reading back: every value the format's, rounded once; rows of no sequence stay
    kt.fill_(1234)
    vt.fill_(1234)
    cache.read(kt, vt, cut, st)
    for got, bits in ((kt, k), (vt, v)):
        got = got.cpu().numpy().view(np.uint16)
        ref = R.round_to_bf16(R.dequantise(*R.quantise(bits[:n])))
        ref = np.where(np.isnan(R.values(ref)), 0x7FC0, ref)
        mine = np.where(np.isnan(R.values(got[:n])), 0x7FC0, got[:n])
        assert np.array_equal(np.where(mine == 0x8000, 0, mine), np.where(ref == 0x8000, 0, ref))
        assert (got[n:] == 1234).all()
    if layout == "fused":
        assert (both[:, :Hkv] == 77).all() and (both[:, 3 * Hkv:] == 77).all()


def test_write_in_chunks_equals_one_write():
    rng = np.random.default_rng(9)
    k, v = bf16_rows(rng, 301, 2, 128), bf16_rows(rng, 301, 2, 128)
    one, two = make_cache(1, 8, 2, 128, 64, 6, 1), make_cache(1, 8, 2, 128, 64, 6, 1)
    for c in (one, two):
        for p in pools(c):
            p.zero_()
    one.write(dev(k), dev(v), dev(np.array([0, 301], np.int32)))
    for a, b in ((0, 1), (1, 130), (130, 301)):
        two.write(dev(k[a:b]), dev(v[a:b]), dev(np.array([0, b - a], np.int32)), dev(np.array([a], np.int32)))
    for a, b in zip(pools(one), pools(two)):
        assert torch.equal(a, b)


def test_many_sequences():
    """More sequences than the kernels keep the bounds of at hand, some of them empty."""
    rng = np.random.default_rng(12)
    B = 300
    lens = rng.integers(0, 4, B)
    start = rng.integers(0, 29, B)
    cu = np.concatenate([[0], np.cumsum(lens)])
    k, v = bf16_rows(rng, cu[-1], 1, 64), bf16_rows(rng, cu[-1], 1, 64)
    cache = make_cache(B, 1, 1, 64, 32, 1, 1)
    for p in pools(cache):
        p.fill_(0xA5)
    cut, st = dev(cu.astype(np.int32)), dev(start.astype(np.int32))
    cache.write(dev(k), dev(v), cut, st)
    check_pages(cache, expected_pages(cache, k, v, cu, start, 0xA5))
    ko, vo = (torch.empty(int(cu[-1]), 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache.read(ko, vo, cut, st)
    for got, bits in ((ko, k), (vo, v)):
        ref = R.round_to_bf16(R.dequantise(*R.quantise(bits)))
        assert np.array_equal(R.values(got.view(torch.int16).cpu().numpy().view(np.uint16)), R.values(ref))


def test_rows_of_no_sequence_and_positions_outside_are_skipped():
    rng = np.random.default_rng(10)
    k, v = bf16_rows(rng, 40, 2, 64), bf16_rows(rng, 40, 2, 64)
    cache = make_cache(3, 4, 2, 64, 32, 2, 1)
    for p in pools(cache):
        p.fill_(0xA5)
    # tokens 0..3 and 30..39 belong to nobody; sequence 1 runs over the end (64), sequence 2 starts before 0
    cu, start = np.array([4, 10, 20, 30], np.int32), np.array([0, 60, -4], np.int32)
    cache.write(dev(k), dev(v), dev(cu), dev(start))
    rc, err = cache.check()
    assert rc == nosa.NOSA_EDEVICE and err == nosa.ERR_FULL
    C0, S0 = R.unpack(np.full((6, 2, 32 * 64 * 9 // 16), 0xA5, np.uint8), 32, 64, True)
    C0, S0 = C0.reshape(6, 64, 2, 32), S0.reshape(6, 64, 2)
    codes, scales = R.quantise(k)
    for h in range(2):
        C0[h, 0:6], S0[h, 0:6] = codes[4:10, h], scales[4:10, h]
        C0[2 + h, 60:64], S0[2 + h, 60:64] = codes[10:14, h], scales[10:14, h]
        C0[4 + h, 0:6], S0[4 + h, 0:6] = codes[24:30, h], scales[24:30, h]
    C, S = held(cache, 0, True)
    assert np.array_equal(C, C0) and np.array_equal(S, S0)
    ko, vo = (torch.full((40, 2, 64), 7, dtype=torch.int16, device="cuda") for _ in range(2))
    cache.read(ko, vo, dev(cu), dev(start))
    skip = [*range(4), *range(14, 24), *range(30, 40)]
    assert (ko[skip] == 7).all() and (vo[skip] == 7).all()
    assert (ko[[t for t in range(40) if t not in skip]] != 7).any()


@pytest.mark.parametrize("d,bs,offload", [(64, 32, False), (128, 64, True)])
def test_what_is_skipped_touches_neither_pool_and_the_rest_comes_back(d, bs, offload):
    """Tokens of no sequence and positions outside the cache, in K and in V: pages and rows read."""
    rng = np.random.default_rng(13)
    k, v = bf16_rows(rng, 40, 2, d), bf16_rows(rng, 40, 2, d)
    cache = make_cache(3, 4, 2, d, bs, 4, 1, offload=offload, slots=3 if offload else None)
    for p in pools(cache):
        p.fill_(0xA5)
    end = 4 * bs
    cu, start = np.array([4, 10, 20, 30], np.int32), np.array([0, end - 4, -4], np.int32)
    cache.write(dev(k), dev(v), dev(cu), dev(start))
    assert cache.check() == (nosa.NOSA_EDEVICE, nosa.ERR_FULL)
    want = []
    for bits, keys in ((k, True), (v, False)):
        C, S = R.unpack(np.full((6, 4, bs * d * 9 // 16), 0xA5, np.uint8), bs, d, keys)
        C, S = C.reshape(6, end, d // 32, 32), S.reshape(6, end, d // 32)
        codes, scales = R.quantise(bits)
        for h in range(2):
            C[h, 0:6], S[h, 0:6] = codes[4:10, h], scales[4:10, h]
            C[2 + h, end - 4:], S[2 + h, end - 4:] = codes[10:14, h], scales[10:14, h]
            C[4 + h, 0:6], S[4 + h, 0:6] = codes[24:30, h], scales[24:30, h]
        want.append((C, S, np.zeros(C.shape[:3], bool)))
    check_pages(cache, want)
    ko, vo = (torch.full((40, 2, d), 7, dtype=torch.int16, device="cuda") for _ in range(2))
    cache.read(ko, vo, dev(cu), dev(start))
    held_ = [*range(4, 14), *range(24, 30)]
    for got, bits in ((ko, k), (vo, v)):
        got = got.cpu().numpy().view(np.uint16)
        ref = np.full_like(got, 7)
        ref[held_] = R.round_to_bf16(R.dequantise(*R.quantise(bits)))[held_]
        assert np.array_equal(np.where(got == 0x8000, 0, got), np.where(ref == 0x8000, 0, ref))


def test_write_to_host_pools():
    rng = np.random.default_rng(11)
    k, v = hard_rows(rng, 400, 2, 128), hard_rows(rng, 400, 2, 128)
    cache = make_cache(2, 8, 2, 128, 64, 6, 2, offload=True, slots=4)
    for p in pools(cache):
        p.fill_(0xA5)
    cu, start = np.array([0, 99, 400]), [0, 10]
    cache.write(dev(k), dev(v), dev(cu.astype(np.int32)), dev(np.array(start, np.int32)))
    torch.cuda.synchronize()
    check_pages(cache, expected_pages(cache, k, v, cu, start, 0xA5))
    ko, vo = torch.empty(400, 2, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(400, 2, 128, dtype=torch.bfloat16, device="cuda")
    cache.read(ko, vo, dev(cu.astype(np.int32)), dev(np.array(start, np.int32)))
    ref = R.round_to_bf16(R.dequantise(*R.quantise(k)))
    ok = ~np.isnan(R.values(ref))
    got = ko.view(torch.int16).cpu().numpy().view(np.uint16)
    assert np.array_equal(R.values(got)[ok], R.values(ref)[ok]) and np.isnan(R.values(got)[~ok]).all()


@pytest.mark.parametrize("d,bs,s,kc16", [(128, 64, 16, 0), (64, 32, 8, 0), (128, 128, 32, 1), (64, 64, 16, 1)])
def test_append(d, bs, s, kc16):
    """Tokens appended one by one: the pages are those of one write, and each sub-block's mean is the
    fp32 mean, in token order, of the values held."""
    rng = np.random.default_rng(d + bs + s)
    n0, n1, Hkv = bs - 3, 2 * s + 5, 2
    k, v = hard_rows(rng, n0 + n1, Hkv, d), hard_rows(rng, n0 + n1, Hkv, d)
    k[(k & 0x7F80) == 0x7F80] = 0x3F80      # means of finite values
    c = nosa.make_config(1, 4, Hkv, d, bs, s, 1, 0, 4, kc_bf16=kc16, kv_bits=4)
    cache = nosa.NosaCache(c)
    for p in pools(cache):
        p.fill_(0xA5)
    cache.write(dev(k[:n0]), dev(v[:n0]), dev(np.array([0, n0], np.int32)))
    cache.init(dev(np.array([n0], np.int32)))
    for t in range(n0, n0 + n1):
        cache.append(dev(k[t]), dev(v[t]))
    assert cache.check() == (nosa.NOSA_OK, 0)
    check_pages(cache, expected_pages(cache, k, v, [0, n0 + n1], [0], 0xA5))
    assert (cache.t["seq_len"] == n0 + n1).all()
    val = R.dequantise(*R.quantise(k)).astype(np.float32)
    kc = cache.t["kc"].view(torch.int32).cpu().numpy().view(np.uint16 if kc16 else np.float32).reshape(Hkv, -1, d)
    with np.errstate(over="ignore"):
        for i in range(-(-(n0 + n1) // s)):
            x = val[i * s:min((i + 1) * s, n0 + n1)]
            mean = np.cumsum(x, 0, dtype=np.float32)[-1] / np.float32(len(x))
            want = R.round_to_bf16(mean.astype(np.float64)) if kc16 else mean
            assert np.array_equal(kc[:, i], want), i


def fill(cache, rng, lens, kscale=1.0, vscale=1.0):
    """Random prefill of the given lengths: the values held, K and V [B*Hkv][tokens, d]."""
    c = cache.cfg
    n = sum(lens)
    k = R.syn.round_bf16(rng.standard_normal((n, c.Hkv, c.d)) * kscale).reshape(n, c.Hkv, c.d)
    v = R.syn.round_bf16(rng.standard_normal((n, c.Hkv, c.d)) * vscale).reshape(n, c.Hkv, c.d)
    cu = np.concatenate([[0], np.cumsum(lens)])
    if not cache.offload:
        for p in pools(cache):   # rows past the context may hold anything, NaN scales among it
            p.fill_(0xFF)
    if n:
        cache.write(dev(k), dev(v), dev(cu.astype(np.int32)))
    res = None
    if cache.offload:
        res = torch.zeros(c.B * c.Hkv, c.max_blocks, dtype=torch.uint8, device="cuda")
        res[:, :c.slots] = 1
    cache.init(dev(np.array(lens, np.int32)), res)
    cache._res = res
    K, V = R.dequantise(*R.quantise(k)), R.dequantise(*R.quantise(v))
    return ([K[cu[b]:cu[b + 1], h] for b in range(c.B) for h in range(c.Hkv)],
            [V[cu[b]:cu[b + 1], h] for b in range(c.B) for h in range(c.Hkv)])


def check_attention(cache, q, sel, out, K, V):
    c = cache.cfg
    G = c.Hq // c.Hkv
    got = out.cpu().numpy().reshape(c.B * c.Hkv, G, c.d)
    qv = R.values(q).reshape(c.B * c.Hkv, G, c.d)
    scale = float(np.float32(c.scale))
    for gi in range(c.B * c.Hkv):
        at = [t for j in sel[gi] if j >= 0 for t in range(j * c.block_size, min((j + 1) * c.block_size, len(K[gi])))]
        want = R.attend(qv[gi], K[gi][at], V[gi][at], scale)
        tol = R.attend_bound(qv[gi], K[gi][at], V[gi][at], scale)[:, None]
        err = np.abs(got[gi] - want)
        assert (err <= tol).all(), (gi, len(at), float((err / np.maximum(tol, 1e-300)).max()))


def draw_sel(rng, cache, lens, short=False):
    c = cache.cfg
    k = c.k_q + c.k_e
    sel = np.full((c.B * c.Hkv, k), -1, np.int32)
    for gi in range(c.B * c.Hkv):
        n = -(-lens[gi // c.Hkv] // c.block_size)
        m = min(k, n) if not short else min(k, n, int(rng.integers(0, k + 1)))
        sel[gi, :m] = np.sort(rng.choice(n, m, replace=False))
    return sel


ATTEND = [  # d, bs, G, Hkv, lengths, k
    (128, 64, 4, 2, [1], 1), (64, 64, 4, 2, [63, 64, 65], 2), (128, 64, 4, 8, [4097, 700], 64),
    (128, 32, 1, 3, [1000, 31, 0], 17), (128, 128, 8, 2, [3000, 129], 9), (64, 128, 8, 1, [2050], 17),
    (64, 32, 2, 5, [513, 96], 11), (128, 64, 2, 1, [9000], 141), (64, 32, 1, 1, [5], 1), (64, 64, 8, 2, [16, 17], 1),
]


@pytest.mark.parametrize("d,bs,G,Hkv,lens,k", ATTEND)
@pytest.mark.parametrize("split", [0, 3, 150])
def test_attention(d, bs, G, Hkv, lens, k, split):
    rng = np.random.default_rng(1000 + d + bs + G + k)
    nb = max(-(-max(lens) // bs), k)
    cache = make_cache(len(lens), G * Hkv, Hkv, d, bs, nb, k, attn_split=split)
    K, V = fill(cache, rng, lens)
    for short in (False, True):
        q = bf16_rows(rng, len(lens) * Hkv, G, d)
        sel = draw_sel(rng, cache, lens, short)
        out = torch.full((len(lens) * Hkv * G * d,), float("nan"), device="cuda")
        for _ in range(2):    # the merge's counters are back at zero after a call
            cache.decode_attn(dev(q), dev(sel), out)
            check_attention(cache, q, sel, out, K, V)
    assert cache.check() == (nosa.NOSA_OK, 0)


@pytest.mark.parametrize("qs,ks,vs", [(30.0, 1.0, 1.0), (1e-6, 1.0, 1e-6), (1e4, 1e-4, 1e6), (1.0, 3e4, 1e-12), (1e-20, 1e20, 1e18),
                                      (1e36, 1e-36, 1.0), (1e-25, 1e25, 1.0)])
def test_attention_over_wide_ranges(qs, ks, vs):
    """Queries, keys and values far from 1: weights sharp or flat, values large and small."""
    rng = np.random.default_rng(77)
    cache = make_cache(1, 8, 2, 128, 64, 20, 20)
    K, V = fill(cache, rng, [1250], ks, vs)
    q = R.syn.round_bf16(rng.standard_normal((2, 4, 128)) * qs).reshape(2, 4, 128)
    sel = draw_sel(rng, cache, [1250])
    out = torch.empty(8 * 128, device="cuda")
    cache.decode_attn(dev(q), dev(sel), out)
    check_attention(cache, q, sel, out, K, V)


@pytest.mark.parametrize("sign", [1, -1])
def test_scores_beyond_any_softmax(sign):
    """Scores of 10^8 and more: the largest takes all the weight (here it leads by far more than an fp32
    score can be off by), whatever came before it, and large negative ones alone are no different."""
    rng = np.random.default_rng(83)
    cache = make_cache(1, 4, 1, 128, 64, 6, 6)
    n = 380
    k = R.syn.round_bf16(rng.standard_normal((n, 1, 128)) * 1e4).reshape(n, 1, 128)
    v = bf16_rows(rng, n, 1, 128)
    q = R.syn.round_bf16(rng.standard_normal((1, 4, 128)) * 1e5).reshape(1, 4, 128)
    if sign < 0:      # every score negative: keys against the mean query
        q = np.repeat(q[:, :1], 4, 1)
        k = R.syn.round_bf16(-R.values(q[0, 0]) * rng.uniform(0.1, 0.3, (n, 1, 1))).reshape(n, 1, 128)
    cache.write(dev(k), dev(v), dev(np.array([0, n], np.int32)))
    cache.init(dev(np.array([n], np.int32)))
    K, V = R.dequantise(*R.quantise(k))[:, 0], R.dequantise(*R.quantise(v))[:, 0]
    out = torch.empty(4, 128, device="cuda")
    cache.decode_attn(dev(q), dev(np.arange(6, dtype=np.int32)[None]), out)
    x = R.values(q)[0] @ K.T * 128**-0.5
    off = 132 * 2.0**-23 * 128**-0.5 * (np.abs(R.values(q)[0]) @ np.abs(K).T).max()
    got = out.cpu().numpy()
    assert np.abs(x).max() > 1e6 and np.isfinite(got).all()
    for h in range(4):
        top = np.argsort(x[h])[::-1]
        lead = x[h][top[0]] - x[h][top[1]]
        if lead > 2 * off + 100:
            # one weight of 1: its hi + lo parts and the two divisions, 2^-21 each at most
            assert np.abs(got[h] - V[top[0]]).max() <= 2.0**-20 * np.abs(V[top[0]]).max()
        else:
            close = x[h] > x[h][top[0]] - 2 * off - 100     # a mean of these rows
            lo, hi = V[close].min(0), V[close].max(0)
            assert ((got[h] >= lo - 1e-5) & (got[h] <= hi + 1e-5)).all()


@pytest.mark.parametrize("vs", [1e30, 1e36, 1e-27, 1e-34])
def test_values_at_the_ends_of_the_range(vs):
    rng = np.random.default_rng(84)
    cache = make_cache(1, 8, 1, 64, 32, 5, 5)
    K, V = fill(cache, rng, [150], 1.0, vs)
    q = bf16_rows(rng, 1, 8, 64)
    out = torch.empty(8, 64, device="cuda")
    cache.decode_attn(dev(q), dev(np.arange(5, dtype=np.int32)[None]), out)
    want = R.attend(R.values(q)[0], K[0], V[0], float(np.float32(cache.cfg.scale)))
    # V of 1e-34 has scales of about 2^-115, so the weights are about 2^(100 - 115) and their two fp16
    # parts hold 2^-25: 2^-10 of them. V of 1e36 (2^119, scales 2^117) drops weights below
    # 2^(-126 + 107) of the largest: 150 of 2^-19. Otherwise the ordinary bound, 1e-5 here.
    tol = 2.0**-9 if vs == 1e-34 else 150 * 2.0**-18 if vs == 1e36 else 1e-5
    assert np.abs(out.cpu().numpy() - want).max() <= tol * np.abs(want).max()


def test_attention_with_unlike_scales_in_a_sequence():
    """Tokens and groups whose values differ by many orders, the largest weight on a small value."""
    rng = np.random.default_rng(78)
    cache = make_cache(1, 4, 1, 64, 32, 8, 8)
    n = 250
    k = bf16_rows(rng, n, 1, 64)
    v = R.syn.round_bf16(rng.standard_normal((n, 1, 64)) * 10.0 ** rng.uniform(-6, 6, (n, 1, 1))).reshape(n, 1, 64)
    v[::7, :, 32:] = 0
    v[3::11] = 0
    for p in pools(cache):
        p.fill_(0xFF)
    cache.write(dev(k), dev(v), dev(np.array([0, n], np.int32)))
    cache.init(dev(np.array([n], np.int32)))
    K, V = R.dequantise(*R.quantise(k))[:, 0], R.dequantise(*R.quantise(v))[:, 0]
    q = R.syn.round_bf16(10 * K[np.argsort(np.abs(V).max(-1))[40:44]]).reshape(1, 4, 64)
    sel = np.arange(8, dtype=np.int32)[None]
    out = torch.empty(4 * 64, device="cuda")
    cache.decode_attn(dev(q), dev(sel), out)
    check_attention(cache, q, sel, out, [K], [V])


def test_nan_in_an_attended_row_is_not_hidden():
    rng = np.random.default_rng(79)
    cache = make_cache(2, 4, 1, 64, 32, 4, 4)
    k, v = bf16_rows(rng, 200, 1, 64), bf16_rows(rng, 200, 1, 64)
    v[150, 0, 3] = 0x7FC0      # sequence 1
    cache.write(dev(k), dev(v), dev(np.array([0, 100, 200], np.int32)))
    cache.init(dev(np.array([100, 100], np.int32)))
    out = torch.zeros(2, 4, 64, device="cuda")
    sel = np.tile(np.arange(4, dtype=np.int32), (2, 1))
    cache.decode_attn(dev(bf16_rows(rng, 2, 4, 64)), dev(sel), out)
    assert torch.isfinite(out[0]).all() and torch.isnan(out[1, :, :32]).all()


def test_bad_selection_is_skipped_and_recorded():
    rng = np.random.default_rng(80)
    cache = make_cache(2, 8, 2, 128, 64, 8, 4)
    lens = [500, 300]
    K, V = fill(cache, rng, lens)
    q, sel = bf16_rows(rng, 4, 4, 128), draw_sel(rng, cache, lens)
    bad = sel.copy()
    bad[3, 0] = 5 + 2        # sequence 1 has 5 blocks
    out = torch.empty(2 * 8 * 128, device="cuda")
    cache.decode_attn(dev(q), dev(bad), out)
    rc, err = cache.check()
    assert rc == nosa.NOSA_EDEVICE and err == nosa.ERR_SEL
    bad[3, 0] = -1
    check_attention(cache, q, bad, out, K, V)


def test_noalloc_attention():
    rng = np.random.default_rng(81)
    cache = make_cache(3, 16, 4, 128, 64, 40, 33)
    lens = [2500, 64, 1]
    K, V = fill(cache, rng, lens)
    q, sel = bf16_rows(rng, 12, 4, 128), draw_sel(rng, cache, lens)
    for _ in range(2):
        out = torch.full((3 * 16 * 128,), float("nan"), device="cuda")
        nosa.decode_attn_noalloc(cache.cfg, cache.state, dev(q), dev(sel), out)
        check_attention(cache, q, sel, out, K, V)


def test_attention_on_a_side_stream_and_in_a_graph():
    """The run of write, append and attention captured once and replayed on new inputs, on a stream of
    its own, beside another cache's calls on the default stream."""
    rng = np.random.default_rng(82)
    lens, nb, k = [130, 61], 6, 4
    cache, other = (make_cache(2, 8, 2, 64, 32, nb, k) for _ in range(2))
    K, V = fill(cache, rng, lens)
    Ko, Vo = fill(other, rng, lens)
    kn, vn = (torch.empty(4, 64, dtype=torch.int16, device="cuda") for _ in range(2))
    q = torch.empty(4, 4, 64, dtype=torch.int16, device="cuda")
    sel = torch.empty(4, k, dtype=torch.int32, device="cuda")
    out, out2 = (torch.empty(2 * 8 * 64, device="cuda") for _ in range(2))
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side, capture_error_mode="relaxed"):
        cache.append(kn, vn)
        cache.decode_attn(q, sel, out)
    for step in range(5):
        a, b = bf16_rows(rng, 4, 64), bf16_rows(rng, 4, 64)
        qq = bf16_rows(rng, 4, 4, 64)
        lens = [n + 1 for n in lens]
        ss = draw_sel(rng, cache, lens)
        kn.copy_(dev(a)), vn.copy_(dev(b)), q.copy_(dev(qq)), sel.copy_(dev(ss))
        so = draw_sel(rng, other, [130, 61])
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            g.replay()
        other.decode_attn(dev(qq), dev(so), out2)
        torch.cuda.synchronize()
        for gi in range(4):
            K[gi] = np.vstack([K[gi], R.dequantise(*R.quantise(a[gi:gi + 1]))])
            V[gi] = np.vstack([V[gi], R.dequantise(*R.quantise(b[gi:gi + 1]))])
        check_attention(cache, qq, ss, out, K, V)
        check_attention(other, qq, so, out2, Ko, Vo)


# ------------------------------------------------------------------ whole steps
def snapped_case(monkeypatch, name, steps=None, lookahead=False):
    make = syn.make_inputs

    def snapped(cfg, **kw):
        inp = make(cfg, **kw)
        inp.pool_k, inp.pool_v = R.snap(inp.pool_k), R.snap(inp.pool_v)
        inp.k_new, inp.v_new = R.snap(inp.k_new), R.snap(inp.v_new)
        return inp

    monkeypatch.setattr(syn, "make_inputs", snapped)
    return O.run_case(CS[name], steps=steps, lookahead=lookahead)


def setup4(cfg, inputs, **kw):
    """gpu_harness.setup with a 4-bit cache: the prefill goes through the cache's own write."""
    import gpu_harness as H
    c = H.c_config(cfg, kw.pop("attn_split", 0))
    c.kv_bits = 4
    cache = nosa.NosaCache(c, offload=cfg.offload)
    cu = np.concatenate([[0], np.cumsum(cfg.T)]).astype(np.int32)
    rows = [torch.cat([torch.from_numpy(p[b, :, :cfg.T[b]].view(np.int16)).transpose(0, 1) for b in range(cfg.B)]).cuda()
            for p in (inputs.pool_k, inputs.pool_v)]
    for p in pools(cache):
        p.fill_(0xFF)
    if cu[-1]:
        cache.write(rows[0], rows[1], dev(cu))
    cache._res = H.dev(inputs.resident.reshape(cfg.B * cfg.Hkv, cfg.max_blocks)) if cfg.offload else None
    cache._plen = dev(np.array(cfg.T, np.int32))
    cache.init(cache._plen, cache._res)
    return cache


STEPS = ["tiny", "tiny_dense", "tiny_forecast", "llama_small", "offload_small", "sink_small", "ragged", "ragged_offload",
         "empty", "bs128_d64", "g8", "short_kq0", "short_kq0_offload", "ragged_softmax", "tiny_window", "ragged_kc16",
         "g8_kc16"]


@pytest.mark.parametrize("name", STEPS)
@pytest.mark.parametrize("mode", ["fused", "staged", "events"])
def test_step_parity(name, mode, monkeypatch):
    import gpu_harness as H
    if mode != "fused" and CS[name].score_mode:
        pytest.skip("scoring variants run in the whole step")
    case = snapped_case(monkeypatch, name, steps=min(CS[name].steps, 40))
    cfg = case.cfg
    cache = setup4(cfg, case.inputs)
    io = H.StepIO(cfg)
    for t, rec in enumerate(case.steps):
        H.run_step(cache, cfg, case.inputs, rec, t, io, mode)
        H.compare_step(cache, cfg, rec, io, t)


@pytest.mark.parametrize("split", [1, 5])
def test_step_parity_with_a_given_split(split, monkeypatch):
    import gpu_harness as H
    case = snapped_case(monkeypatch, "llama_small", steps=3)
    cache = setup4(case.cfg, case.inputs, attn_split=split)
    io = H.StepIO(case.cfg)
    for t, rec in enumerate(case.steps):
        H.run_step(cache, case.cfg, case.inputs, rec, t, io)
        H.compare_step(cache, case.cfg, rec, io, t)


@pytest.mark.parametrize("name", ["lookahead_small", "lookahead_hbm", "lookahead_ragged", "lookahead_tiny"])
def test_lookahead_parity(name, monkeypatch):
    import gpu_harness as H
    case = snapped_case(monkeypatch, name, lookahead=True)
    cache = setup4(case.cfg, case.inputs)
    io = H.StepIO(case.cfg)
    for t, rec in enumerate(case.steps):
        H.run_step(cache, case.cfg, case.inputs, rec, t, io, "lookahead")
        H.compare_step(cache, case.cfg, rec, io, t)


@pytest.mark.parametrize("name", ["tiny", "offload_small"])
def test_step_in_a_graph(name, monkeypatch):
    import gpu_harness as H
    from kv_cache_offload_nosa_b200.graph import StepGraph
    case = snapped_case(monkeypatch, name)
    cfg = case.cfg
    cache = setup4(cfg, case.inputs)
    io0 = H.StepIO(cfg)
    H.run_step(cache, cfg, case.inputs, case.steps[0], 0, io0)
    H.compare_step(cache, cfg, case.steps[0], io0, 0)
    g = StepGraph(cache)
    io = types.SimpleNamespace(sel=g.sel, out=g.out, miss=g.miss[:cfg.B * cfg.Hkv])
    for t, rec in enumerate(case.steps):
        if t:
            g.run(H.dev(rec.q), H.dev(case.inputs.k_new[t]), H.dev(case.inputs.v_new[t]), H.dev(case.inputs.evict[t]))
            torch.cuda.synchronize()
            H.compare_step(cache, cfg, rec, io, t)


def test_flag_that_never_arrives_times_out(monkeypatch):
    """nosa_attend without its plan, every selected entry -1: each wait gives up after 20 ms, the error
    is recorded, and the library runs the workload again on a rebuilt state."""
    import gpu_harness as H
    case = snapped_case(monkeypatch, "offload_small", steps=2)
    cfg = case.cfg
    cache = setup4(cfg, case.inputs)
    cache.cfg.wait_us = 20000
    NG = cfg.B * cfg.Hkv
    sel = torch.full((NG * cfg.k,), -1, dtype=torch.int32, device="cuda")
    out = torch.empty(cfg.B * cfg.Hq * cfg.d, device="cuda")
    kn, vn = H.dev(case.inputs.k_new[0]), H.dev(case.inputs.v_new[0])
    cache.attend(H.dev(case.steps[0].q), kn, vn, sel, out)
    rc, err = cache.check()
    assert rc == nosa.NOSA_ETIMEOUT and err & nosa.ERR_TIMEOUT
    cache = setup4(cfg, case.inputs)
    io = H.StepIO(cfg)
    for t, rec in enumerate(case.steps):
        H.run_step(cache, cfg, case.inputs, rec, t, io)
        H.compare_step(cache, cfg, rec, io, t)
