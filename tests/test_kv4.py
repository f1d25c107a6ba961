"""The 4-bit cache on the host: the reference's own consistency, configuration and argument checks.

Nothing is launched: every refusal comes before the first CUDA call that needs a device.
"""
import ctypes

import numpy as np
import pytest
import torch

import kv4_reference as R
import kv_cache_offload_nosa_b200 as nosa
from kv_cache_offload_nosa_b200 import build as nb
from kv_cache_offload_nosa_b200.cache import NosaCache, check_run


@pytest.fixture(scope="module")
def lib():
    nb.build()
    return nosa.load()


def cfg(**kw):
    base = dict(B=2, Hq=8, Hkv=2, d=128, block_size=64, sub_block=16, k_q=4, k_e=4, max_blocks=40, kv_bits=4)
    base.update(kw)
    return nosa.make_config(**base)


def state():
    """A state of addresses that are never read (16-byte aligned, no host pools)."""
    fake = [0x10000 * (i + 1) for i in range(12)]
    return nosa.nosa_state(*fake[:9], None, None, fake[9])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("keys", [True, False])
def test_reference_pages_hold_their_rows(d, keys):
    rng = np.random.default_rng(5)
    bits = R.syn.round_bf16(rng.standard_normal((3, 32, d))).reshape(3, 32, d)
    codes, scales = R.quantise(bits)
    page = R.pack(codes, scales, keys)
    assert page.shape == (3, 32 * d * 9 // 16)
    c2, s2 = R.unpack(page, 32, d, keys)
    assert np.array_equal(codes, c2) and np.array_equal(scales, s2)
    # every value within half a step of the scale, the largest within what rounding the scale
    # (half a step of bf16, 2^-8 of it) moves it: 7 * 2^-8 of a step
    err = np.abs(R.dequantise(codes, scales) - R.values(bits)).reshape(3, 32, -1, 32)
    assert (err <= R.values(scales)[..., None] * (0.5 + 7 * 2.0**-8)).all()


def test_reference_ties_go_away_from_zero():
    x = np.zeros((1, 64))
    x[0, :6] = [7, 2.5, -2.5, 0.5, -0.5, 6.5]
    x[0, 32:34] = [-14, 5]
    codes, scales = R.quantise(R.syn.round_bf16(x).reshape(1, 64))
    assert R.values(scales).tolist() == [[1.0, 2.0]]
    assert (codes[0, 0, :6].astype(int) - 8).tolist() == [7, 3, -3, 1, -1, 7]
    assert (codes[0, 1, :2].astype(int) - 8).tolist() == [-7, 3]


def test_snapped_rows_are_held_exactly():
    rng = np.random.default_rng(6)
    bits = R.snap(R.syn.round_bf16(rng.standard_normal((40, 128)) * 3).reshape(40, 128))
    assert np.array_equal(R.dequantise(*R.quantise(bits)), R.values(bits))


@pytest.mark.parametrize("bad", [dict(kv_bits=1), dict(kv_bits=8), dict(kv_bits=-4), dict(stop_tau=0.1)])
def test_bad_config_is_rejected(lib, bad):
    c, n = cfg(**bad), ctypes.c_size_t()
    assert lib.nosa_workspace_size(ctypes.byref(c), ctypes.byref(n)) == nosa.NOSA_EINVAL


def test_pools_take_nine_sixteenths_of_a_byte_per_value(lib):
    s4, s16 = nosa.state_sizes(cfg()), nosa.state_sizes(cfg(kv_bits=0))
    for name in ("k_pool", "v_pool", "host_k", "host_v"):
        assert getattr(s4, name) * 32 == getattr(s16, name) * 9
    assert s4.kc == s16.kc
    assert nosa.state_sizes(cfg(kv_bits=16)).k_pool == s16.k_pool
    # a page keeps the pools' 16-byte alignment at every block size and head dim
    for d in (64, 128):
        for bs in (32, 64, 128):
            assert (bs * d * 9 // 16) % 16 == 0


GOOD = dict(k=0x100000, v=0x200000, strides=None, n=5, cu=0x300000, start=0x400000)


@pytest.mark.parametrize("write", [True, False])
@pytest.mark.parametrize("bad", [
    dict(k=None), dict(v=None), dict(cu=None), dict(k=0x100002), dict(v=0x200008), dict(cu=0x300004),
    dict(start=0x400004), dict(n=-1), dict(n=2**30), dict(n=2**29),
    dict(strides=(256, 128, 256, 124)), dict(strides=(-256, 128, 256, 128)),
])
def test_runs_are_refused_on_host(lib, write, bad):
    kw = dict(GOOD, **bad)
    c, st = cfg(), state()
    ns = nosa.nosa_kv_strides(*kw["strides"]) if kw["strides"] else None
    f = lib.nosa_write_kv if write else lib.nosa_read_kv
    rc = f(ctypes.byref(c), ctypes.byref(st), kw["k"], kw["v"], ctypes.byref(ns) if ns else None, kw["n"],
           kw["cu"], kw["start"], None)
    assert rc == nosa.NOSA_EINVAL and lib.nosa_last_error()


@pytest.mark.parametrize("strides", [(256, 64, 256, 128), (128, 128, 256, 128), (256, 128, 0, 128), (256, 128, 256, 0)])
def test_reading_into_rows_that_overlap_is_refused(lib, strides):
    c, st, ns = cfg(), state(), nosa.nosa_kv_strides(*strides)
    args = (ctypes.byref(ns), 5, 0x300000, None, None)
    assert lib.nosa_read_kv(ctypes.byref(c), ctypes.byref(st), 0x100000, 0x200000, *args) == nosa.NOSA_EINVAL
    assert lib.nosa_read_kv(ctypes.byref(c), ctypes.byref(st), 0x100000, 0x100000, None, *args[1:]) == nosa.NOSA_EINVAL


def test_an_empty_run_launches_nothing(lib):
    c, st = cfg(), state()
    for f in (lib.nosa_write_kv, lib.nosa_read_kv):
        assert f(ctypes.byref(c), ctypes.byref(st), 0x100000, 0x200000, None, 0, 0x300000, None, None) == nosa.NOSA_OK
        assert f(ctypes.byref(c), ctypes.byref(st), None, None, None, 0, None, None, None) == nosa.NOSA_OK


@pytest.mark.parametrize("bits", [0, 16])
def test_runs_need_a_4_bit_cache(lib, bits):
    c, st = cfg(kv_bits=bits), state()
    assert lib.nosa_write_kv(ctypes.byref(c), ctypes.byref(st), 0x100000, 0x200000, None, 5, 0x300000, None,
                             None) == nosa.NOSA_EINVAL
    assert b"kv_bits" in lib.nosa_last_error()


class _OnCuda(torch.Tensor):
    """A CPU tensor that says it is on cuda:0 (checks only)."""
    is_cuda = True
    device = torch.device("cuda", 0)

    def get_device(self):
        return 0


def on_cuda(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(_OnCuda)


def test_cache_checks_the_rows_it_is_given():
    c, dev, rows = cfg(), torch.device("cuda", 0), on_cuda
    cu, start = on_cuda(3, dtype=torch.int32), on_cuda(2, dtype=torch.int32)
    assert check_run(c, rows(5, 2, 128), rows(5, 2, 128), cu, start, dev) is None
    assert check_run(c, rows(0, 2, 128), rows(0, 2, 128), cu, None, dev) is None
    qkv = rows(5, 12, 128)
    s = check_run(c, qkv[:, 8:10], qkv[:, 10:12], cu, start, dev)
    assert (s.k_tok, s.k_head, s.v_tok, s.v_head) == (1536, 128, 1536, 128)
    assert check_run(c, qkv[:1, 8:10], rows(2, 1, 128).transpose(0, 1), cu, start, dev) is None
    s = check_run(c, qkv[:1, 8:10], rows(1, 4, 128)[:, ::2], cu, start, dev)
    assert (s.k_tok, s.k_head, s.v_tok, s.v_head) == (256, 128, 256, 256)
    good = rows(5, 2, 128)
    for k, v in [(rows(5, 2, 64), good), (good, rows(4, 2, 128)), (rows(5, 2, 128, dtype=torch.float16), good),
                 (good, rows(5, 2, 128, dtype=torch.float32)), (rows(10, 128), rows(10, 128)),
                 (rows(5, 2, 256)[..., ::2], good), (torch.zeros(5, 2, 128, dtype=torch.bfloat16), good)]:
        with pytest.raises(nosa.NosaError) as e:
            check_run(c, k, v, cu, start, dev)
        assert e.value.status == nosa.NOSA_EINVAL
    i32 = torch.int32
    for cu_, start_ in [(on_cuda(2, dtype=i32), start), (on_cuda(3, dtype=torch.int64), start), (cu, on_cuda(1, dtype=i32)),
                        (cu, on_cuda(2, dtype=torch.int64)), (on_cuda(6, dtype=i32)[::2], start),
                        (torch.zeros(3, dtype=i32), start), (cu, torch.zeros(2, dtype=i32))]:
        with pytest.raises(nosa.NosaError):
            check_run(c, good, good, cu_, start_, dev)
    cache = NosaCache.__new__(NosaCache)
    cache.cfg, cache.device = c, dev
    for call in (cache.write, cache.read):
        with pytest.raises(nosa.NosaError):
            call(good, rows(4, 2, 128), cu, start)


def test_geometry_of_a_4_bit_cache(lib):
    """The tasks are covered, and no group has more ranges than partial slots."""
    for B, k, nbk in ((1, 1, 1), (1, 16, 64), (16, 64, 514), (1, 2048, 2048), (64, 32, 257), (3, 8192, 8192), (5000, 3, 3)):
        for host in (False, True):
            for split in (0, 1, 5, 100):
                g = nosa.step_geometry(cfg(B=B, k_q=k, k_e=0, max_blocks=nbk, attn_split=split), host, 148, 3)
                W, ctas, ng = g["attn_tasks_per_cta"], g["attn_ctas"], 2 * B
                slots = min(max(16, -(-1184 // ng)), 128)
                linear, aligned = -(-ng * k // W), ng * -(-k // W)
                assert ctas in (linear, aligned)
                if ctas == aligned:
                    assert -(-k // W) <= slots
                else:
                    assert -(-(k - 1) // W) + 1 <= slots
                if split:
                    assert W >= split and ctas == linear


def test_split_of_a_4_bit_cache(lib):
    """Even shares over long axes; ranges within the groups where that costs the fullest SM little."""
    def g(**kw):
        x = nosa.step_geometry(cfg(**kw), False, 148, 4 if kw.get("d") == 64 else 3)
        return x["attn_tasks_per_cta"], x["attn_ctas"]

    assert g(B=4, Hq=32, Hkv=8, k_q=2048, k_e=0, max_blocks=2048) == (148, 443)
    assert g(B=8, Hq=16, Hkv=16, d=64, block_size=32, k_q=77, k_e=0, max_blocks=256) == (26, 384)
    assert g(B=6, Hq=64, Hkv=8, block_size=128, k_q=24, k_e=0, max_blocks=128) == (4, 288)
    assert g(B=1, Hq=8, Hkv=2, d=64, k_q=16, k_e=0, max_blocks=65) == (1, 32)


@pytest.mark.parametrize("name", ["k", "v", "cu_tokens", "start"])
@pytest.mark.parametrize("what", [None, 0x100000, [0, 1, 2]])
def test_what_is_not_a_tensor_is_refused(name, what):
    i32 = torch.int32
    run = dict(k=on_cuda(5, 2, 128), v=on_cuda(5, 2, 128), cu_tokens=on_cuda(3, dtype=i32), start=on_cuda(2, dtype=i32))
    run[name] = what
    cache = NosaCache.__new__(NosaCache)
    cache.cfg, cache.device = cfg(), torch.device("cuda", 0)
    if name == "start" and what is None:
        assert check_run(cache.cfg, *run.values(), cache.device) is None
        return
    for call in (cache.write, cache.read):
        with pytest.raises(nosa.NosaError) as e:
            call(**run)
        assert e.value.status == nosa.NOSA_EINVAL and name in str(e.value)
