"""Host-side checks of the scored decode, the 4-bit writer and the eviction that need no GPU: workspaces, and the
refusals made before anything is launched; models of the arithmetic that their kernels use."""
import ctypes
import math

import numpy as np
import pytest
import torch

import paged_split_decode_gb300 as pd
from paged_split_decode_gb300 import binding, build

FP4, FP4_BF16 = 6, 7
NULL, SHAPE, DTYPE, UNSUPPORTED, ALIGN, WORKSPACE = 1, 2, 3, 4, 5, 6


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def _dims(**kw):
    base = dict(B=32, Hq=24, Hkv=4, D=256, block_size=16, num_blocks=10000, max_blocks_per_seq=256)
    kind = kw.pop("kind", None)
    base.update(kw)
    d = binding.make_dims(**base)
    if kind is not None:
        d.kv_dtype = kind
    return d


def up(x):
    return (x + 255) // 256 * 256


def _scored(lib, dims, q=16, k=16, v=16, bt=16, sl=16, qs=None, T=32, out=16, qlen=1, splits=1, scale=0.1, ws=None, ws_bytes=0,
            score=True, **parts):
    s = binding.PdScore(**parts)
    return lib.decode_paged_scored(q, k, v, bt, sl, qs, T, scale, 0, qlen, splits, ctypes.byref(s) if score else None, out,
                                   ctypes.byref(dims) if dims else None, ws, ws_bytes, None, None)


@pytest.mark.parametrize("kind", (0, FP4, FP4_BF16))
def test_scored_refusals(lib, kind):
    d = _dims(kind=kind)
    sf = dict(k_block_scale=16, v_block_scale=16) if kind >= FP4 else {}
    assert _scored(lib, None, **sf) == NULL
    assert _scored(lib, d, score=False) == NULL
    assert _scored(lib, _dims(kind=kind, D=64), **sf) == UNSUPPORTED
    assert _scored(lib, _dims(kind=kind, block_size=8), **sf) == UNSUPPORTED
    assert _scored(lib, _dims(kind=kind, Hkv=5), **sf) == SHAPE
    assert _scored(lib, _dims(kind=kind, Hq=132), qlen=1, **sf) == UNSUPPORTED
    assert _scored(lib, _dims(kind=8)) == DTYPE
    for name in ("q", "k", "v", "bt", "sl", "out"):
        assert _scored(lib, d, **{name: None}, **sf) == NULL
    for name in ("q", "k", "v", "out"):
        assert _scored(lib, d, **{name: 0x1008}, **sf) == ALIGN
    for name in ("alibi_slopes", "prefix_lens", "lse", "key_weights", "key_weights_out"):
        assert _scored(lib, d, **{name: 18}, **sf) == ALIGN
    assert _scored(lib, d, k_block_scale=24, v_block_scale=16) == ALIGN
    for cap in (-1.0, math.nan, math.inf, 1e-38, 3e38):
        assert _scored(lib, d, cap=cap, **sf) == SHAPE
    assert _scored(lib, d, splits=-1, **sf) == SHAPE
    assert _scored(lib, d, qlen=0, **sf) == SHAPE
    assert _scored(lib, d, scale=math.nan, **sf) == SHAPE
    assert _scored(lib, d, qs=16, T=-1, **sf) == SHAPE
    assert _scored(lib, _dims(kind=kind, num_blocks=0), **sf) == SHAPE
    assert _scored(lib, _dims(kind=kind, B=0), **sf) == 0  # nothing to do
    assert _scored(lib, d, qs=16, T=0, **sf) == 0


def test_fp4_decode_kind_is_the_scored_decodes(lib):
    d = _dims(kind=FP4)
    assert lib.pd_workspace_bytes(ctypes.byref(d), 1, 0, 152) == 0
    assert lib.decode_paged(16, 16, 16, 16, 16, 0.1, 0, 1, 1, 16, ctypes.byref(d), None, 0, None, None) == DTYPE
    k = torch.zeros(2, dtype=torch.int64)
    assert lib.write_kv_cache(16, 16, k.data_ptr(), 2, 16, 16, ctypes.byref(d), None, None) == DTYPE
    big = _dims(kind=FP4, num_blocks=1 << 26, Hkv=4)  # rows of (key, head) beyond 31 bits
    assert _scored(lib, big, k_block_scale=16, v_block_scale=16) == UNSUPPORTED


def test_scored_workspace(lib):
    """Partials as the plain decode's, then the rows' (m, l), then 16 x 8 scores for every tile and row tile."""
    for kind in (0, FP4):
        d = _dims(kind=kind)
        plain = binding.scored_workspace_bytes(d, 1, 0, False, sm_count=152)
        assert plain > 0
        both = binding.scored_workspace_bytes(d, 1, 0, True, sm_count=152)
        assert both == up(plain) + up(32 * 24 * 8) + 32 * 4 * 256 * 512
        one = binding.scored_workspace_bytes(d, 1, 1, False, sm_count=152)
        assert one == 0 and binding.scored_workspace_bytes(d, 1, 1, True, sm_count=152) == up(32 * 24 * 8) + 32 * 4 * 256 * 512
        assert binding.scored_workspace_bytes(d, 9, 0, True, sm_count=152) == 0  # (54 rows of a head)


def _write(lib, dims, k=32, v=32, slots=8, T=2, kc=32, vc=32, ks=32, vs=32):
    return lib.write_kv_cache_fp4(k, v, slots, T, kc, vc, ks, vs, ctypes.byref(dims) if dims else None, None, None)


def test_writer_refusals(lib):
    d = _dims(kind=FP4)
    assert _write(lib, None) == NULL
    for name in ("k", "v", "slots", "kc", "vc", "ks", "vs"):
        assert _write(lib, d, **{name: None}) == NULL
    for kw in (dict(k=8), dict(v=8), dict(kc=4), dict(vc=4), dict(slots=4)):
        assert _write(lib, d, **kw) == ALIGN
    assert _write(lib, _dims(kind=0)) == DTYPE
    assert _write(lib, _dims(kind=FP4, D=24)) == SHAPE
    assert _write(lib, d, T=-1) == SHAPE
    for name in ("k_scale", "v_scale"):
        for g in (0.0, -1.0, math.nan, math.inf):
            bad = _dims(kind=FP4)
            setattr(bad, name, g)
            assert _write(lib, bad) == SHAPE
    assert _write(lib, d, T=0) == 0


def _evict(lib, dims, keep=64, trigger=None, first=0, recent=0, k=16, v=16, ks=None, vs=None, w=16, bt=16, sl=16, bto=None,
           cols=0, slo=16, free=None, count=None, ws=256, ws_bytes=1 << 40):
    e = binding.PdEviction(keep=keep, trigger=keep if trigger is None else trigger, first=first, recent=recent)
    return lib.evict_kv_cache(k, v, ks, vs, w, bt, sl, ctypes.byref(e), bto, cols, slo, free, count,
                              ctypes.byref(dims) if dims else None, ws, ws_bytes, None, None)


def test_evict_refusals(lib):
    d, d4 = _dims(), _dims(kind=FP4)
    assert _evict(lib, None) == NULL
    for kw in (dict(keep=0), dict(trigger=63), dict(first=-1), dict(recent=-1), dict(first=60, recent=5),
               dict(first=2 ** 31 - 1, recent=2 ** 31 - 1)):
        assert _evict(lib, d, **kw) == SHAPE
    assert _evict(lib, _dims(kind=8)) == DTYPE
    assert _evict(lib, _dims(D=24)) == SHAPE
    assert _evict(lib, _dims(D=1024)) == UNSUPPORTED
    assert _evict(lib, _dims(num_blocks=1 << 28)) == UNSUPPORTED
    assert _evict(lib, _dims(kind=FP4, D=32), ks=16, vs=16) == UNSUPPORTED  # (two bytes of scales a row)
    for name in ("k", "v", "w", "bt", "sl", "slo"):
        assert _evict(lib, d, **{name: None}) == NULL
    assert _evict(lib, d4) == NULL  # no block scales
    for kw in (dict(k=8), dict(v=8), dict(w=18), dict(bt=18), dict(sl=18), dict(slo=18), dict(ws=64)):
        assert _evict(lib, d, **kw) == ALIGN
    assert _evict(lib, d4, ks=8, vs=16) == ALIGN
    assert _evict(lib, d, free=16) == NULL and _evict(lib, d, count=16) == NULL
    assert _evict(lib, d, free=16, count=16, bto=16, cols=4) == SHAPE
    assert _evict(lib, d, bto=16, cols=3) == SHAPE  # 48 slots for 64 keys
    assert _evict(lib, d, trigger=100, bto=16, cols=6) == SHAPE  # and for the 100 of a sequence that is not cut
    assert _evict(lib, d, ws=None) == WORKSPACE
    e = binding.PdEviction(keep=64, trigger=80, first=0, recent=0)
    need = lib.pd_evict_workspace_bytes(ctypes.byref(d), ctypes.byref(e))
    assert need == up(32 * 4 * 80 * 20) + 32 * 4
    assert _evict(lib, d, trigger=80, ws_bytes=need - 1) == WORKSPACE
    assert _evict(lib, _dims(B=0)) == 0
    e = binding.PdEviction(keep=64, trigger=10 ** 9, first=0, recent=0)  # never more than the table holds
    assert lib.pd_evict_workspace_bytes(ctypes.byref(d), ctypes.byref(e)) == up(32 * 4 * 4096 * 20) + 32 * 4


def test_python_refusals():
    """What the binding refuses before it asks for a device."""
    h, i32, f32, u8 = torch.float16, torch.int32, torch.float32, torch.uint8
    q, c = torch.zeros(2, 8, 128, dtype=h), torch.zeros(4, 16, 4, 128, dtype=h)
    table, lens = torch.zeros(2, 3, dtype=i32), torch.zeros(2, dtype=i32)
    c4, sf, w = torch.zeros(4, 4, 16, 64, dtype=u8), torch.zeros(4, 4, 16, 8, dtype=u8), torch.zeros(4, 4, 16)
    ok = dict(q=q, k_cache=c, v_cache=c, block_table=table, seq_lens=lens, scale=0.1)
    for kw in (dict(qlen=2), dict(out=q[:1]), dict(query_start_loc=lens), dict(v_cache=c[:1]), dict(alibi_slopes=torch.zeros(4)),
               dict(prefix_lens=lens[:1]), dict(lse=torch.zeros(2, 7)), dict(key_weights=w[:, :2]), dict(key_weights_out=w),
               dict(k_cache=c4, v_cache=c4, k_block_scale=sf), dict(k_cache=c4, v_cache=c4, k_block_scale=sf[:3], v_block_scale=sf),
               dict(k_cache=c[0], v_cache=c[0])):
        with pytest.raises(ValueError):
            pd.decode_paged_scored(**{**ok, **kw})
    for kw in (dict(k_block_scale=sf, v_block_scale=sf), dict(k_cache=c.int(), v_cache=c.int()), {}):  # ({}: not on a GPU)
        with pytest.raises(TypeError):
            pd.decode_paged_scored(**{**ok, **kw})
    x, slots = torch.zeros(2, 4, 128, dtype=h), torch.zeros(2, dtype=torch.int64)
    with pytest.raises(TypeError):
        pd.write_kv_cache_fp4(x.float(), x.float(), slots, c4, c4, sf, sf)
    for args in ((x[:1], x[:1], slots, c4, c4, sf, sf), (x, x[:1], slots, c4, c4, sf, sf), (x, x, slots, c4, c4[:1], sf, sf),
                 (x, x, slots, c4, c4, sf[..., :4], sf[..., :4])):
        with pytest.raises(ValueError):
            pd.write_kv_cache_fp4(*args)
    free, count = torch.zeros(4, dtype=i32), torch.zeros(1, dtype=i32)
    for kw in (dict(block_table=table[0]), dict(seq_lens=lens[:1]), dict(block_table_out=table[:1]), dict(seq_lens_out=free),
               dict(key_weights=w[:1]), dict(free_blocks=free[:2], free_count=count), dict(free_blocks=free, free_count=lens)):
        a = dict(k_cache=c, v_cache=c, key_weights=w, block_table=table, seq_lens=lens, keep=8)
        with pytest.raises(ValueError):
            pd.evict_kv_cache(**{**a, **kw})


def test_division_by_multiplication():
    """n / d = (mulhi(m, n) + n) >> l for n < 2^31 (the eviction's block numbers)."""
    rng = np.random.default_rng(0)
    for d in [1, 2, 3, 5, 7, 16, 17, 31, 32, 33, 48, 80, 641, 65535, 65536, 65537, 2 ** 30 - 1, 2 ** 30, 2 ** 31 - 1]:
        l = 0
        while (1 << l) < d:
            l += 1
        m = ((1 << 32) * ((1 << l) - d)) // d + 1
        assert m < 1 << 32
        k = rng.integers(0, (2 ** 31 - 1) // d + 1, 2000)
        for n in np.concatenate([rng.integers(0, 2 ** 31, 2000), k * d, np.maximum(k * d - 1, 0), [0, 1, 2 ** 31 - 1]]).tolist():
            t = (m * n) >> 32
            assert t + n < 1 << 32
            assert (t + n) >> l == n // d


def test_tanh_model():
    """The kernels' tanh in fp32: a Taylor polynomial below 1/2, 1 - 2 / (1 + e^2u) above; within 2^-21 of itself (the
    exponential and the quotient to two units in the last place each)."""
    f = np.float32
    u = np.concatenate([np.linspace(1e-6, 12, 200_001), 10.0 ** np.linspace(-30, 2, 1001)]).astype(f)
    v = u * u
    s = f(21844 / 6081075)
    for c in (-1382 / 155925, 62 / 2835, -17 / 315, 2 / 15, -1 / 3):
        s = (s.astype(np.float64) * v + c).astype(f) if isinstance(s, np.ndarray) else (np.float64(s) * v + c).astype(f)
    s = (s.astype(np.float64) * v * u + u).astype(f)
    for wobble in (1 - 2.0 ** -22, 1.0, 1 + 2.0 ** -22):
        with np.errstate(over="ignore"):
            e = (np.exp(2 * u.astype(np.float64)) * wobble).astype(f)
            t = (1 - (2.0 / (1 + e).astype(np.float64) * wobble).astype(f)).astype(f)
        got = np.where(v < 0.25, s, t).astype(np.float64)
        want = np.tanh(u.astype(np.float64))
        assert np.max(np.abs(got - want) / want) < 2.0 ** -21


def test_corrected_quotient():
    """The 4-bit writer's quotients by a reciprocal and one residual equal the divided ones: scales of groups, and values up
    to seven times the divisor."""
    rng = np.random.default_rng(1)
    f = np.float32
    fma = lambda a, b, c: (a.astype(np.longdouble) * b.astype(np.longdouble) + c.astype(np.longdouble)).astype(f)
    assert np.finfo(np.longdouble).nmant >= 60 or pytest.skip("no 64-bit mantissa here")
    for _ in range(20):
        x = rng.standard_normal(20_000).astype(np.float16).astype(f)
        for d in (np.abs(x[::-1]) + f(0.2), np.full_like(x, f(6 * rng.random() + 1e-3))):
            d = d.astype(f)
            r = (f(1) / d).astype(f)
            q0 = (x * r).astype(f)
            q1 = fma(fma(-q0, d, x), r, q0)
            assert np.array_equal(q1, (x / d).astype(f))
