"""The differential decode where numbers are extreme: infinite queries and keys, and
maps with one key far above the rest.

The error bound is ref_diff.py's with the weights' rounding u as an argument:
d = (u + f) (A_1 + |lambda| A_2), |gpu - ref| <= d + u_out |ref|."""
import numpy as np
import pytest
import torch

import ref_diff
from paged_split_decode_gb300 import inputs
from test_diff_gpu import factors, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_split_decode_gb300 as pd
    pd.load()
    return pd


def reference(w, lam, u, f, norm_weight=None, eps=1e-5, gain=1.0, extra=0.0):
    """(out, bound) of ref_diff.reference with u, f and an absolute term d_0 = ``extra``."""
    out, full = ref_diff.reference(w, lam)
    own = (2.0 ** -11 if (w.kv_fp8 or w.kv_int8) else ref_diff.HALF_STEP[w.q.dtype]) + 2.0 ** (-11 if w.kv_fp8 else -12)
    half = ref_diff.HALF_STEP[w.q.dtype]
    d = (full - half * np.abs(out) - 2.0 ** -24) * ((u + f) / own) + extra
    if norm_weight is not None:
        rms = np.sqrt(np.mean(out ** 2, axis=-1, keepdims=True))
        e = np.sqrt(np.mean(d ** 2, axis=-1, keepdims=True))
        k, lo, hi = (gain / np.sqrt(x ** 2 + eps) for x in (rms, rms + e, np.maximum(rms - e, 0.0)))
        d = np.abs(norm_weight) * (d * hi + np.abs(out) * np.maximum(hi - k, k - lo))
        out = out * k * norm_weight
    return out, d + half * np.abs(out) + 2.0 ** -24


def check(got, ref, bound):
    g = got.float().cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(g))
    excess = np.abs(g - ref) / bound
    assert excess.max() <= 1.0, f"error {excess.max():.2f}x the bound"


# ---------------------------------------------------------------------------
@pytest.mark.parametrize("S", (0, 1, 3))
@pytest.mark.parametrize("sign", (1.0, -1.0))
@pytest.mark.parametrize("kv,qlen", [("f16", 1), ("f16", 3), ("bf16", 1), ("bf16", 3), ("fp8", 1), ("fp8", 3),
                                     ("fp8_bf16q", 1), ("fp8_bf16q", 4), ("int8", 1), ("int8", 3), ("int8_bf16q", 3)])
@pytest.mark.parametrize("Hkv", (2, 4))
def test_an_infinite_query_silences_its_map(pd, Hkv, kv, qlen, sign, S):
    """An infinity in a half of a query row makes every score of that map +infinity,
    -infinity or NaN: no softmax exists, the map contributes zeros."""
    w = inputs.make_workload(B=2, Hq=6 * Hkv, Hkv=Hkv, D=256, seq_lens=[700, 91], qlen=qlen, kv=kv, seed=89,
                             scale=128 ** -0.5)
    lam, _ = factors(w)
    want, alone = run(pd, w, lam, S), run(pd, w, torch.zeros(6 * Hkv), S)
    w.q[1, 7, 200] = sign * float("inf")
    want[1, 7] = alone[1, 7]
    assert torch.equal(run(pd, w, lam, S), want)
    w.q[1, 7, 20] = -sign * float("inf")
    want[1, 7] = 0
    assert torch.equal(run(pd, w, lam, S), want)


@pytest.mark.parametrize("code", (0x00, 0x01, 0x81))
@pytest.mark.parametrize("kv,qlen", [("fp8", 1), ("fp8", 3), ("fp8_bf16q", 3), ("fp8", 5), ("int8", 1), ("int8", 3)])
def test_an_infinite_query_against_small_keys(pd, kv, qlen, code):
    """The same where every key's element beside the infinity is zero (NaN scores) or the smallest there is."""
    w = inputs.make_workload(B=2, Hq=12, Hkv=2, D=256, seq_lens=[700, 5], qlen=qlen, kv=kv, seed=89, scale=128 ** -0.5)
    w.k_cache.view(torch.uint8)[..., 200] = code
    lam, _ = factors(w)
    want, alone = run(pd, w, lam), run(pd, w, torch.zeros(12))
    for i in (0, qlen):  # the first token of each sequence
        w.q[i, 7, 200] = float("inf")
        want[i, 7] = alone[i, 7]
    assert torch.equal(run(pd, w, lam), want)


@pytest.mark.parametrize("qlen", (1, 3))
@pytest.mark.parametrize("kv", ("f16", "bf16"))
def test_an_infinite_key(pd, kv, qlen):
    """An infinity in the second half of a visible key: rows whose score it makes
    +infinity lose that map, the others' softmax gives the key no weight."""
    w = inputs.make_workload(B=2, Hq=12, Hkv=2, D=256, seq_lens=[700, 91], qlen=qlen, kv=kv, seed=93, scale=128 ** -0.5)
    lam, _ = factors(w)
    alone = run(pd, w, torch.zeros(12))
    blk, at = int(w.block_table[0, 5]), 3
    row = w.k_cache[blk, at, 1].clone()
    w.k_cache[blk, at, 1, 130] = float("inf")
    got = run(pd, w, lam)
    # a weight of zero: the same key with a score far below the others
    w.k_cache[blk, at, 1] = row
    plus = w.q[:qlen, 6:, 130] > 0
    for i in range(qlen):
        for h in range(6):
            if plus[i, h]:
                assert torch.equal(got[i, 6 + h], alone[i, 6 + h])
    k = w.k_cache.double()[w.block_table[0].long()].reshape(-1, 2, 256)[:700, 1]
    v = w.v_cache.double()[w.block_table[0].long()].reshape(-1, 2, 256)[:700, 1]
    rest = torch.arange(700) != 5 * 16 + at
    u = ref_diff.HALF_STEP[w.q.dtype]
    for i in range(qlen):
        for h in range(6):
            if plus[i, h]:
                continue
            q, seen = w.q[i, 6 + h].double(), torch.arange(700) <= 700 - qlen + i
            o = a = 0.0
            for m, c in ((0, 1.0), (1, -float(lam[6 + h]))):
                x = k[:, 128 * m:128 * m + 128] @ q[128 * m:128 * m + 128] * w.scale
                p = torch.softmax(torch.where(seen & (rest if m else seen), x, -torch.inf), 0)
                o, a = o + c * (p @ v), a + abs(c) * (p @ v.abs())
            err = (got[i, 6 + h].double().cpu() - o).abs()
            assert torch.all(err <= (u + 2.0 ** -12) * a + u * o.abs() + 2.0 ** -24)


# ---------------------------------------------------------------------------
def peaked(kv, L, qlen, G, seed, peak_value):
    """One key near the middle with a score about 16 above all others in both maps; the
    other keys' values have a common offset of 2.

    q = (+-1 rows of a fixed sign vector) + 0.25 N(0, 1), the peak key 1.45 times
    that vector: its score is 1.45 128 128^-1/2 (1 +- 0.02) = 16.4 +- 0.5; the
    others' N(0, 1) rows score N(0, 1.06)."""
    g = torch.Generator().manual_seed(seed)
    w = inputs.make_workload(B=1, Hq=G, Hkv=1, D=256, seq_lens=[L], qlen=qlen, kv=kv, seed=seed, scale=128 ** -0.5)
    u = torch.where(torch.rand(256, generator=g) < 0.5, -1.0, 1.0)
    w.q = (u + 0.25 * torch.randn(w.q.shape, generator=g)).to(w.q.dtype)
    at = L // 2 + 5
    blk, off = int(w.block_table[0, at // 16]), at % 16

    def codes(x, s):
        if w.kv_int8:
            return (x / s).round().clamp(-127, 127).to(torch.int8).view(torch.uint8)
        if w.kv_fp8:
            return (x / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        return x.to(w.k_cache.dtype)

    noise = torch.randn(w.v_cache.shape, generator=g)
    if w.kv_int8 or w.kv_fp8:
        w.v_scale = 8.0 / (127 if w.kv_int8 else 448)
    w.v_cache = codes(2.0 + noise, w.v_scale)
    w.k_cache[blk, off, 0] = codes(1.45 * u, w.k_scale)
    w.v_cache[blk, off, 0] = codes(peak_value * noise[blk, off, 0], w.v_scale)
    return w


def weight_step(w):
    return 2.0 ** -11 if w.kv_int8 or w.kv_fp8 else ref_diff.HALF_STEP[w.q.dtype]


# The scores' fp32 part of f (2^-13 for scores whose terms sum to less than 11) is
# twice that here (17.5 for the peak); the exponentials and sums stay below it as
# there: f = 2^-12 + 2^-13, and 2^-11 + 2^-13 with e4m3 terms of q.
def peaked_f(w):
    return (2.0 ** -11 if w.kv_fp8 else 2.0 ** -12) + 2.0 ** -13


@pytest.mark.parametrize("S", (0, 1, 3))
@pytest.mark.parametrize("L", (8192, 32768))
@pytest.mark.parametrize("G,qlen", [(6, 3), (4, 3), (6, 4), (8, 4), (6, 1)])
@pytest.mark.parametrize("kv", ("fp8", "fp8_bf16q", "int8", "f16", "bf16"))
def test_the_tail_of_a_peaked_map(pd, kv, G, qlen, L, S):
    """The peak's value is zero, so the output is the tail's alone: weights 2^-23 of
    the peak's, which hold as many bits as any."""
    w = peaked(kv, L, qlen, G, 5 + L + G, 0.0)
    lam = torch.full((G,), 0.97)
    ref, bound = reference(w, lam.double().numpy(), weight_step(w), peaked_f(w))
    assert np.abs(ref).max() > 4e-5  # the tail is there
    check(run(pd, w, lam, S), ref, bound)
    weight = (1 + 0.1 * torch.randn(256, generator=torch.Generator().manual_seed(3))).to(w.q.dtype)
    ref, bound = reference(w, lam.double().numpy(), weight_step(w), peaked_f(w), weight.double().numpy(), 1e-12, 0.4)
    check(run(pd, w, lam, S, weight, norm_eps=1e-12, norm_gain=0.4), ref, bound)


@pytest.mark.parametrize("kv", ("fp8", "int8", "f16"))
@pytest.mark.parametrize("L", (8192, 32768))
@pytest.mark.parametrize("qlen", (1, 3))
def test_a_peak_with_a_value(pd, kv, L, qlen):
    """The peak's own value in the output. Every key's product is added to an
    accumulator of the peak's size, where it loses at most a last place of that
    accumulator, 2^-23 of it: L 2^-23 |v_peak| more."""
    w = peaked(kv, L, qlen, 6, 9 + L, 1.0)
    lam = torch.full((6,), 0.97)
    at = L // 2 + 5
    v = w.v_cache[int(w.block_table[0, at // 16]), at % 16, 0]
    if kv != "f16":
        v = v.view(torch.int8 if kv == "int8" else torch.float8_e4m3fn)
    v = v.double().abs().numpy() * w.v_scale
    ref, bound = reference(w, lam.double().numpy(), weight_step(w), peaked_f(w), extra=1.97 * L * 2.0 ** -23 * v)
    check(run(pd, w, lam), ref, bound)


# ---------------------------------------------------------------------------
@pytest.mark.parametrize("S", (0, 1, 2))
@pytest.mark.parametrize("Hq,Hkv,D,qlen", [(24, 4, 256, 1), (32, 8, 128, 1), (6, 3, 128, 1), (12, 2, 256, 2), (8, 1, 128, 2),
                                           (32, 8, 128, 4), (6, 3, 256, 5)])
@pytest.mark.parametrize("kv", ("f16", "bf16"))
def test_weights_of_two_operands(pd, kv, Hq, Hkv, D, qlen, S):
    """Up to 16 rows per map over 16-bit caches: nothing of a weight's rounding is seen
    where the two maps nearly cancel (lambda = 1, halves alike to 5 %), short
    sequences, so that a single weight's error shows.

    u = 2^-16 (bfloat16) or 2^-22: the rest of a rounded weight, rounded. f: scores
    whose terms sum to less than 3 take at most D / 2 <= 128 additions of 2^-23 of
    that, 2^-14.4; exponentials, sums over 10 keys and the last division stay below
    2^-18: f = 2^-14."""
    B = 40
    lens = [qlen + 2 + i % 8 for i in range(B)]
    w = inputs.make_workload(B=B, Hq=Hq, Hkv=Hkv, D=D, seq_lens=lens, qlen=qlen, kv=kv, seed=D + qlen,
                             scale=(D // 2) ** -0.5)
    h = D // 2
    g = torch.Generator().manual_seed(77)
    w.q = (0.2 * w.q.float()).to(w.q.dtype)
    for x in (w.q, w.k_cache):
        x[..., h:] = (x[..., :h].float() * (1 + 0.05 * torch.randn(x[..., :h].shape, generator=g))).to(x.dtype)
    terms = w.q[..., :h].float().abs().view(-1, h) @ w.k_cache[..., :h].float().abs().view(-1, h).T * w.scale
    assert float(terms.max()) < 3.0
    u = 2.0 ** -22 if kv == "f16" else 2.0 ** -16
    ref, bound = reference(w, np.ones(Hq), u, 2.0 ** -14)
    check(run(pd, w, torch.ones(Hq), S), ref, bound)
