"""What the scored decode's precision is, held tightly: the norm of the outputs' error beside what rounding the result alone
leaves, and log-sum-exp and key weights where every product is exact.

Error norm. A row's error is what rounding the exact output leaves, e0, and what rounding the weights leaves, e1, independent
of it: err^2 <= e0^2 + e1^2 (norms relative to the output's). Weights' roundings are independent of each other, so that with
each at most u the sum over a row's keys moves by less than u of its norm. u = 2^-20 for two fp16 operands, 2^-15 for two of
bfloat16, 2^-11 for one of fp16 (a bfloat16 output over 8- and 4-bit caches), 2^-12 for three e4m3 ones. The fp32 parts:
D = 256 products summed 16 at a time, each partial sum of at most 2^5 cut at 2^-23 of it, times the scale of 1 / 16: 2^-18 of a
weight; ex2 2^-22. So e1 = 2^-16 beside u, and twice as much is allowed: e1 = 2 (u + 2^-16).

Exact products. q is one and K's rows are constant multiples of a power of two, so that a score s is exact in fp32. Then
x = s c with c = scale log2(e) k_scale has three roundings (scale and k_scale as fp32, their product, this one) of at most
|x| <= 5.2 at 2^-24: 2^-20 log2 units, and a weight moves by ln 2 of it, 2^-20.5. ex2 adds 2^-22, a lane's sum over at most 512
keys 64 additions of 2^-24: 2^-18, the joins, the quotient and the logarithm less than 2^-20: f = 2^-17 for all of it, 2^6 below
what one 16-bit rounding of a weight could hide in."""
import pytest
import torch

from ref_scored import Work, check

KINDS = [("f16", "f16"), ("bf16", "bf16"), ("fp8", "f16"), ("fp8", "bf16"), ("int8", "f16"), ("int8", "bf16"),
         ("fp4", "f16"), ("fp4", "bf16")]


def rounding(w):
    """u of the module's text."""
    if w.qt == torch.bfloat16:
        return 2.0 ** -15 if w.kv == "bf16" else 2.0 ** -11
    return 2.0 ** -12 if w.kv == "fp8" and w.Hq // w.Hkv * w.qlen > 8 else 2.0 ** -20


def error_norms(out, ref, qt):
    """(of `out`, of the rounded reference), relative to the reference's."""
    norm = float(ref.norm())
    return float((out.double().cpu() - ref).norm()) / norm, float((ref.to(qt).double() - ref).norm()) / norm


def within(out, ref, qt, u):
    err, e0 = error_norms(out, ref, qt)
    return err ** 2 <= e0 ** 2 + (2 * (u + 2.0 ** -16)) ** 2, (err, e0)


@pytest.fixture(scope="module")
def pd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_split_decode_gb300 as pd
    pd.load()
    return pd


@pytest.mark.gpu
@pytest.mark.parametrize("S", (0, 1, 3))
@pytest.mark.parametrize("qlen", (1, 3))
@pytest.mark.parametrize("kv,q", KINDS)
def test_error_norm(pd, kv, q, qlen, S):
    w = Work(kv, 24, 4, 256, [900, 1500, 260], qlen=qlen, q=q, seed=81)
    out = w.run(pd, S)[0]
    ok, norms = within(out, w.reference()[0], w.qt, rounding(w))
    assert ok, norms


@pytest.mark.parametrize("kv,q,one", [("f16", "f16", torch.float16), ("bf16", "bf16", torch.bfloat16), ("fp4", "f16", torch.float16),
                                      ("int8", "f16", torch.float16), ("fp4", "bf16", torch.bfloat16), ("fp8", "bf16", torch.bfloat16)])
def test_a_dropped_operand_is_seen(kv, q, one):
    """On the host: weights rounded once more coarsely than documented fail the bound, as documented they hold it."""
    w = Work(kv, 6, 1, 256, [900, 260], q=q, seed=82)
    ref, K, V = w.reference()[0], w.value(0), w.value(1)

    def outputs(operands):
        out = torch.zeros_like(ref)
        for b, L in enumerate(w.lens.tolist()):
            j = torch.arange(L)
            at = (w.table[b, j // 16].long(), j % 16, 0)
            y = w.q[b].double() @ K[at].T * w.scale
            p = torch.exp(y - y.amax(-1, keepdim=True)) * 128
            used, rest = torch.zeros_like(p), p
            for t in operands:
                used, rest = used + rest.to(t).double(), rest - rest.to(t).double()
            out[b] = used @ V[at] / p.sum(-1, keepdim=True)
        return out.to(w.qt)

    given = [torch.float16] if rounding(w) == 2.0 ** -11 else [one, one]
    assert within(outputs(given), ref, w.qt, rounding(w))[0]
    ok, norms = within(outputs([one]), ref, w.qt, rounding(w))
    assert not ok, norms


def exact_work(kv, q, qlen):
    w = Work(kv, 12, 2, 128, [512, 1, 130, 37], qlen=qlen, q=q, seed=83)
    g = torch.Generator().manual_seed(84)
    w.q = torch.ones_like(w.q)
    if kv == "fp4":
        c = torch.randint(0, 8, w.caches[0].shape[:3] + (1,), generator=g).to(torch.uint8)
        w.caches[0] = (c | (c << 4)).expand(w.caches[0].shape).contiguous()
        w.sf[0] = torch.full_like(w.sf[0].float(), 8.0).to(torch.float8_e4m3fn)
    else:
        step = {"f16": 1 / 16, "bf16": 1 / 16, "fp8": 4.0, "int8": 1.0}[kv]
        top = {"f16": 6, "bf16": 6, "fp8": 7, "int8": 9}[kv]
        c = torch.randint(0, top, w.caches[0].shape[:3] + (1,), generator=g) * step
        w.caches[0] = c.expand(w.caches[0].shape).contiguous().to(w.caches[0].dtype)
    return w


@pytest.mark.gpu
@pytest.mark.parametrize("S", (0, 1, 3))
@pytest.mark.parametrize("qlen", (1, 3))
@pytest.mark.parametrize("kv,q", KINDS)
def test_exact_products(pd, kv, q, qlen, S):
    w = exact_work(kv, q, qlen)
    f = 2.0 ** -17
    ref = list(w.reference())
    got = (ref[5] - 2.0 ** -22 * ref[4]) * 2.0 ** 11  # the call's own weights
    ref[3] = f + 2.0 ** -22 * ref[2].abs()
    ref[5] = f * got + 2.0 ** -22 * ref[4]
    out = w.run(pd, S)
    check(w, out, ref)
    live = ~torch.isnan(ref[2])
    ok, norms = within(out[0][live], ref[0][live], w.qt, rounding(w) + f)
    assert ok, norms


@pytest.mark.gpu
@pytest.mark.parametrize("S", (0, 1, 3))
@pytest.mark.parametrize("qlen", (1, 3))
@pytest.mark.parametrize("kv", ("f16", "bf16"))
def test_rows_of_minus_infinity(pd, kv, qlen, S):
    """Keys are visible, but every score is -infinity: zeros, with a log-sum-exp of -infinity and no weight to any key."""
    import math
    w = Work(kv, 24, 4, 256, [300, 20], qlen=qlen, seed=85)
    want = w.run(pd, S)
    w.q = torch.ones_like(w.q)
    rows = w.table[1].long()
    w.caches[0][rows] = -math.inf
    out, lse, kw, flag = w.run(pd, S)
    assert flag == 0 and bool((out[qlen:] == 0).all()) and bool((lse[qlen:] == -math.inf).all())
    at = w.table[1].long()[torch.arange(20) // 16]
    old = w.key_weights[at, :, torch.arange(20) % 16]
    old[20 - qlen:] = 0
    assert torch.equal(kw.cpu()[at, :, torch.arange(20) % 16], old)
    assert bool(torch.isfinite(out).all()) and want[3] == 0
