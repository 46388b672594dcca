"""The scored decode against 64 bits: every cache kind, head layout, query count, split and mask; its refusals on the
device, replays and streams."""
import math

import pytest
import torch

from ref_scored import Work, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_split_decode_gb300 as pd
    pd.load()
    return pd


KINDS = [("f16", "f16"), ("bf16", "bf16"), ("fp8", "f16"), ("fp8", "bf16"), ("int8", "f16"), ("int8", "bf16"),
         ("fp4", "f16"), ("fp4", "bf16")]
HEADS = [(24, 4, 256), (8, 4, 128), (6, 3, 256), (5, 1, 128)]


@pytest.mark.parametrize("S", (0, 1, 3))
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("kv,q", KINDS)
def test_kinds_and_splits(pd, kv, q, Hq, Hkv, D, S):
    w = Work(kv, Hq, Hkv, D, [700, 0, 1, 16, 17, 1041, 255], cap=30.0, q=q, seed=1)
    check(w, w.run(pd, S))


# (Hq, Hkv, D, qlen): one to four row tiles of eight rows per KV head
ROWS = [(8, 8, 128, 1), (16, 2, 256, 1), (9, 1, 256, 1), (8, 2, 128, 3), (6, 2, 256, 5), (24, 4, 256, 3), (28, 1, 128, 1),
        (4, 1, 256, 8), (32, 4, 128, 4)]
MASKS = [dict(), dict(window=90), dict(window=1), dict(prefix=[40, 0, 5, 700, 33, 300]), dict(window=64, prefix=[40, 0, 5, 700, 33, 300]),
         dict(window=17, prefix=[2, 1, 5, 16, 100, 250], alibi=True, cap=15.0), dict(alibi=True)]


@pytest.mark.parametrize("mask", range(len(MASKS)))
@pytest.mark.parametrize("Hq,Hkv,D,qlen", ROWS)
@pytest.mark.parametrize("kv", ("f16", "bf16", "fp8", "int8", "fp4"))
def test_rows_and_masks(pd, kv, Hq, Hkv, D, qlen, mask):
    """Sequences shorter than their query tokens, of new tokens only, ending on, before and behind a tile's end."""
    S = (0, 2, 5)[(mask + qlen) % 3]
    w = Work(kv, Hq, Hkv, D, [600, 2, qlen, 703, 704, 321], qlen=qlen, q="f16" if mask % 2 else "bf16", seed=mask, **MASKS[mask])
    check(w, w.run(pd, S, in_place=mask % 2 == 0))


@pytest.mark.parametrize("kv", ("f16", "fp8", "fp4"))
@pytest.mark.parametrize("bs", (32, 48, 64))
def test_block_sizes(pd, kv, bs):
    w = Work(kv, 8, 2, 128, [500, 47, 49, 1], window=100, prefix=[70, 3, 0, 1], bs=bs, seed=3)
    check(w, w.run(pd))


@pytest.mark.parametrize("kv", ("f16", "bf16", "int8", "fp4"))
def test_query_counts_of_their_own(pd, kv):
    w = Work(kv, 24, 4, 256, [500, 40, 1200, 0, 3, 768], qlen=5, qlens=[1, 0, 5, 2, 3, 4], cap=50.0, seed=4)
    out = torch.full((w.q.shape[0] + 3, w.Hq, w.D), 9.0, dtype=w.qt, device="cuda")
    q = w.q
    w.q = torch.cat([q, torch.ones(3, w.Hq, w.D, dtype=w.qt)])  # a padded token buffer
    got = w.run(pd, out=out)
    ref = w.reference()
    check(w, got, ref)
    assert bool((got[0][-3:] == 9.0).all()) and bool((got[1][-3:] == 7.0).all())


def test_bad_query_ranges_and_lengths(pd):
    w = Work("f16", 8, 2, 128, [100, 200, 300], qlen=2, qlens=[1, 2, 1], seed=5)
    ref = w.reference()
    w.starts[2] = 9  # sequence 1 has too many, sequence 2 a negative count
    out, lse, kw, flag = w.run(pd)
    assert flag == pd.DEVERR_QUERY_START
    assert bool(((out.double().cpu() - ref[0]).abs()[0] <= ref[1][0]).all())
    w = Work("fp4", 8, 2, 128, [100, 200, 300], seed=5)
    w.lens[1] = 10 ** 6
    assert w.run(pd, weights=False)[3] == pd.DEVERR_SEQ_LEN
    for kv in ("f16", "fp4"):
        w = Work(kv, 8, 2, 128, [100, 200, 300], seed=5)
        ref = w.reference()
        w.table[1, 3] = 10 ** 6
        w.table[2, 1] = -1
        out, _, _, flag = w.run(pd)
        assert flag == pd.DEVERR_BLOCK_ID
        assert bool(((out.double().cpu() - ref[0]).abs()[0] <= ref[1][0]).all())


def poison(w, i, b, key, head, value):
    """Plants a value at one key and head of cache i (its whole row)."""
    blk, off = int(w.table[b, key // w.bs]), key % w.bs
    if w.kv == "fp4":
        w.sf[i].view(torch.uint8)[blk, head, off] = 0x7F
    elif w.kv == "fp8":
        w.caches[i].view(torch.uint8)[blk, off, head] = 0x7F
    else:
        w.caches[i][blk, off, head] = value


@pytest.mark.parametrize("S", (0, 1, 3))
@pytest.mark.parametrize("kv,Hq,Hkv,D,qlen", [("f16", 24, 4, 256, 1), ("bf16", 8, 2, 128, 3), ("fp8", 6, 2, 256, 2),
                                             ("fp4", 24, 4, 256, 1), ("fp4", 12, 2, 128, 4), ("f16", 4, 1, 256, 8)])
def test_values_that_are_no_numbers(pd, kv, Hq, Hkv, D, qlen, S):
    """NaN and infinities of K and V at keys behind the end, outside a window, in the gap between a prefix and a window,
    and of later query tokens reach the rows that see them and change no bit of the others."""
    lens = [500, 321, 64, 700]
    for i in (0, 1):
        w = Work(kv, Hq, Hkv, D, lens, qlen=qlen, window=100, prefix=[20, 0, 33, 5], seed=7)
        want = w.run(pd, S)
        nan = torch.zeros(w.q.shape, dtype=torch.bool)
        G = Hq // Hkv
        for b, L in enumerate(lens):
            keys = [L - 1, L - qlen, 21, L - qlen - 100, L - 100, 3, L + 1] + ([L - qlen - 99] if qlen > 1 else [])
            for k, key in enumerate(keys):
                if not 0 <= key < w.table.shape[1] * w.bs or (b + k) % 3 == 0:
                    continue
                head = (b + k) % Hkv
                poison(w, i, b, key, head, math.inf if k % 2 else math.nan)
                for t in range(qlen):
                    if bool(w.sees(b, L - qlen + t, torch.tensor(key))):
                        nan[b * qlen + t, head * G:(head + 1) * G] = True
        got = w.run(pd, S)
        bad = ~torch.isfinite(got[0]).cpu()
        if i == 0 and kv in ("f16", "bf16"):  # (an infinite K row: scores of either sign)
            assert not bool((bad & ~nan).any())
        else:
            assert torch.equal(bad, nan)
        assert torch.equal(got[0].cpu()[~nan], want[0].cpu()[~nan])
        rows = ~nan.any(-1)
        assert torch.equal(got[1].cpu()[rows], want[1].cpu()[rows])


@pytest.mark.parametrize("kv", ("f16", "fp8", "fp4"))
def test_rows_of_q_that_are_no_numbers(pd, kv):
    w = Work(kv, 8, 2, 128, [300, 20], q="bf16" if kv == "fp8" else "f16", seed=8)
    want = w.run(pd)[0].cpu()
    w.q[0, 3, 17] = math.nan
    w.q[1, 5, 100] = math.nan
    got = w.run(pd)[0].cpu()
    nan = torch.zeros(w.q.shape[:2], dtype=torch.bool)
    nan[0, 3] = nan[1, 5] = True
    assert torch.equal(torch.isnan(got), nan[..., None].expand_as(got))
    assert torch.equal(got[~nan], want[~nan])


@pytest.mark.parametrize("kv,q", KINDS)
def test_peaked_rows(pd, kv, q):
    """Scores far apart: the reference maximum is raised again and again, and low weights survive."""
    w = Work(kv, 12, 2, 256 if kv != "int8" else 128, [900, 700, 33], q=q, seed=9, spread=6.0)
    out, lse, _, flag = w.run(pd, weights=False)
    r_out, b_out, r_lse, b_lse, _, _ = w.reference()
    assert flag == 0
    # scores are six times as large, and so is what rounding moves a weight by
    assert bool(((out.double().cpu() - r_out).abs() <= 6 * b_out).all())
    assert bool(((lse.double().cpu() - r_lse).abs() <= 6 * b_lse).all())


def test_negative_and_zero_scales(pd):
    for kv in ("f16", "fp4"):
        for scale in (-0.1, 0.0):
            w = Work(kv, 8, 4, 128, [200, 31], window=50, seed=10)
            w.scale = scale
            check(w, w.run(pd))


@pytest.mark.parametrize("kv", ("f16", "fp4"))
def test_replayed_and_on_two_streams(pd, kv):
    """Captured with its own workspace, replayed beside eager calls on another stream."""
    works = [Work(kv, 24, 4, 256, [900, 40, 3000], cap=50.0, seed=s) for s in (1, 2)]
    up = lambda t: None if t is None else t.cuda()
    state = [dict(q=up(w.q), k=up(w.caches[0]), v=up(w.caches[1]), t=up(w.table), l=up(w.lens), ks=up(w.sf[0]), vs=up(w.sf[1]),
                  w_in=up(w.key_weights), w_out=up(w.key_weights), out=torch.empty(w.q.shape, dtype=w.qt, device="cuda"),
                  lse=torch.empty(w.q.shape[:2], device="cuda")) for w in works]

    def call(w, s):
        pd.decode_paged_scored(s["q"], s["k"], s["v"], s["t"], s["l"], w.scale, out=s["out"], score_cap=w.cap, k_block_scale=s["ks"],
                               v_block_scale=s["vs"], k_scale=w.c_scale, v_scale=w.c_scale, lse=s["lse"], key_weights=s["w_in"],
                               key_weights_out=s["w_out"])

    call(works[0], state[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(works[0], state[0])
    side = torch.cuda.Stream()
    for _ in range(20):
        graph.replay()
        with torch.cuda.stream(side):
            call(works[1], state[1])
    torch.cuda.synchronize()
    for w, s in zip(works, state):
        check(w, (s["out"], s["lse"], s["w_out"], 0))


def test_same_bits_whatever_the_batch(pd):
    """A fixed split's result does not depend on the other sequences, nor on where the blocks lie."""
    for kv in ("f16", "fp4"):
        w = Work(kv, 8, 2, 128, [600, 300, 900], seed=11)
        want = w.run(pd, 3)
        order = torch.randperm(w.caches[0].shape[0], generator=torch.Generator().manual_seed(1))
        back = torch.argsort(order)
        for i in range(2):
            w.caches[i] = w.caches[i].view(torch.uint8)[order].view(w.caches[i].dtype)
            if w.sf[i] is not None:
                w.sf[i] = w.sf[i].view(torch.uint8)[order].view(w.sf[i].dtype)
        w.table = back[w.table.long()].int()
        w.key_weights = w.key_weights[order]
        got = w.run(pd, 3)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(got[2].cpu()[back], want[2].cpu())


def test_a_wait_that_runs_out(pd):
    from paged_split_decode_gb300 import binding
    w = Work("f16", 24, 4, 256, [500, 900], seed=12)
    binding.set_wait_limit_ns(20_000_000)
    binding.set_fault_injection(1)
    try:
        assert w.run(pd, weights=False)[3] == pd.DEVERR_TIMEOUT
    finally:
        binding.set_fault_injection(0)
        binding.set_wait_limit_ns(0)
    check(w, w.run(pd))


def test_nothing_to_do(pd):
    w = Work("fp4", 8, 2, 128, [0, 0], seed=13)
    out, lse, kw, flag = w.run(pd)
    assert flag == 0 and bool((out == 0).all()) and bool((lse == -math.inf).all())
    assert torch.equal(kw.cpu(), w.key_weights)


def test_binding_refusals(pd):
    w = Work("fp4", 8, 2, 128, [30], seed=14)
    up = lambda t: t.cuda()
    args = [up(w.q), up(w.caches[0]), up(w.caches[1]), up(w.table), up(w.lens), w.scale]
    sf = dict(k_block_scale=up(w.sf[0]), v_block_scale=up(w.sf[1]))
    with pytest.raises(ValueError):
        pd.decode_paged_scored(*args, k_block_scale=sf["k_block_scale"])
    with pytest.raises(ValueError):
        pd.decode_paged_scored(*args, k_block_scale=sf["k_block_scale"][..., :4], v_block_scale=sf["v_block_scale"][..., :4])
    with pytest.raises(ValueError):
        pd.decode_paged_scored(*args, **sf, alibi_slopes=torch.ones(3, device="cuda"))
    with pytest.raises(ValueError):
        pd.decode_paged_scored(*args, **sf, key_weights_out=up(w.key_weights))
    with pytest.raises(ValueError):
        pd.decode_paged_scored(*args, **sf, key_weights=up(w.key_weights)[:, :1])
    with pytest.raises(TypeError):
        pd.decode_paged_scored(*args, **sf, prefix_lens=torch.zeros(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(pd.DecodeError):
        pd.decode_paged_scored(*args, **sf, score_cap=-1.0)
    with pytest.raises(pd.DecodeError):
        pd.decode_paged_scored(*args, **sf, key_weights=up(w.key_weights), workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises((TypeError, ValueError, pd.DecodeError)):
        pd.decode_paged(*args)  # 4-bit caches are the scored decode's


@pytest.mark.parametrize("q", ("f16", "bf16"))
@pytest.mark.parametrize("kv,one", [("f16", 0.92), ("bf16", 0.92), ("fp8", 72.0), ("int8", 24.0), ("fp4", None)])
@pytest.mark.parametrize("qlen", (1, 3))
def test_a_dominant_key(pd, kv, one, q, qlen):
    """One key weighs 2^15 times as much as each of 8000 others, which together count for a fifth of the output. Three-term
    weights are held to 2^-22 of the largest, for each key: 2^-22 sum |v| beside the usual bound."""
    w = Work(kv, 6, 1, 128, [8000], qlen=qlen, q=q, seed=15)
    w.q = torch.ones_like(w.q)
    at = (int(w.table[0, 0]), slice(None), 0) if kv == "fp4" else (int(w.table[0, 0]), 0)
    w.caches[0] = torch.zeros_like(w.caches[0])
    if kv == "fp4":
        w.caches[0][at], w.sf[0][at] = 0x66, 40.0  # (code 4)
        w.caches[1] &= 0x77
    else:
        w.caches[0][at] = torch.tensor(one).to(w.caches[0].dtype)
        w.caches[1] = w.caches[1].float().abs().to(w.caches[1].dtype)
    ref = list(w.reference())
    ref[1] = ref[1] + 2.0 ** -22 * w.value(1)[w.table[0].long()].flatten(0, 1).abs().sum(0).max()
    check(w, w.run(pd), ref)
