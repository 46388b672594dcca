"""GPU parity of the differential decode (decode_paged_diff) against 64 bits;
the error bound is derived in ref_diff.py."""
import numpy as np
import pytest
import torch

import ref_diff
from paged_split_decode_gb300 import inputs

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
KINDS = ("f16", "bf16", "fp8", "int8", "fp8_bf16q", "int8_bf16q")


@pytest.fixture(scope="module")
def pd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_split_decode_gb300 as pd
    pd.load()
    return pd


def caches(w):
    k, v = w.k_cache.to(DEV), w.v_cache.to(DEV)
    return (k.view(torch.int8), v.view(torch.int8)) if w.kv_int8 else (k, v)


def factors(w, seed=0):
    g = torch.Generator().manual_seed(seed)
    lam = 0.2 + 0.6 * torch.rand(w.Hq, generator=g)
    weight = (1 + 0.1 * torch.randn(w.D, generator=g)).to(w.q.dtype)
    return lam, weight


def run(pd, w, lam, S=0, weight=None, out=None, flag=None, **kw):
    k, v = caches(w)
    res = pd.decode_paged_diff(w.q.to(DEV), k, v, w.block_table.to(DEV), w.seq_lens.to(DEV), lam.to(DEV), w.scale,
                               w.window, w.qlen, S, out=out,
                               query_start_loc=None if w.q_start is None else w.q_start.to(DEV),
                               norm_weight=None if weight is None else weight.to(DEV), k_scale=w.k_scale,
                               v_scale=w.v_scale, error_flag=flag, **kw)
    torch.cuda.synchronize()
    return res


def check(got, ref, bound):
    g = got.float().cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(g))
    excess = np.abs(g - ref) / bound
    assert excess.max() <= 1.0, f"error {excess.max():.2f}x the bound"
    empty = np.all(ref == 0.0, axis=-1)
    assert np.all(g[empty] == 0.0), "rows without a key are not zero"


def parity(pd, w, S=0, norm=False, **kw):
    lam, weight = factors(w, w.meta.get("seed", 0))
    weight = weight if norm else None
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = run(pd, w, lam, S, weight, flag=flag, **kw)
    assert int(flag.item()) == 0
    ref, bound = ref_diff.reference(w, lam.double().numpy(), None if weight is None else weight.double().numpy(),
                                    kw.get("norm_eps", 1e-5), kw.get("norm_gain", 1.0))
    check(got, ref, bound)
    return got


# every cache kind, head size, tile grouping (Hkv % 4) and count of row tiles
# per map (G * qlen of 1 to 32), with empty, one-key and ragged sequences
@pytest.mark.parametrize("norm", (False, True))
@pytest.mark.parametrize("Hq,Hkv,D,qlen", [
    (4, 4, 256, 1), (24, 4, 256, 1), (32, 8, 128, 1), (12, 2, 256, 1), (3, 3, 128, 1), (12, 2, 256, 2),
    (28, 4, 128, 2), (24, 4, 256, 3), (12, 2, 128, 3), (8, 1, 256, 4), (32, 8, 128, 8)])
@pytest.mark.parametrize("kv", KINDS)
def test_parity(pd, kv, Hq, Hkv, D, qlen, norm):
    w = inputs.make_workload(B=5, Hq=Hq, Hkv=Hkv, D=D, seq_lens=[300, 0, max(1, qlen - 1), 17, 129], qlen=qlen, kv=kv,
                             seed=Hq + D + qlen, scale=(D // 2) ** -0.5, stale="nan")
    parity(pd, w, norm=norm)


@pytest.mark.parametrize("S", (0, 1, 2, 3, 8, 40))
@pytest.mark.parametrize("kv", ("f16", "bf16", "fp8_bf16q", "int8"))
def test_splits_agree(pd, kv, S):
    w = inputs.make_workload(B=3, Hq=12, Hkv=4, D=256, seq_lens=[1000, 5, 2049], kv=kv, seed=7, scale=128 ** -0.5)
    parity(pd, w, S, norm=True, norm_gain=0.4)


@pytest.mark.parametrize("window", (1, 15, 16, 100, 5000))
@pytest.mark.parametrize("S", (0, 1, 5))
def test_window(pd, window, S):
    w = inputs.make_workload(B=4, Hq=8, Hkv=2, D=128, seq_lens=[700, 64, 0, 33], qlen=3, window=window, kv="f16",
                             seed=11, scale=0.125)
    parity(pd, w, S)


@pytest.mark.parametrize("block_size", (16, 48, 128))
def test_block_sizes(pd, block_size):
    w = inputs.make_workload(B=3, Hq=8, Hkv=4, D=128, seq_lens=[700, 1, 333], kv="bf16", block_size=block_size, seed=13,
                             scale=0.125, stale="nan")
    parity(pd, w, norm=True)


@pytest.mark.parametrize("B", (1, 2, 200, 300, 1200))
def test_batches(pd, B):
    """One sequence over all SMs, more units than SMs (finished by their own
    piece), and batches beyond the cached (256) and the balanced (1024) ones."""
    rng = np.random.RandomState(B)
    lens = [3000] if B == 1 else [int(x) for x in rng.randint(0, 60, B)]
    w = inputs.make_workload(B=B, Hq=8, Hkv=4, D=128, seq_lens=lens, kv="f16", seed=17, scale=0.125)
    parity(pd, w, norm=True)


@pytest.mark.parametrize("kv", ("f16", "fp8"))
@pytest.mark.parametrize("S", (0, 1, 4))
def test_varlen(pd, kv, S):
    w = inputs.make_varlen_workload(B=6, qlens=[1, 0, 4, 2, 3, 1], Hq=24, Hkv=4, D=256,
                                    seq_lens=[500, 40, 1200, 0, 2, 77], kv=kv, seed=19, scale=128 ** -0.5)
    parity(pd, w, S, norm=True)


def test_varlen_leaves_other_rows(pd):
    w = inputs.make_varlen_workload(B=3, qlens=[2, 1, 1], Hq=8, Hkv=2, D=128, seq_lens=[50, 20, 30], kv="f16", seed=23,
                                    scale=0.125)
    lam, _ = factors(w)
    q = torch.cat([w.q, w.q[:3]])
    k, v = caches(w)
    out = torch.full((q.shape[0], 8, 128), 7.0, dtype=torch.float16, device=DEV)
    pd.decode_paged_diff(q.to(DEV), k, v, w.block_table.to(DEV), w.seq_lens.to(DEV), lam.to(DEV), w.scale, qlen=2,
                         out=out, query_start_loc=w.q_start.to(DEV))
    ref, bound = ref_diff.reference(w, lam.double().numpy())
    check(out[:4], ref, bound)
    assert torch.all(out[4:] == 7.0)


def test_lambda_zero_is_the_first_map_alone(pd):
    """lambda = 0: the plain decode on q and K whose second halves are zero."""
    w = inputs.make_workload(B=2, Hq=8, Hkv=4, D=256, seq_lens=[400, 90], kv="f16", seed=29, scale=128 ** -0.5)
    got = run(pd, w, torch.zeros(8))
    ref, bound = ref_diff.reference(w, np.zeros(8))
    check(got, ref, bound)
    q, k = w.q.clone(), w.k_cache.clone()
    q[..., 128:] = 0
    plain = pd.decode_paged(q.to(DEV), k.to(DEV), w.v_cache.to(DEV), w.block_table.to(DEV), w.seq_lens.to(DEV), w.scale)
    check(plain, ref, bound)


def test_norm_weight_in_float32_and_zero_eps(pd):
    w = inputs.make_workload(B=3, Hq=8, Hkv=4, D=128, seq_lens=[200, 0, 65], kv="f16", seed=31, scale=0.125)
    lam, weight = factors(w)
    got = run(pd, w, lam, 0, weight.float(), norm_eps=0.0, norm_gain=2.5)
    ref, bound = ref_diff.reference(w, lam.double().numpy(), weight.double().numpy(), 1e-300, 2.5)
    check(got, ref, bound)


def test_same_bits_again_and_after_other_calls(pd):
    w = inputs.make_workload(B=4, Hq=24, Hkv=4, D=256, seq_lens=[900, 31, 2000, 64], kv="bf16", seed=37,
                             scale=128 ** -0.5)
    lam, weight = factors(w)
    a = run(pd, w, lam, 0, weight).clone()
    other = inputs.make_workload(B=2, Hq=8, Hkv=2, D=128, seq_lens=[3000, 100], kv="f16", seed=38, scale=0.125)
    run(pd, other, factors(other)[0])
    assert torch.equal(a, run(pd, w, lam, 0, weight))


def test_bad_tables_and_lengths_raise_bits(pd):
    w = inputs.make_workload(B=3, Hq=8, Hkv=4, D=128, seq_lens=[100, 40, 64], kv="f16", seed=41, scale=0.125)
    lam, _ = factors(w)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    w.block_table[1, 0] = 10_000
    got = run(pd, w, lam, flag=flag)
    assert int(flag.item()) == pd.DEVERR_BLOCK_ID
    w.block_table[1, 0] = 0
    w.seq_lens[1] = 7000
    flag.zero_()
    run(pd, w, lam, flag=flag)
    assert int(flag.item()) & pd.DEVERR_SEQ_LEN
    ref, bound = ref_diff.reference(inputs.make_workload(B=3, Hq=8, Hkv=4, D=128, seq_lens=[100, 40, 64], kv="f16",
                                                         seed=41, scale=0.125), lam.double().numpy())
    check(got[0:1], ref[0:1], bound[0:1])  # the other sequences are not disturbed
    check(got[2:3], ref[2:3], bound[2:3])


@pytest.mark.parametrize("Hq,Hkv,qlen,kv", [(8, 4, 1, "f16"), (8, 4, 1, "fp8"), (6, 2, 1, "f16"), (12, 4, 3, "bf16"),
                                            (12, 2, 3, "int8"), (24, 4, 4, "f16"), (24, 4, 5, "fp8")])
def test_a_wait_that_runs_out_reports(pd, Hq, Hkv, qlen, kv):
    """Every kernel shape gives up its waits, reports, and works again."""
    from paged_split_decode_gb300 import binding
    w = inputs.make_workload(B=2, Hq=Hq, Hkv=Hkv, D=128, seq_lens=[1000, 40], qlen=qlen, kv=kv, seed=43, scale=0.125)
    lam, weight = factors(w)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    binding.set_wait_limit_ns(2_000_000)
    binding.set_fault_injection(1)
    try:
        for S in (0, 1):
            run(pd, w, lam, S, weight, flag=flag)
    finally:
        binding.set_fault_injection(0)
        binding.set_wait_limit_ns(0)
    assert int(flag.item()) == pd.DEVERR_TIMEOUT
    parity(pd, w, norm=True)


@pytest.mark.parametrize("scale", (-0.125, 0.0, 1.5))
@pytest.mark.parametrize("kv", ("f16", "fp8_bf16q", "int8"))
def test_scales(pd, kv, scale):
    """A negative factor, none, and one that makes the maps peaked (scores of
    up to about 60: the fp32 part of the bound, 2^-13 for scores whose terms sum
    to less than 11, grows with them)."""
    w = inputs.make_workload(B=2, Hq=8, Hkv=4, D=128, seq_lens=[300, 37], kv=kv, seed=61, scale=scale)
    lam, _ = factors(w)
    got = run(pd, w, lam)
    ref, bound = ref_diff.reference(w, lam.double().numpy())
    check(got, ref, bound * (12.0 if scale > 1 else 1.0))


def test_rising_scores_raise_the_reference(pd):
    """Keys that grow along the sequence: every tile passes the running maximum,
    by little and by much."""
    w = inputs.make_workload(B=2, Hq=8, Hkv=4, D=128, seq_lens=[600, 91], kv="f16", seed=67, scale=0.125)
    ramp = torch.linspace(0.0, 3.0, 600)
    for b, L in enumerate((600, 91)):
        for j in range(L):
            w.k_cache[int(w.block_table[b, j // 16]), j % 16] *= ramp[j]
    for S in (0, 1, 3):
        lam, _ = factors(w)
        ref, bound = ref_diff.reference(w, lam.double().numpy())
        check(run(pd, w, lam, S), ref, 4.0 * bound)  # (rows three times as large: scores' fp32 part with them)


def test_offsets_past_32_bits(pd):
    """Blocks at the end of caches of about 10 GB each give what the same
    blocks give in a small cache."""
    w = inputs.make_workload(B=2, Hq=8, Hkv=4, D=256, seq_lens=[333, 64], kv="f16", seed=71, scale=128 ** -0.5)
    lam, weight = factors(w)
    want = run(pd, w, lam, 0, weight)
    n, pool = 300_000, w.k_cache.shape[0]
    big = [torch.empty(n, 16, 4, 256, dtype=torch.float16, device=DEV) for _ in range(2)]
    for c, small in zip(big, (w.k_cache, w.v_cache)):
        c[n - pool:] = small.to(DEV)
    table = torch.where(w.block_table >= 0, w.block_table + (n - pool), w.block_table).int()
    got = pd.decode_paged_diff(w.q.to(DEV), *big, table.to(DEV), w.seq_lens.to(DEV), lam.to(DEV), w.scale,
                               norm_weight=weight.to(DEV))
    assert torch.equal(got, want)


@pytest.mark.parametrize("kv,qlen", [("f16", 1), ("fp8_bf16q", 3), ("int8", 4)])
def test_two_streams_and_two_captured_graphs(pd, kv, qlen):
    """Calls without a workspace on two streams, and two graphs captured on
    one stream and replayed on two, do not share partials."""
    ws = [inputs.make_workload(B=2, Hq=24, Hkv=4, D=256, seq_lens=[3000, 2000], qlen=qlen, kv=kv, seed=s,
                               scale=128 ** -0.5) for s in (47, 48)]
    lams = [factors(w)[0] for w in ws]
    want = [run(pd, w, lam).clone() for w, lam in zip(ws, lams)]
    args = []
    for w, lam in zip(ws, lams):
        k, v = caches(w)
        args.append(dict(q=w.q.to(DEV), k_cache=k, v_cache=v, block_table=w.block_table.to(DEV),
                         seq_lens=w.seq_lens.to(DEV), lam=lam.to(DEV), scale=w.scale, qlen=qlen, k_scale=w.k_scale,
                         v_scale=w.v_scale))
    outs = [torch.empty_like(a["q"]) for a in args]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, a, o in zip(streams, args, outs):
            with torch.cuda.stream(s):
                pd.decode_paged_diff(**a, out=o)
    torch.cuda.synchronize()
    assert all(torch.equal(o, x) for o, x in zip(outs, want))
    graphs = []
    for a, o in zip(args, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[0]):
            pd.decode_paged_diff(**a, out=o)
        graphs.append(g)
        o.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, x) for o, x in zip(outs, want))


def test_an_explicit_stream_handle(pd):
    w = inputs.make_workload(B=2, Hq=8, Hkv=4, D=128, seq_lens=[900, 33], kv="f16", seed=53, scale=0.125)
    lam, weight = factors(w)
    want = run(pd, w, lam, 0, weight)
    s = torch.cuda.Stream()
    got = run(pd, w, lam, 0, weight, stream=s.cuda_stream)
    assert torch.equal(got, want)


def test_a_workspace_too_small_is_refused(pd):
    w = inputs.make_workload(B=2, Hq=8, Hkv=4, D=128, seq_lens=[900, 33], kv="f16", seed=53, scale=0.125)
    lam, _ = factors(w)
    with pytest.raises(pd.DecodeError, match="workspace"):
        run(pd, w, lam, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    need = pd.diff_workspace_bytes(pd.dims_of(w.q, w.k_cache, w.block_table, 1), 1, 0)
    parity(pd, w, workspace=torch.empty(need, dtype=torch.uint8, device=DEV))


# byte caches with 9 to 32 query rows per map: the tensor-memory engine (three
# sizes of units, both head sizes), rings that wrap, pieces that start inside a
# sequence, windows whose first block is cut
@pytest.mark.parametrize("window", (0, 700))
@pytest.mark.parametrize("S", (0, 1, 3, 9, 40))
@pytest.mark.parametrize("Hq,Hkv,D,qlen", [(12, 2, 256, 3), (12, 2, 128, 5), (8, 2, 256, 3), (8, 2, 128, 8)])
@pytest.mark.parametrize("kv", ("fp8", "fp8_bf16q", "int8"))
def test_many_rows_long(pd, kv, Hq, Hkv, D, qlen, S, window):
    w = inputs.make_workload(B=4, Hq=Hq, Hkv=Hkv, D=D, seq_lens=[2600, 0, 1301, 70], qlen=qlen, window=window, kv=kv,
                             seed=73 + D, scale=(D // 2) ** -0.5, stale="nan")
    parity(pd, w, S, norm=S != 3)


@pytest.mark.parametrize("kv", ("fp8", "int8_bf16q"))
def test_many_rows_varlen(pd, kv):
    """Units of 24, 0, 6, 12 and 18 rows in one batch, more units than SMs."""
    qlens = [4, 0, 1, 2, 3] * 16
    rng = np.random.RandomState(3)
    w = inputs.make_varlen_workload(B=80, qlens=qlens, Hq=24, Hkv=4, D=256,
                                    seq_lens=[max(q, int(x)) for q, x in zip(qlens, rng.randint(0, 900, 80))], kv=kv,
                                    seed=79, scale=128 ** -0.5)
    parity(pd, w, norm=True)


@pytest.mark.parametrize("S", (1, 3))
@pytest.mark.parametrize("kv", ("fp8", "int8"))
def test_many_rows_rising_scores(pd, kv, S):
    """Keys that grow along the sequence: thresholds rise in late blocks, the
    accumulators are rescaled. (Scores of twice the usual size: 4 bounds.)"""
    w = inputs.make_workload(B=2, Hq=12, Hkv=2, D=256, seq_lens=[1500, 291], qlen=2, kv=kv, seed=83, scale=0.25)
    for b, L in enumerate((1500, 291)):
        for j in range(L):
            row = w.k_cache[int(w.block_table[b, j // 16]), j % 16]
            codes = row.view(torch.int8 if kv == "int8" else torch.float8_e4m3fn)
            x = codes.float() * (j / 1500)
            row.copy_((x.round() if kv == "int8" else x).to(codes.dtype).view(row.dtype))
    lam, _ = factors(w)
    ref, bound = ref_diff.reference(w, lam.double().numpy())
    check(run(pd, w, lam, S), ref, 4.0 * bound)


@pytest.mark.parametrize("S", (0, 1, 3))
@pytest.mark.parametrize("kv,qlen", [("f16", 1), ("bf16", 3), ("fp8", 1), ("fp8_bf16q", 3), ("int8", 3)])
def test_a_nan_score_silences_its_map(pd, kv, qlen, S):
    """A NaN in the second half of one head's query row: that row's second map
    contributes nothing (as with lambda = 0), no other row changes. A NaN in the
    first half too: the row is zero."""
    w = inputs.make_workload(B=2, Hq=12, Hkv=2, D=256, seq_lens=[700, 91], qlen=qlen, kv=kv, seed=89, scale=128 ** -0.5)
    lam, _ = factors(w)
    want, alone = run(pd, w, lam, S), run(pd, w, torch.zeros(12), S)
    w.q[1, 7, 200] = float("nan")
    want[1, 7] = alone[1, 7]
    assert torch.equal(run(pd, w, lam, S), want)
    w.q[1, 7, 20] = float("nan")
    want[1, 7] = 0
    assert torch.equal(run(pd, w, lam, S), want)


@pytest.mark.parametrize("qlen", (1, 3))
def test_nan_codes_of_visible_keys(pd, qlen):
    """A NaN code in a K row silences the map of its half for the KV head's rows that
    see the key, one in a V row shows in its dimension of the rows that see it."""
    w = inputs.make_workload(B=2, Hq=12, Hkv=2, D=256, seq_lens=[700, 91], qlen=qlen, kv="fp8", seed=101, scale=128 ** -0.5)
    lam, _ = factors(w)
    want, alone = run(pd, w, lam), run(pd, w, torch.zeros(12))
    w.k_cache.view(torch.uint8)[int(w.block_table[0, 5]), 3, 1, 130] = 0x7F  # second half, KV head 1
    w.v_cache.view(torch.uint8)[int(w.block_table[1, 2]), 9, 0, 77] = 0xFF
    got = run(pd, w, lam)
    want[:qlen, 6:] = alone[:qlen, 6:]
    assert torch.isnan(got[qlen:, :6, 77]).all()
    got[qlen:, :6, 77] = want[qlen:, :6, 77]
    assert torch.equal(got, want)


@pytest.mark.parametrize("B,L,kv,qlen", [(4, 600, "fp8", 3), (16, 900, "int8", 3), (1, 1500, "fp8_bf16q", 4),
                                         (1, 16, "f16", 1), (48, 128, "f16", 1), (100, 60, "bf16", 3), (1, 300, "int8", 3),
                                         (48, 200, "fp8_bf16q", 3), (80, 500, "fp8", 2), (300, 33, "fp8", 1)])
def test_short_tables(pd, B, L, kv, qlen):
    """Tables of few blocks, where the automatic plan leaves units whole or cuts
    them into the pieces of a cluster."""
    lens = [L if i % 7 == 0 else (i * 37) % (L + 1) for i in range(B)]
    w = inputs.make_workload(B=B, Hq=24, Hkv=4, D=256, seq_lens=lens, qlen=qlen, kv=kv, seed=97, scale=128 ** -0.5,
                             stale="nan")
    parity(pd, w, norm=True)


@pytest.mark.parametrize("S", (0, 1, 5))
@pytest.mark.parametrize("Hq,Hkv,D,qlen", [(12, 2, 256, 2), (24, 4, 256, 3), (28, 4, 128, 3), (6, 3, 128, 1), (32, 8, 128, 1)])
@pytest.mark.parametrize("kv", ("f16", "bf16", "fp8", "int8_bf16q"))
def test_empty_units_between_odd_ones(pd, kv, Hq, Hkv, D, qlen, S):
    """Units without keys between units of odd tile counts, many to a CTA: an
    empty one takes nothing from the ring, wherever the last one left it."""
    lens = [(qlen, 0, 17, 0, 0, 33, 40, 0, 5, 0, 90, 0)[i % 12] if i % 5 else 0 for i in range(400)]
    w = inputs.make_workload(B=400, Hq=Hq, Hkv=Hkv, D=D, seq_lens=lens, qlen=qlen, kv=kv, seed=103 + D,
                             scale=(D // 2) ** -0.5, stale="nan")
    for _ in range(3):
        parity(pd, w, S, norm=True)


@pytest.mark.parametrize("seed", range(48))
def test_drawn_calls(pd, seed):
    """Heads, lengths, query counts, windows, splits and kinds drawn together."""
    r = np.random.RandomState(7000 + seed)
    pick = lambda *v: v[r.randint(len(v))]
    D, Hkv, G, q = pick(128, 256), pick(1, 2, 3, 4, 5, 8), pick(1, 2, 3, 4, 6, 7), pick(1, 1, 2, 3, 4, 5, 8)
    q = min(q, 32 // G)
    B, top = pick((1, 1500), (3, 1500), (7, 400), (20, 200), (60, 100))
    lens = [pick(0, r.randint(top + 1), r.randint(top + 1)) for _ in range(B - 1)] + [top]
    kw = dict(B=B, Hq=G * Hkv, Hkv=Hkv, D=D, seq_lens=lens, kv=pick(*KINDS), window=pick(0, 0, 1, 9, 100), seed=seed,
              scale=(D // 2) ** -0.5)
    if r.randint(2):
        w = inputs.make_varlen_workload(qlens=[r.randint(q + 1) for _ in range(B - 1)] + [q], **kw)
    else:
        w = inputs.make_workload(qlen=q, block_size=pick(16, 32, 48), stale="nan", **kw)
    parity(pd, w, pick(0, 0, 1, 2, 3, 7, 16, 33), norm=bool(r.randint(2)))
