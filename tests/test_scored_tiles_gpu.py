"""The scored decode's kernels for two to four row tiles (tensor memory for e4m3, and for int8 under a bfloat16 q; a warp a
row tile else): masked NaN codes, waits that run out; and for every kernel many sequences and caches past 4 GiB."""

import pytest
import torch

from ref_scored import Work, check
from test_fp4_writer_gpu import quantise

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_split_decode_gb300 as pd
    pd.load()
    return pd


@pytest.mark.parametrize("S", (0, 1, 3))
@pytest.mark.parametrize("q", ("f16", "bf16"))
@pytest.mark.parametrize("Hq,Hkv,D,qlen", [(12, 2, 256, 3), (6, 1, 128, 5), (8, 2, 128, 3), (20, 1, 256, 1)])
def test_masked_nan_codes(pd, Hq, Hkv, D, qlen, q, S):
    """NaN codes of V and K at keys that some rows see, and some do not, reach the former and change no bit of the latter."""
    lens = [500, 321, 64, 700]
    G = Hq // Hkv
    for i in (0, 1):
        w = Work("fp8", Hq, Hkv, D, lens, qlen=qlen, q=q, window=100, prefix=[20, 0, 33, 5], seed=7)
        want = w.run(pd, S)
        nan = torch.zeros(w.q.shape, dtype=torch.bool)
        for b, L in enumerate(lens):
            for k, key in enumerate((L - 1, L - qlen, 21, L - qlen - 100, L - 100, 3, L + 1, L - qlen - 99)):
                if not 0 <= key < w.table.shape[1] * w.bs or (b + k) % 3 == 0:
                    continue
                head = (b + k) % Hkv
                blk, off = int(w.table[b, key // w.bs]), key % w.bs
                dims = slice(None) if i == 0 else slice(k, D, 37)  # (of V: the outputs of these dims only)
                w.caches[i].view(torch.uint8)[blk, off, head, dims] = 0x7F if k % 2 else 0xFF
                for t in range(qlen):
                    if bool(w.sees(b, L - qlen + t, torch.tensor(key))):
                        nan[b * qlen + t, head * G:(head + 1) * G, dims] = True
        got = w.run(pd, S)
        assert torch.equal(~torch.isfinite(got[0]).cpu(), nan)
        assert torch.equal(got[0].cpu()[~nan], want[0].cpu()[~nan])
        rows = ~nan.any(-1) if i == 0 else torch.ones(nan.shape[:2], dtype=torch.bool)
        assert torch.equal(got[1].cpu()[rows], want[1].cpu()[rows])


@pytest.mark.parametrize("kv,q,qlen", [("f16", "f16", 2), ("f16", "f16", 5), ("fp8", "f16", 3), ("fp8", "bf16", 3), ("int8", "bf16", 3),
                                      ("int8", "f16", 2), ("int8", "f16", 1)])
def test_a_wait_that_runs_out(pd, kv, q, qlen):
    from paged_split_decode_gb300 import binding
    w = Work(kv, 24, 4, 256, [500, 900], qlen=qlen, q=q, seed=12)
    binding.set_wait_limit_ns(20_000_000)
    binding.set_fault_injection(1)
    try:
        assert w.run(pd, weights=False)[3] == pd.DEVERR_TIMEOUT
    finally:
        binding.set_fault_injection(0)
        binding.set_wait_limit_ns(0)
    check(w, w.run(pd))


@pytest.mark.parametrize("kv,q,qlen", [("f16", "f16", 1), ("bf16", "bf16", 3), ("fp8", "bf16", 3), ("int8", "bf16", 2), ("fp4", "f16", 1),
                                      ("fp4", "bf16", 4)])
def test_many_sequences(pd, kv, q, qlen):
    """More sequences than the balanced split plans and than its cache of lengths holds."""
    for B in (700, 2100):
        lens = [(37 * b) % 70 for b in range(B)]
        w = Work(kv, 12, 2, 128, lens, qlen=qlen, q=q, window=30, prefix=[b % 9 for b in range(B)], seed=16)
        check(w, w.run(pd))


@pytest.mark.parametrize("kv,q,qlen", [("f16", "f16", 1), ("f16", "f16", 3), ("fp8", "bf16", 3), ("int8", "bf16", 3), ("int8", "f16", 3),
                                      ("fp4", "f16", 1), ("fp4", "bf16", 3)])
def test_blocks_past_4gib(pd, kv, q, qlen):
    """Blocks beyond 4 GiB of every cache, decoded, and moved down to the first ones."""
    w = Work(kv, 24, 4, 256, [1000, 37, 2049], qlen=qlen, q=q, window=300, prefix=[30, 0, 90], seed=17)
    ref = w.reference()
    small = w.caches[0].shape[0]
    per_block = w.caches[0][0].numel() * w.caches[0].element_size()
    n = (9 << 29) // per_block + small
    if kv == "fp4":  # rows of (key, head) stay below 2^31
        assert n * 64 < 1 << 31
    dev = {}

    def grow(t):
        big = torch.empty((n,) + tuple(t.shape[1:]), dtype=t.dtype, device="cuda")
        big[n - small:] = t.cuda()
        return big

    args = [grow(c) for c in w.caches]
    dev = dict(zip(("k_block_scale", "v_block_scale"), (grow(s) for s in w.sf))) if kv == "fp4" else {}
    weights = grow(w.key_weights)
    lse = torch.empty(w.q.shape[:2], device="cuda")
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = pd.decode_paged_scored(w.q.cuda(), *args, (w.table + (n - small)).cuda(), w.lens.cuda(), w.scale, w.window, qlen,
                                 prefix_lens=w.prefix.cuda(), k_scale=w.c_scale, v_scale=w.c_scale, lse=lse, key_weights=weights,
                                 error_flag=flag, **dev)
    torch.cuda.synchronize()
    check(w, (out, lse, weights[n - small:], int(flag.item())), ref)
    # the rows of blocks past 4 GiB, moved down to the first ones
    low = torch.arange(3 * 8, dtype=torch.int32).view(3, 8)
    lens = pd.evict_kv_cache(*args, weights, (w.table + (n - small)).cuda(), w.lens.cuda(), 100, recent=100,
                             block_table_out=low.cuda(), error_flag=flag, **dev)
    torch.cuda.synchronize()
    assert int(flag.item()) == 0 and lens.tolist() == [100, 37, 100]
    for b, L in enumerate((1000, 37, 2049)):
        i = torch.arange(min(L, 100))
        src = max(0, L - 100) + i
        sb, tb = w.table[b, src // 16].long(), low[b, i // 16].long()
        for j in range(2):
            got = args[j][:24].view(torch.uint8).cpu()
            have = w.caches[j].view(torch.uint8)
            if kv == "fp4":
                assert torch.equal(got[tb, :, i % 16], have[sb, :, src % 16])
            else:
                assert torch.equal(got[tb, i % 16], have[sb, src % 16])
    del args, dev, weights
    torch.cuda.empty_cache()


def test_4bit_writer_past_4gib(pd):
    Hkv, D, bs, T = 4, 256, 16, 100
    n = (9 << 29) // (Hkv * bs * D // 2)
    caches = [torch.empty(n, Hkv, bs, D // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
    sfs = [torch.empty(n, Hkv, bs, D // 16, dtype=torch.uint8, device="cuda") for _ in range(2)]
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(T, Hkv, D, generator=g).half() for _ in range(2))
    slots = n * bs - 1 - torch.randperm(400, generator=g)[:T]
    for t in caches + sfs:
        t[-25:] = 0x11
    pd.write_kv_cache_fp4(k.cuda(), v.cuda(), slots.cuda(), *caches, *sfs, k_scale=0.1, v_scale=0.1)
    torch.cuda.synchronize()
    for x, c, s in ((k, caches[0], sfs[0]), (v, caches[1], sfs[1])):
        codes, sf = quantise(x, 0.1)
        want_c = torch.full((25, Hkv, bs, D // 2), 0x11, dtype=torch.uint8)
        want_s = torch.full((25, Hkv, bs, D // 16), 0x11, dtype=torch.uint8)
        at = slots - (n - 25) * bs
        want_c[at // bs, :, at % bs], want_s[at // bs, :, at % bs] = codes, sf
        assert torch.equal(c[-25:].cpu(), want_c) and torch.equal(s[-25:].cpu(), want_s)
    del caches, sfs
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kv,q", [("fp8", "f16"), ("fp8", "bf16"), ("int8", "bf16"), ("f16", "f16")])
def test_log_sum_exp_of_few_keys(pd, kv, q):
    """Products of q with codes are exact, their sums fp32's: a row of one or two keys has its log-sum-exp to D 2^-24 of
    sum |q k| scale (D = 256, each product at most 2^-24 of the sum so far off), and a few roundings of itself."""
    w = Work(kv, 24, 4, 256, [1, 2] * 20, qlen=3, q=q, seed=18)
    lse = w.run(pd)[1].double().cpu()
    want = w.reference()[2]
    K = w.value(0)
    for b, L in enumerate(w.lens.tolist()):
        for t in range(3 - L, 3):
            n = t - (3 - L) + 1  # keys that the token sees
            at = w.table[b, 0].long()
            for h in range(4):
                mag = (w.q[b * 3 + t, h * 6:(h + 1) * 6].double().abs() @ K[at, :n, h].abs().T).max(-1).values * w.scale
                err = (lse[b * 3 + t, h * 6:(h + 1) * 6] - want[b * 3 + t, h * 6:(h + 1) * 6]).abs()
                assert bool((err <= 256 * 2.0 ** -24 * mag + 2.0 ** -21 * (want[b * 3 + t, h * 6:(h + 1) * 6].abs() + 1)).all())
    rel = float((lse - want)[torch.isfinite(want)].norm() / want[torch.isfinite(want)].norm())
    assert rel <= 1e-6  # (and as a whole: random roundings add as a root of their number, 16 2^-24 of a score)
