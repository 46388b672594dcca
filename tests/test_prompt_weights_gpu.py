"""A prompt written into recycled blocks, whose weights are cleared as the documentation says, decoded and cut by the weights
that it collects: against a host model that knows nothing of the blocks' last owner."""
import pytest
import torch

from ref_scored import fp4_values
from test_fp4_writer_gpu import quantise

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ("fp4", "f16"))
def test_prompt_in_recycled_blocks(kv):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_split_decode_gb300 as pd
    pd.load()
    B, Hq, Hkv, D, bs, g0 = 2, 8, 2, 128, 16, 0.05
    n, cols, keep, first, recent = 16, 8, 48, 2, 8
    gen = torch.Generator().manual_seed(71)
    i32 = dict(dtype=torch.int32, device="cuda")
    if kv == "fp4":
        caches = [torch.zeros(n, Hkv, bs, D // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
        sf = [torch.zeros(n, Hkv, bs, D // 16, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)]
        scales, gains = dict(k_block_scale=sf[0], v_block_scale=sf[1]), dict(k_scale=g0, v_scale=g0)
    else:
        caches, sf, scales, gains = [torch.zeros(n, bs, Hkv, D, dtype=torch.float16, device="cuda") for _ in range(2)], [], {}, {}
    table, lens = torch.full((B, cols), -1, **i32), torch.zeros(B, **i32)
    free, count, flag = torch.randperm(n, generator=gen).int().cuda(), torch.full((1,), n, **i32), torch.zeros(1, **i32)
    weights = torch.empty(n, Hkv, bs, device="cuda").uniform_(0.0, 100.0)  # (a buffer that was never cleared)
    stored = (lambda x: fp4_values(*quantise(x, g0), float(torch.tensor(g0)))) if kv == "fp4" else (lambda x: x.double())

    def bring(counts):
        T = sum(counts)
        k, v = (torch.randn(T, Hkv, D, generator=gen).half() for _ in range(2))
        _, start, slots, _ = pd.build_block_tables(lens, torch.tensor(counts, **i32), table, free, count, bs, T, seq_lens=lens, error_flag=flag)
        if kv == "fp4":
            pd.write_kv_cache_fp4(k.cuda(), v.cuda(), slots, *caches, *sf, error_flag=flag, **gains)
        else:
            pd.write_kv_cache(k.cuda(), v.cuda(), slots, *caches, error_flag=flag)
        return k, v, start, slots

    for owner in range(3):
        prompt = [(101, 60), (75, 126), (120, 98)][owner]
        model = [dict(k=torch.zeros(0, Hkv, D, dtype=torch.float64), w=torch.zeros(0, Hkv, dtype=torch.float64)) for _ in range(B)]
        k, v, _, slots = bring(list(prompt))
        new = slots[slots >= 0]
        weights.transpose(1, 2)[new // 16, new % 16] = 0
        at = 0
        for b in range(B):
            model[b]["k"] = stored(k)[at:at + prompt[b]]
            model[b]["w"] = torch.zeros(prompt[b], Hkv, dtype=torch.float64)
            at += prompt[b]
        for _ in range(2):
            k, v, start, _ = bring([1, 1])
            q = torch.randn(B, Hq, D, generator=gen).half() * 2
            pd.decode_paged_scored(q.cuda(), *caches, table, lens, D ** -0.5, query_start_loc=start, key_weights=weights,
                                   error_flag=flag, **scales, **gains)
            for b, m in enumerate(model):
                m["k"] = torch.cat([m["k"], stored(k)[b:b + 1]])
                m["w"] = torch.cat([m["w"], torch.zeros(1, Hkv, dtype=torch.float64)])
                y = torch.einsum("hgd,jhd->hgj", q[b].double().view(Hkv, -1, D), m["k"]) * D ** -0.5
                m["w"] += torch.softmax(y, -1).sum(1).T
        pd.evict_kv_cache(*caches, weights, table, lens, keep, first=first, recent=recent, free_blocks=free, free_count=count,
                          error_flag=flag, **scales)
        torch.cuda.synchronize()
        assert int(flag.item()) == 0 and lens.tolist() == [keep] * B
        j = torch.arange(keep)
        for b, m in enumerate(model):
            L = m["w"].shape[0]
            for h in range(Hkv):
                w = m["w"][:, h]
                mid = torch.sort(w[first:L - recent], descending=True, stable=True)
                want = keep - first - recent
                # (kept and dropped weights lie apart by more than the kernels' rounding, or the test's data is changed)
                assert float(mid.values[want - 1] - mid.values[want]) > 1e-5 * float(mid.values[want])
                idx = torch.cat([torch.arange(first), torch.sort(mid.indices[:want]).values + first, torch.arange(L - recent, L)])
                got = weights[table[b].long().cpu()[j // bs].cuda(), h, (j % bs).cuda()].double().cpu()
                # (fp32 scores of 128 products and two steps' sums: ref_scored's bound)
                assert bool(((got - w[idx]).abs() <= 2.0 ** -11 * w[idx]).all())
        pd.release_blocks(table, lens, torch.ones(B, dtype=torch.bool, device="cuda"), free, count, bs, error_flag=flag)
        torch.cuda.synchronize()
        assert int(count.item()) == n and lens.tolist() == [0] * B
