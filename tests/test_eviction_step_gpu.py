"""Serving steps over a bounded cache: block tables, the 4-bit (or fp16) writer, the scored decode with its keys' weights,
and the eviction that goes by them, captured in one graph each and replayed; against a host model that keeps every
head's keys itself."""
import pytest
import torch

from ref_scored import HALF_STEP, fp4_values
from test_fp4_writer_gpu import quantise

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ("fp4", "f16"))
def test_steps(kv):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_split_decode_gb300 as pd
    pd.load()
    B, Hq, Hkv, D, bs, keep, trigger, first, recent = 3, 8, 2, 128, 16, 40, 55, 2, 8
    cols, n, steps, g0 = 5, 3 * 4 + 1, 130, 0.05
    gen = torch.Generator().manual_seed(4)
    i32 = dict(dtype=torch.int32, device="cuda")
    if kv == "fp4":
        caches = [torch.zeros(n, Hkv, bs, D // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
        sf = [torch.zeros(n, Hkv, bs, D // 16, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)]
        scales = dict(k_block_scale=sf[0], v_block_scale=sf[1])
    else:
        caches = [torch.zeros(n, bs, Hkv, D, dtype=torch.float16, device="cuda") for _ in range(2)]
        scales = {}
    gains = dict(k_scale=g0, v_scale=g0) if kv == "fp4" else {}
    table, lens, query = torch.full((B, cols), -1, **i32), torch.zeros(B, **i32), torch.zeros(B, **i32)
    free, count, flag = torch.randperm(n, generator=gen).int().cuda(), torch.full((1,), n, **i32), torch.zeros(1, **i32)
    weights = torch.full((n, Hkv, bs), float("nan"), device="cuda")  # new keys start from zero by themselves
    T = 2 * B
    q, k, v = (torch.zeros(T, h, D, dtype=torch.float16, device="cuda") for h in (Hq, Hkv, Hkv))
    out = torch.zeros_like(q)

    def step():
        _, start, slots, _ = pd.build_block_tables(lens, query, table, free, count, bs, T, seq_lens=lens, error_flag=flag)
        if kv == "fp4":
            pd.write_kv_cache_fp4(k, v, slots, *caches, *sf, error_flag=flag, **gains)
        else:
            pd.write_kv_cache(k, v, slots, *caches, error_flag=flag)
        pd.decode_paged_scored(q, *caches, table, lens, D ** -0.5, qlen=2, out=out, query_start_loc=start, score_cap=30.0,
                               key_weights=weights, error_flag=flag, **scales, **gains)
        pd.evict_kv_cache(*caches, weights, table, lens, keep, trigger=trigger, first=first, recent=recent, free_blocks=free,
                          free_count=count, error_flag=flag, **scales)

    state = (table, lens, free, count, weights, *caches, *(sf if kv == "fp4" else ()))
    saved = [t.clone() for t in state]
    query.fill_(1)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, s in zip(state, saved):
        t.copy_(s)
    flag.zero_()

    # the model: keys, values and weights of every sequence and head, in slot order
    model = [[dict(k=torch.zeros(0, D, dtype=torch.float64), v=torch.zeros(0, D, dtype=torch.float64),
                   w=torch.zeros(0, dtype=torch.float64)) for _ in range(Hkv)] for _ in range(B)]
    stored = (lambda x: fp4_values(*quantise(x, g0), float(torch.tensor(g0, dtype=torch.float32)))) if kv == "fp4" else (lambda x: x.double())
    cuts = 0
    for s in range(steps):
        counts = [(s + b) % 3 if s % 4 else 1 + (b & 1) for b in range(B)]
        q.copy_(torch.randn(T, Hq, D, generator=gen) * 2)
        k.copy_(torch.randn(T, Hkv, D, generator=gen))
        v.copy_(torch.randn(T, Hkv, D, generator=gen))
        query.copy_(torch.tensor(counts, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert int(flag.item()) == 0
        K, V, Q, got = stored(k.cpu()), stored(v.cpu()), q.double().cpu(), out.double().cpu()
        row = 0
        for b in range(B):
            c = counts[b]
            for h in range(Hkv):
                m = model[b][h]
                m["k"], m["v"] = torch.cat([m["k"], K[row:row + c, h]]), torch.cat([m["v"], V[row:row + c, h]])
                m["w"] = torch.cat([m["w"], torch.zeros(c, dtype=torch.float64)])
                L = m["w"].numel()
                G = Hq // Hkv
                for i in range(c):
                    see = L - c + i + 1
                    y = 30.0 * torch.tanh(Q[row + i, h * G:(h + 1) * G] @ m["k"][:see].T * D ** -0.5 / 30.0)
                    p = torch.softmax(y, -1)
                    m["w"][:see] += p.sum(0)
                    ref, A = p @ m["v"][:see], p @ m["v"][:see].abs()
                    err = (got[row + i, h * G:(h + 1) * G] - ref).abs()
                    assert bool((err <= (2.0 ** -10) * A + HALF_STEP[torch.float16] * ref.abs() + 2.0 ** -24).all()), (s, b, h)
                if L > trigger:
                    cuts += 1
                    # (weights of keys that are kept or not lie apart by more than the kernels' rounding, or the test's data is changed)
                    mid = m["w"][first:L - recent]
                    at = torch.sort(mid, descending=True, stable=True).values
                    want = keep - first - recent
                    assert float(at[want - 1] - at[want]) > 1e-5 * float(at[want])
                    idx = torch.sort(torch.sort(mid, descending=True, stable=True).indices[:want]).values + first
                    idx = torch.cat([torch.arange(first), idx, torch.arange(L - recent, L)])
                    for name in ("k", "v", "w"):
                        m[name] = m[name][idx]
            row += c
        assert lens.tolist() == [model[b][0]["w"].numel() for b in range(B)]
        held = sum(-(-x // bs) for x in lens.tolist())
        assert int(count.item()) == n - held
    assert cuts > 6
    live = torch.cat([table[b, :-(-int(lens[b]) // bs)] for b in range(B)]).tolist()
    assert sorted(live + free[:int(count.item())].tolist()) == list(range(n))  # no block lost, none twice
    for b in range(B):
        j = torch.arange(int(lens[b]))
        for h in range(Hkv):
            w = weights[table[b].long().cpu()[j // bs].cuda(), h, (j % bs).cuda()].double().cpu()
            assert bool(((w - model[b][h]["w"]).abs() <= 2.0 ** -10 * model[b][h]["w"] + 1e-6).all())
