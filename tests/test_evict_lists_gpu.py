"""Evictions queued one behind another through one workspace: each reads the lists of its own selection and the weights and
tables that the call before it left, whatever lay at the same addresses before."""
import pytest
import torch

from test_evict_gpu import Pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv,D,Hkv", [("f16", 128, 2), ("fp4", 128, 4), ("int8", 256, 1)])
def test_queued_calls_share_a_workspace(kv, D, Hkv):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_split_decode_gb300 as pd
    pd.load()
    cuts = [(300, dict(first=3, recent=40)), (170, dict(recent=20)), (169, dict(first=8)), (64, dict(trigger=100, first=1, recent=9)), (1, {})]
    pools = [Pool(kv, 4, Hkv, D, 16, [900 - 31 * s, 310, 0, 41 + 13 * s], seed=40 + s, zeros=0.1) for s in range(3)]
    wants = []
    for p in pools:  # every cut of every pool, on the host
        data, w, lens = p.data, p.w, p.lens
        for keep, kw in cuts:
            q = Pool.__new__(Pool)
            q.__dict__ = dict(p.__dict__, data=data, w=w, lens=lens)
            data, w, lens = q.expect(keep, **kw)
        wants.append((data, w, lens))
    gpu = []
    for p in pools:
        t = [p.view(i, d) for i, d in enumerate(p.data)]
        sf = dict(k_block_scale=t[2], v_block_scale=t[3]) if kv == "fp4" else {}
        gpu.append((t, p.w.cuda(), p.table.cuda(), p.lens.cuda(), sf))
    ws = torch.full((1 << 20,), 0x7F, dtype=torch.uint8, device="cuda")
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    start = [[x.clone() for x in (*t, w, lens)] for t, w, _, lens, _ in gpu]

    def calls():
        for keep, kw in cuts:
            for t, w, table, lens, sf in gpu:
                pd.evict_kv_cache(t[0], t[1], w, table, lens, keep, workspace=ws, error_flag=flag, **sf, **kw)

    def check():
        torch.cuda.synchronize()
        assert int(flag.item()) == 0
        for p, want, (t, w, _, lens, _) in zip(pools, wants, gpu):
            p.gpu, p.gw = t, w
            p.check(want)
            assert torch.equal(lens.cpu(), want[2])

    calls()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for _ in range(3):
        for (t, w, _, lens, _), saved in zip(gpu, start):
            for x, s in zip((*t, w, lens), saved):
                x.copy_(s)
        graph.replay()
        check()
