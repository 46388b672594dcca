"""A serving loop as a program writes it: block tables and slot maps built on
the GPU, the writer, the differential decode with its head norm, the block's
norm with the residual and an 8-bit output, and the release of finished
sequences -- a prompt phase in the decode's token counts, then steps captured in
one CUDA graph, whose caches, tables and outputs are checked against a plain
host model of the whole loop in 64 bits."""
import numpy as np
import pytest
import torch

import ref_diff
from paged_split_decode_gb300 import inputs

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def pd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_split_decode_gb300 as pd
    pd.load()
    return pd


class Model:
    """The host's view: each sequence's keys, and what a decode of them gives."""

    def __init__(self, B, Hq, Hkv, D, kind, scale):
        self.B, self.Hq, self.Hkv, self.D, self.kind, self.scale = B, Hq, Hkv, D, kind, scale
        self.k = [[] for _ in range(B)]
        self.v = [[] for _ in range(B)]

    def decode(self, q, query, lam, weight):
        """(ref, bound) for q [sum query, Hq, D], the last query[b] keys being the tokens themselves."""
        lens = [len(k) for k in self.k]
        w = inputs.make_varlen_workload(B=self.B, qlens=query, Hq=self.Hq, Hkv=self.Hkv, D=self.D, seq_lens=lens,
                                        kv=self.kind, scale=self.scale)
        w.q = q
        for b in range(self.B):
            for j in range(lens[b]):
                blk = int(w.block_table[b, j // 16])
                w.k_cache[blk, j % 16], w.v_cache[blk, j % 16] = self.k[b][j], self.v[b][j]
        return ref_diff.reference(w, lam.double().numpy(), weight.double().numpy(), 1e-5, 0.6)


@pytest.mark.parametrize("kind", ("f16", "bf16"))
def test_a_serving_loop(pd, kind):
    B, Hq, Hkv, D, bs, cols, steps = 5, 8, 4, 128, 16, 8, 24
    dt = torch.bfloat16 if kind == "bf16" else torch.float16
    u = ref_diff.HALF_STEP[dt]
    g = torch.Generator().manual_seed(5)
    nb = 24
    caches = [torch.zeros(nb, bs, Hkv, D, dtype=dt, device=DEV) for _ in range(2)]
    free, count = torch.randperm(nb, generator=g).int().to(DEV), torch.tensor([nb], dtype=torch.int32, device=DEV)
    table = torch.full((B, cols), -1, dtype=torch.int32, device=DEV)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    lam = 0.2 + 0.6 * torch.rand(Hq, generator=g)
    weight = (1 + 0.1 * torch.randn(D, generator=g)).to(dt)
    wide = (1 + 0.1 * torch.randn(Hq * D, generator=g)).to(dt)
    lam_d, weight_d, wide_d = lam.to(DEV), weight.to(DEV), wide.to(DEV)
    model = Model(B, Hq, Hkv, D, kind, 0.125)
    T = 32  # token buffer: padded
    qlen = 8

    bufs = dict(query=torch.zeros(B, dtype=torch.int32, device=DEV), q=torch.zeros(T, Hq, D, dtype=dt, device=DEV),
                k=torch.zeros(T, Hkv, D, dtype=dt, device=DEV), v=torch.zeros(T, Hkv, D, dtype=dt, device=DEV),
                res=torch.zeros(T, Hq * D, dtype=dt, device=DEV))
    out = torch.zeros(T, Hq, D, dtype=dt, device=DEV)
    codes = torch.zeros(T, Hq * D, dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.zeros(T, Hq, dtype=torch.float32, device=DEV)
    start = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    slots = torch.zeros(T, dtype=torch.int64, device=DEV)
    pos = torch.zeros(T, dtype=torch.int32, device=DEV)
    held = torch.zeros(T, Hq * D, dtype=dt, device=DEV)

    def step():
        pd.build_block_tables(lens, bufs["query"], table, free, count, bs, seq_lens=lens, query_start_loc=start,
                              slot_mapping=slots, positions=pos, error_flag=flag)
        pd.write_kv_cache(bufs["k"], bufs["v"], slots, *caches, error_flag=flag)
        pd.decode_paged_diff(bufs["q"], *caches, table, lens, lam_d, 0.125, qlen=qlen, out=out, query_start_loc=start,
                             norm_weight=weight_d, norm_gain=0.6, error_flag=flag)
        pd.rms_norm(out.view(T, Hq * D), wide_d, residual=bufs["res"], residual_out=held, out=codes, out_scale=scales,
                    scale_size=D)

    graph = None
    for i in range(steps):
        query = [int(x) for x in torch.randint(0 if i else 1, 5, (B,), generator=g)]
        if i == 7:
            query[1] = 0
        n = sum(query)
        fresh = {name: torch.randn(n, *bufs[name].shape[1:], generator=g).to(dt) for name in ("q", "k", "v", "res")}
        bufs["query"].copy_(torch.tensor(query, dtype=torch.int32))
        for name, x in fresh.items():
            bufs[name][:n] = x.to(DEV)
        out.fill_(3.0)
        if graph is None and i == 2:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        if graph is None:
            step()
        else:
            graph.replay()
        torch.cuda.synchronize()
        at = 0
        for b in range(B):
            for _ in range(query[b]):
                assert int(pos[at]) == len(model.k[b])
                model.k[b].append(fresh["k"][at])
                model.v[b].append(fresh["v"][at])
                at += 1
        assert lens.tolist() == [len(k) for k in model.k]
        assert (slots[n:] == -1).all()
        ref, bound = model.decode(fresh["q"], query, lam, weight)
        got = out.float().cpu().double().numpy()
        assert np.all(np.abs(got[:n] - ref) <= bound)
        assert np.all(got[n:] == 3.0)  # the padded rows are left as they were
        # the norm, from the decode's own output: h = out + residual in fp32, then
        # 2^-4 of a code's half step, r = (N / 2 + 16) 2^-24 as for rms_norm alone
        h = got[:n].reshape(n, -1) + fresh["res"].double().numpy()
        y = h / np.sqrt(np.mean(h * h, -1, keepdims=True) + 1e-5) * wide.double().numpy()
        r = (Hq * D / 2 + 16) * 2.0 ** -24
        assert np.all(np.abs(held[:n].float().cpu().double().numpy() - h) <= (u + 2.0 ** -24) * np.abs(h) + 2.0 ** -25)
        s = scales[:n].double().cpu().numpy().repeat(D, 1)
        c = codes[:n].float().cpu().double().numpy()
        assert np.all(np.abs(c * s - y) <= (2.0 ** -4 + 2 * r) * np.abs(y) + 2.0 ** -10 * s * (1 + 2.0 ** -20))
        assert int(flag.item()) == 0
        # sequences that pass 96 keys end: their blocks go back, their rows start anew
        done = torch.tensor([len(k) > 96 or (i == 11 and b == 2) for b, k in enumerate(model.k)])
        pd.release_blocks(table, lens, done.to(DEV), free, count, bs, error_flag=flag)
        for b in range(B):
            if done[b]:
                model.k[b], model.v[b] = [], []
        used = sum(-(-len(k) // bs) for k in model.k)
        assert int(count.item()) == nb - used
        owned = [int(table[b, x]) for b in range(B) for x in range(-(-len(model.k[b]) // bs))]
        assert sorted(owned + free[:nb - used].tolist()) == list(range(nb))


def test_a_pool_that_runs_dry_zeroes_the_refused_row(pd):
    """A sequence that gets no block has length 0: its decode writes zeros, its
    tokens are not stored, the others are served."""
    dt, bs = torch.float16, 16
    caches = [torch.randn(3, bs, 4, 128, device=DEV).to(dt) for _ in range(2)]
    before = [c.clone() for c in caches]
    table = torch.tensor([[0, -1], [1, -1], [2, -1]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([5, 16, 7], dtype=torch.int32, device=DEV)
    free, count = torch.full((3,), -1, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    seq, start, slots, _ = pd.build_block_tables(lens, torch.ones_like(lens), table, free, count, bs, 3, error_flag=flag)
    assert int(flag.item()) == pd.DEVERR_FREE_LIST and seq.tolist() == [6, 0, 8] and slots.tolist() == [5, -1, 39]
    k = torch.randn(3, 4, 128, device=DEV).to(dt)
    pd.write_kv_cache(k, k, slots, *caches)
    out = pd.decode_paged_diff(torch.randn(3, 8, 128, device=DEV).to(dt), *caches, table, seq,
                               torch.full((8,), 0.5, device=DEV), 0.125, qlen=1, query_start_loc=start)
    torch.cuda.synchronize()
    assert (out[1] == 0).all() and (out[0] != 0).any() and (out[2] != 0).any()
    assert torch.equal(caches[0][1], before[0][1]) and torch.equal(caches[0][0, 5], k[0]) and torch.equal(caches[1][2, 7], k[2])
