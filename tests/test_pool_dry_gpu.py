"""Steps that refuse sequences, in the in-place form: an empty free list, a full
table row and a token buffer that is too short are ordinary events of a serving
loop, and none of them may lose a sequence or its blocks."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def pd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_split_decode_gb300 as pd
    pd.load()
    return pd


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("captured", (False, True))
@pytest.mark.parametrize("B,cols,nb,T", [(4, 6, 7, 64), (4, 3, 40, 64), (5, 6, 9, 11), (300, 4, 500, 700)])
def test_refused_sequences_keep_their_blocks(pd, B, cols, nb, T, captured):
    """A loop over a pool that runs dry (first case), over rows that fill up
    (second), over a short token buffer (third) and over all of them (last):
    refused sequences keep their length, are served again as soon as there is
    room, and every block comes back at the end."""
    bs, rng = 16, np.random.RandomState(B + cols)
    lens, query, done = ints(*[0] * B), ints(*[0] * B), torch.zeros(B, dtype=torch.bool, device=DEV)
    table = torch.full((B, cols), -1, dtype=torch.int32, device=DEV)
    free, count, flag = torch.randperm(nb, device=DEV).int(), ints(nb), ints(0)
    start, slots = ints(*[0] * (B + 1)), torch.zeros(T, dtype=torch.int64, device=DEV)

    def step():
        pd.build_block_tables(lens, query, table, free, count, bs, seq_lens=lens, query_start_loc=start,
                              slot_mapping=slots, error_flag=flag)
        pd.release_blocks(table, lens, done, free, count, bs, error_flag=flag)

    graph = None
    if captured:
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    host, refusals = [0] * B, 0
    for i in range(60):
        q = rng.randint(0, 6, B)
        d = rng.rand(B) < (0.05 if i < 40 else 0.3)
        query.copy_(torch.from_numpy(q.astype(np.int32)))
        done.copy_(torch.from_numpy(d))
        flag.zero_()
        (graph.replay if graph else step)()
        torch.cuda.synchronize()
        left = nb - sum(-(-n // bs) for n in host)
        off, at, full, bits = 0, 0, False, 0
        want = np.full(T, -2, np.int64)
        for b in range(B):
            n = int(q[b])
            served = True
            if host[b] + n > cols * bs:
                served, bits, need = False, bits | pd.DEVERR_SEQ_LEN, 0
            else:
                need = -(-(host[b] + n) // bs) - -(-host[b] // bs)
            if n and at + n > T:
                served, bits = False, bits | pd.DEVERR_QUERY_START
            if need and (full or off + need > left):
                served, bits, full = False, bits | pd.DEVERR_FREE_LIST, True
            off += need
            if not served:
                refusals += 1
                want[at:at + n] = -1
            elif n:
                host[b] += n
            at += n
        want[at:] = -1
        got = slots.cpu().numpy()
        assert np.array_equal(got == -1, want == -1)
        assert int(flag.item()) == bits
        for b in np.nonzero(d)[0]:
            host[b] = 0
        assert lens.tolist() == host
        used = sum(-(-n // bs) for n in host)
        assert int(count.item()) == nb - used
        owned = [int(table[b, x]) for b in range(B) for x in range(-(-host[b] // bs))] if B < 10 or i % 20 == 19 else None
        if owned is not None:
            assert sorted(owned + free[:nb - used].tolist()) == list(range(nb))
    assert refusals > 5
    done.fill_(True)
    pd.release_blocks(table, lens, done, free, count, bs)
    torch.cuda.synchronize()
    assert int(count.item()) == nb and sorted(free.tolist()) == list(range(nb))


def test_bad_lengths_stay_in_place(pd):
    """Nothing of a refused entry is lost or made up: a negative length and one past the row stay."""
    lens = ints(-3, 5, 99, 7)
    table = torch.tensor([[9, 9], [0, 9], [9, 9], [1, 9]], dtype=torch.int32, device=DEV)
    free, count, flag = ints(2, 3), ints(2), ints(0)
    seq, start, slots, pos = pd.build_block_tables(lens, ints(1, 1, 1, -1), table, free, count, 16, 4, seq_lens=lens,
                                                   error_flag=flag)
    assert seq.data_ptr() == lens.data_ptr()
    assert lens.tolist() == [-3, 6, 99, 7] and slots.tolist() == [-1, 5, -1, -1] and int(count.item()) == 2
    assert int(flag.item()) == pd.DEVERR_SEQ_LEN and start.tolist() == [0, 1, 2, 3, 3]


def test_a_refused_row_decodes_its_old_keys(pd):
    """The decode behind a refusal reads the sequence's own keys only and raises
    nothing; the served rows are what they are without the refused one."""
    dt, bs = torch.float16, 16
    caches = [torch.randn(3, bs, 4, 128, device=DEV).to(dt) for _ in range(2)]
    table = torch.tensor([[0, -1], [1, -1], [2, -1], [-1, -1]], dtype=torch.int32, device=DEV)
    lens, flag = ints(5, 16, 7, 0), ints(0)
    query = ints(1, 2, 1, 3)
    free, count = ints(-1, -1, -1), ints(0)
    q, lam = torch.randn(7, 8, 128, device=DEV).to(dt), torch.full((8,), 0.5, device=DEV)
    seq, start, slots, _ = pd.build_block_tables(lens, query, table, free, count, bs, 7, seq_lens=lens, error_flag=flag)
    assert int(flag.item()) == pd.DEVERR_FREE_LIST and lens.tolist() == [6, 16, 8, 0]
    assert slots.tolist() == [5, -1, -1, 39, -1, -1, -1]
    flag.zero_()
    out = pd.decode_paged_diff(q, *caches, table, lens, lam, 0.125, qlen=3, query_start_loc=start, error_flag=flag)
    alone = pd.decode_paged_diff(q[1:3].contiguous(), *caches, table[1:2].contiguous(), ints(16), lam, 0.125, qlen=2)
    torch.cuda.synchronize()
    assert int(flag.item()) == 0 and (out[4:] == 0).all()
    assert torch.allclose(out[1:3].float(), alone.float(), atol=2e-3, rtol=0)
