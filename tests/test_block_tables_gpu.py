"""build_block_tables and release_blocks against plain Python, entry by entry
(whole numbers: equality), on sentinel-filled buffers so that stray writes
show."""
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


def ceil_div(a, b):
    return -(-a // b)


def ref_build(context, query, table, free, count, bs, T, num_blocks):
    """The step in plain Python: (seq_lens, starts, table, slots, positions, count, error bits)."""
    B, cols = table.shape
    table, bits = table.copy(), 0
    seq, starts = np.zeros(B, np.int32), np.zeros(B + 1, np.int32)
    slots, pos = np.full(T, -1, np.int64), np.zeros(T, np.int32)
    start, off, full, taken = 0, 0, False, 0
    for b in range(B):
        c, n = int(context[b]), int(query[b])
        starts[b] = min(start, 2 ** 31 - 1)
        end = start + max(n, 0)
        ok = True
        if c < 0 or n < 0 or c + n > cols * bs:
            bits, ok = bits | 2, False
            need = 0
        else:
            need = ceil_div(c + n, bs) - ceil_div(c, bs)
        if n > 0 and end > T:
            bits, ok = bits | 16, False
        if need > 0 and (full or off + need > count):
            bits, ok, full = bits | 32, False, True
        if ok:
            seq[b] = c + n
            held = ceil_div(c, bs)
            for i in range(need):
                table[b, held + i] = free[count - 1 - (off + i)]
                if not 0 <= table[b, held + i] < num_blocks:
                    bits |= 1
            if need:
                taken = off + need
            for i in range(n):
                p = c + i
                blk = int(table[b, p // bs])
                pos[start + i] = p
                if 0 <= blk < num_blocks:
                    slots[start + i] = blk * bs + p % bs
                else:
                    bits |= 1
        off += need
        start = end
    starts[B] = min(start, 2 ** 31 - 1)
    return seq, starts, table, slots, pos, count - taken, bits


def step_inputs(rng, B, cols, bs, spare, most_new, rest=0.2):
    """Random contexts and tables over one pool; the free blocks follow."""
    context = rng.randint(0, cols * bs + 1, B)
    context[rng.rand(B) < 0.2] = 0
    context[rng.rand(B) < 0.2] //= bs
    context = np.where(rng.rand(B) < 0.2, context // bs * bs, context)
    query = np.minimum(rng.randint(0, most_new + 1, B), cols * bs - context)
    query[rng.rand(B) < rest] = 0
    held = [ceil_div(int(c), bs) for c in context]
    num_blocks = B * cols + spare
    ids = rng.permutation(num_blocks).astype(np.int32)
    table = np.full((B, cols), -9, np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    free = np.concatenate([ids[at:], np.full(at, -7, np.int32)])
    return context.astype(np.int32), query.astype(np.int32), table, free, num_blocks - at, num_blocks


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def run_build(pd, context, query, table, free, count, bs, T, in_place=False, stream=None):
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    ctx, tab, cnt = dev(context), dev(table), dev(np.array([count], np.int32))
    out = torch.full((1,), -5, dtype=torch.int32, device=DEV)
    seq, starts, slots, pos = pd.build_block_tables(
        ctx, dev(query), tab, dev(free), cnt, bs, T, seq_lens=ctx if in_place else None,
        free_count_out=None if in_place else out, error_flag=flag, stream=stream)
    torch.cuda.synchronize()
    left = cnt if in_place else out
    return [x.cpu().numpy() for x in (seq, starts, tab, slots, pos)] + [int(left.item()), int(flag.item())]


def same(got, want):
    for name, a, b in zip(("seq_lens", "query_start_loc", "block_table", "slot_mapping", "positions"), got, want):
        bad = np.nonzero(a.reshape(-1) != b.reshape(-1))[0]
        assert bad.size == 0, f"{name}: {bad.size} differ, first at {bad[:4]}"
    assert got[5:] == [want[5], want[6]], "count left, error bits"


@pytest.mark.parametrize("in_place", (False, True))
@pytest.mark.parametrize("B,cols,bs,most,pad", [
    (1, 4, 16, 1, 0), (1, 1, 1, 1, 3), (3, 7, 16, 40, 5), (32, 256, 16, 1, 0), (33, 9, 48, 300, 64), (257, 20, 16, 90, 100),
    (1024, 6, 32, 3, 1), (1025, 5, 16, 60, 0), (5000, 3, 16, 2, 77), (40, 300, 16, 2000, 500), (16384, 2, 16, 1, 0)])
def test_build_matches_plain_python(pd, B, cols, bs, most, pad, in_place):
    rng = np.random.RandomState(B + cols)
    context, query, table, free, count, nb = step_inputs(rng, B, cols, bs, 3, most)
    T = int(query.sum()) + pad
    want = ref_build(context, query, table, free, count, bs, T, nb)
    assert want[6] == 0
    same(run_build(pd, context, query, table, free, count, bs, T, in_place), want)


def test_one_token_each_needs_no_slot_map_size(pd):
    rng = np.random.RandomState(3)
    context, query, table, free, count, nb = step_inputs(rng, 8, 5, 16, 0, 1)
    slots = torch.empty(8, dtype=torch.int64, device=DEV)
    out = pd.build_block_tables(dev(context), dev(query), dev(table), dev(free), dev(np.array([count], np.int32)), 16,
                                slot_mapping=slots)
    assert out[2] is slots
    want = ref_build(context, query, table, free, count, 16, 8, nb)
    assert np.array_equal(slots.cpu().numpy(), want[3])


@pytest.mark.parametrize("left", (0, 1, 7, 20))
def test_too_few_free_blocks(pd, left):
    """Sequences are served in order until the list runs out; those that need
    no block still are."""
    rng = np.random.RandomState(left)
    context, query, table, free, count, nb = step_inputs(rng, 40, 6, 16, 0, 50)
    free, count = free[count - left:], left  # the list's top `left` blocks
    free = np.concatenate([free, np.full(nb - free.size, -7, np.int32)])
    T = int(query.sum())
    want = ref_build(context, query, table, free, count, 16, T, nb)
    assert want[6] == 32
    same(run_build(pd, context, query, table, free, count, 16, T), want)


def test_bad_lengths_short_maps_and_bad_ids(pd):
    rng = np.random.RandomState(9)
    context, query, table, free, count, nb = step_inputs(rng, 30, 6, 16, 0, 30, rest=0.0)
    context[3], query[8], context[11], query[20] = -1, -4, 97, 2 ** 31 - 1
    for cut in (0, 37):  # the token buffer too short for the last sequences
        T = int(np.maximum(query[:20], 0).sum()) + 40 - cut
        want = ref_build(context, query, table, free, count, 16, T, nb)
        assert want[6] & 18 == 18
        same(run_build(pd, context, query, table, free, count, 16, T), want)
    context, query, table, free, count, nb = step_inputs(rng, 30, 6, 16, 0, 30, rest=0.0)
    free[count - 2] = nb
    part = next(b for b in range(30) if context[b] % 16 and query[b])
    table[part, context[part] // 16] = -1
    T = int(query.sum())
    want = ref_build(context, query, table, free, count, 16, T, nb)
    assert want[6] == 1
    same(run_build(pd, context, query, table, free, count, 16, T), want)


@pytest.mark.parametrize("count", (-1, 200))
def test_a_bad_count(pd, count):
    context, query = np.zeros(2, np.int32), np.ones(2, np.int32)
    table, free = np.full((2, 2), -9, np.int32), np.arange(4, dtype=np.int32)
    got = run_build(pd, context, query, table, free, count, 16, 2)
    want = ref_build(context, query, table, free, 0 if count < 0 else 4, 16, 2, 4)
    same(got, list(want[:6]) + [32])


def test_empty_batches(pd):
    none = np.zeros(0, np.int32)
    got = run_build(pd, none, none, np.zeros((0, 4), np.int32), np.arange(4, dtype=np.int32), 4, 16, 5)
    assert got[1].tolist() == [0] and got[3].tolist() == [-1] * 5 and got[5:] == [4, 0]
    got = run_build(pd, np.array([5], np.int32), np.array([0], np.int32), np.full((1, 1), 2, np.int32),
                    np.arange(4, dtype=np.int32), 2, 16, 0)
    assert got[0].tolist() == [5] and got[5:] == [2, 0]


# ---------------------------------------------------------------------------
def ref_release(table, lens, released, free, count, bs, num_blocks):
    free, lens, bits = free.copy(), lens.copy(), 0
    at, full = count, False
    off = 0
    for b in range(len(lens)):
        if not released[b]:
            continue
        L = int(lens[b])
        if L < 0 or L > table.shape[1] * bs:
            bits |= 2
            continue
        n = ceil_div(L, bs)
        if n and count + off + n > num_blocks:
            bits |= 32
        elif n:
            for i in range(n):
                blk = int(table[b, i])
                if not 0 <= blk < num_blocks:
                    bits, blk = bits | 1, -1
                free[at + i] = blk
            at += n
            lens[b] = 0
        off += n
    return lens, free, at, bits


def run_release(pd, table, lens, released, free, count, bs, in_place):
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    ln, fr, cnt = dev(lens), dev(free), dev(np.array([count], np.int32))
    lo, co = torch.full_like(ln, -3), torch.full_like(cnt, -3)
    got = pd.release_blocks(dev(table), ln, dev(released), fr, cnt, bs, seq_lens_out=None if in_place else lo,
                            free_count_out=None if in_place else co, error_flag=flag)
    torch.cuda.synchronize()
    return got.cpu().numpy(), fr.cpu().numpy(), int((cnt if in_place else co).item()), int(flag.item())


@pytest.mark.parametrize("in_place", (False, True))
@pytest.mark.parametrize("B,cols,bs,share", [(1, 1, 16, 1.0), (5, 7, 16, 0.5), (32, 256, 16, 0.1), (300, 40, 48, 0.5),
                                             (1500, 9, 16, 0.9), (16384, 2, 16, 0.5), (7, 3, 16, 0.0)])
def test_release_matches_plain_python(pd, B, cols, bs, share, in_place):
    rng = np.random.RandomState(B + cols)
    context, _, table, free, count, nb = step_inputs(rng, B, cols, bs, 3, 1)
    released = rng.rand(B) < share
    want = ref_release(table, context, released, free, count, bs, nb)
    assert want[3] == 0
    got = run_release(pd, table, context, released, free, count, bs, in_place)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1]) and got[2:] == want[2:]


def test_release_refuses_what_does_not_fit(pd):
    rng = np.random.RandomState(5)
    context, _, table, free, count, nb = step_inputs(rng, 20, 6, 16, 0, 1)
    context[4], context[6] = -2, 97
    released = np.ones(20, bool)
    count = nb - 9  # as if those blocks were free already
    want = ref_release(table, context, released, free, count, 16, nb)
    assert want[3] & 34 == 34
    table2 = table.copy()
    first = next(b for b in range(20) if 0 < context[b] <= 96)
    table2[first, 0] = nb
    got = run_release(pd, table, context, released, free, count, 16, False)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1]) and got[2:] == want[2:]
    want = ref_release(table2, context, released, free, 0, 16, nb)
    assert want[3] & 1
    got = run_release(pd, table2, context, released, free, 0, 16, True)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1]) and got[2:] == want[2:]


def test_steps_in_a_captured_graph(pd):
    """One step captured and replayed: lengths and the count advance in place,
    every step's blocks are distinct, and a release gives them back."""
    B, cols, bs, steps = 6, 4, 16, 40
    lens = torch.tensor([0, 3, 16, 15, 1, 20], dtype=torch.int32, device=DEV)
    nb = B * cols
    free = torch.arange(nb, dtype=torch.int32, device=DEV)
    count = torch.tensor([nb], dtype=torch.int32, device=DEV)
    table = torch.full((B, cols), -1, dtype=torch.int32, device=DEV)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    zero, one = torch.zeros_like(lens), torch.ones_like(lens)
    start = lens.clone()
    # the prompts, then one token a step
    pd.build_block_tables(zero, lens, table, free, count, bs, 64, seq_lens=lens, error_flag=flag)
    starts, slots, pos = (torch.empty(n, dtype=t, device=DEV) for n, t in ((B + 1, torch.int32), (B, torch.int64), (B, torch.int32)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pd.build_block_tables(lens, one, table, free, count, bs, seq_lens=lens, query_start_loc=starts,
                              slot_mapping=slots, positions=pos, error_flag=flag)
    seen = [set() for _ in range(B)]
    for i in range(steps):
        g.replay()
        torch.cuda.synchronize()
        want = start.cpu() + i
        assert torch.equal(pos.cpu(), want) and torch.equal(lens.cpu(), want + 1)
        for b, s in enumerate(slots.tolist()):
            assert s == int(table[b, int(want[b]) // bs]) * bs + int(want[b]) % bs
            seen[b].add(s // bs)
    assert int(flag.item()) == 0
    held = [ceil_div(int(x), bs) for x in lens.tolist()]
    used = [int(table[b, i]) for b in range(B) for i in range(held[b])]
    assert len(set(used)) == len(used) and int(count.item()) == nb - len(used)
    pd.release_blocks(table, lens, torch.ones(B, dtype=torch.bool, device=DEV), free, count, bs, error_flag=flag)
    torch.cuda.synchronize()
    assert int(count.item()) == nb and sorted(free.tolist()) == list(range(nb)) and lens.tolist() == [0] * B
