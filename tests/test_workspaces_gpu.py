"""Calls without a workspace of their own: two threads on one stream, and
captures made through a stream handle."""
import threading

import pytest
import torch

from paged_split_decode_gb300 import binding, inputs

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def pd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_split_decode_gb300 as pd
    pd.load()
    return pd


def prepared(kind, seed):
    """A call whose units are split and joined by a second launch."""
    w = inputs.make_workload(B=24, Hq=24, Hkv=4, D=256, seq_lens=[2048 + 16 * (i % 5) for i in range(24)], kv="f16",
                             seed=seed, scale=1 / 16)
    args = dict(q=w.q.to(DEV), k_cache=w.k_cache.to(DEV), v_cache=w.v_cache.to(DEV), block_table=w.block_table.to(DEV),
                seq_lens=w.seq_lens.to(DEV), scale=w.scale, out=torch.empty_like(w.q, device=DEV))
    if kind == "diff":
        args["lam"] = torch.full((24,), 0.5, device=DEV)
    return args


@pytest.mark.parametrize("kinds", (("plain", "plain"), ("diff", "diff"), ("plain", "diff")))
def test_two_threads_on_one_stream(pd, kinds):
    """Each thread's results are those of the call alone, bit for bit. (The launch queue
    fills, so that both threads stand inside their calls.)"""
    calls = {"plain": pd.decode_paged, "diff": pd.decode_paged_diff}
    args = [prepared(k, 11 + i) for i, k in enumerate(kinds)]
    want = []
    for k, a in zip(kinds, args):
        want.append(calls[k](**a).clone())
    torch.cuda.synchronize()
    bad = [torch.zeros((), dtype=torch.int64, device=DEV) for _ in kinds]
    failed = []

    def work(i):
        try:
            for _ in range(1500):
                calls[kinds[i]](**args[i])
                bad[i].add_((args[i]["out"] != want[i]).any())
        except BaseException as e:  # noqa: BLE001 - shown below
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    assert [int(b) for b in bad] == [0, 0]


def test_a_capture_through_a_stream_handle_has_its_own_workspace(pd):
    """The captured stream is the call's, not the current one: the graph's
    workspace is not the one that eager calls of that stream use."""
    s, other = torch.cuda.Stream(), torch.cuda.Stream()
    args = prepared("diff", 5)
    torch.cuda.synchronize()
    pd.decode_paged_diff(**args, stream=s.cuda_stream)  # the stream's eager workspace
    torch.cuda.synchronize()
    want = args["out"].clone()
    eager = binding._workspaces[("cuda", 0, s.cuda_stream)]
    seen = []
    keep = binding._diff_workspace

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        with torch.cuda.stream(other):
            seen.append(keep(1 << 16, 0, s.cuda_stream))
            pd.decode_paged_diff(**args, stream=s.cuda_stream)
        seen.append(keep(1 << 16, 0, None))
    assert all(x.data_ptr() != eager.data_ptr() for x in seen)
    assert keep(1 << 16, 0, s.cuda_stream).data_ptr() == eager.data_ptr()
    args["out"].zero_()
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(args["out"], want)
