"""A row's output and log-sum-exp depend on its own query alone: no bit changes with the other rows of
its tile, however far their scores lie."""
import pytest
import torch

from ref_scored import Work

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("S", (0, 1, 3))
@pytest.mark.parametrize("qlen", (1, 3))
@pytest.mark.parametrize("kv,q", [("f16", "f16"), ("bf16", "bf16"), ("fp8", "f16"), ("fp8", "bf16"), ("int8", "f16"), ("int8", "bf16"),
                                  ("fp4", "f16"), ("fp4", "bf16")])
def test_rows_alone(kv, q, qlen, S):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_split_decode_gb300 as pd
    pd.load()
    for Hq, Hkv, D in ((24, 4, 256), (12, 2, 128)):
        w = Work(kv, Hq, Hkv, D, [500, 130, 700], qlen=qlen, q=q, seed=61, spread=2.0)
        want = w.run(pd, S)
        g = torch.Generator().manual_seed(62)
        keep = torch.rand(w.q.shape[:2], generator=g) < 0.4
        factor = torch.tensor([0.0, -1.0, 7.0, 0.1])[torch.randint(0, 4, keep.shape, generator=g)]
        w.q = torch.where(keep[..., None], w.q, (w.q.float() * factor[..., None]).to(w.qt))
        got = w.run(pd, S)
        assert torch.equal(got[0].cpu()[keep], want[0].cpu()[keep])
        assert torch.equal(got[1].cpu()[keep], want[1].cpu()[keep])
