"""Host-side checks of the differential decode, the block tables and the
root-mean-square norm that need no GPU: plans, and the refusals made before
anything is launched."""
import ctypes

import pytest
import torch

import paged_split_decode_gb300 as pd
from paged_split_decode_gb300 import binding, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def _dims(**kw):
    base = dict(B=32, Hq=24, Hkv=4, D=256, block_size=16, num_blocks=10000, max_blocks_per_seq=256)
    base.update(kw)
    return binding.make_dims(**base)


def test_diff_workspace_holds_two_maps(lib):
    up = lambda x: (x + 255) // 256 * 256
    # head-group tiles of four KV heads, 8 padded rows per map: 4 x 2 x 8 rows per slot
    assert binding.diff_workspace_bytes(_dims(), 1, 0, sm_count=152) == up(304 * 64 * 2 * 4) + 304 * 64 * 256 * 4
    assert binding.diff_workspace_bytes(_dims(), 1, 1, sm_count=152) == 0
    assert binding.diff_workspace_bytes(_dims(), 1, 3, sm_count=152) == up(96 * 64 * 2 * 4) + 96 * 64 * 256 * 4


@pytest.mark.parametrize("kw,qlen", [
    (dict(D=64), 1), (dict(block_size=8), 1), (dict(Hq=24, Hkv=5), 1), (dict(Hq=40, Hkv=1), 1), (dict(), 9), (dict(), 6)])
def test_diff_unsupported_shapes(lib, kw, qlen):
    assert binding.diff_workspace_bytes(_dims(**kw), qlen, 0, sm_count=152) == 0


def _diff(lib, dims, q=16, k=16, v=16, bt=16, sl=16, qs=None, T=32, lam=16, out=16, qlen=1, splits=1, norm=None, f32=0,
          eps=1e-5, gain=1.0, scale=0.1):
    return lib.decode_paged_diff(q, k, v, bt, sl, qs, T, lam, scale, 0, qlen, splits, norm, f32, eps, gain, out,
                                 ctypes.byref(dims), None, 0, None, None)


def test_diff_refusals(lib):
    d = _dims()
    assert _diff(lib, _dims(D=64)) == 4
    assert _diff(lib, _dims(Hkv=5)) == 2
    bad = _dims()
    bad.kv_dtype = 9
    assert _diff(lib, bad) == 3
    for name in ("q", "k", "v", "bt", "sl", "out"):
        assert _diff(lib, d, **{name: None}) == 1
    assert _diff(lib, d, q=0x1008) == 5
    assert _diff(lib, d, splits=-1) == 2
    assert _diff(lib, d, qlen=0) == 2
    assert _diff(lib, d, scale=float("nan")) == 2
    assert _diff(lib, d, norm=16, eps=-1.0) == 2
    assert _diff(lib, d, norm=16, eps=float("nan")) == 2
    assert _diff(lib, d, norm=16, gain=float("inf")) == 2
    assert _diff(lib, d, qs=16, T=-1) == 2
    assert _diff(lib, d, lam=None) == 1
    assert _diff(lib, d, lam=18) == 5
    assert _diff(lib, d, norm=17) == 5
    assert _diff(lib, d, norm=18, f32=1) == 5
    assert _diff(lib, _dims(B=0)) == 0           # nothing to do
    assert _diff(lib, d, qs=16, T=0) == 0
    assert lib.decode_paged_diff(*([16] * 5), None, 1, 16, 0.1, 0, 1, 1, None, 0, 0.0, 1.0, 16, None, None, 0, None,
                                 None) == 1


def _build(lib, d, ctx=16, query=16, T=4, table=16, free=16, count=16, count_out=16, seq=16, start=16, slots=16, pos=16):
    return lib.build_block_tables(ctx, query, T, table, free, count, count_out, seq, start, slots, pos,
                                  ctypes.byref(d), None, None)


def _release(lib, d, table=16, lens=16, released=16, free=16, count=16, count_out=16, lens_out=16):
    return lib.release_blocks(table, lens, released, free, count, count_out, lens_out, ctypes.byref(d), None, None)


def test_block_table_refusals(lib):
    d = _dims()
    for name in ("ctx", "query", "table", "free", "count", "count_out", "seq", "start", "slots"):
        assert _build(lib, d, **{name: None}) == 1, name
        assert _build(lib, d, **{name: 0x1002}) == 5, name
    assert _build(lib, d, pos=0x1002) == 5
    assert _build(lib, d, slots=0x1004) == 5     # 8-byte entries
    assert _build(lib, d, T=-1) == 2
    for kw, st in ((dict(B=-1), 2), (dict(block_size=0), 2), (dict(num_blocks=-1), 2), (dict(max_blocks_per_seq=-1), 2),
                   (dict(B=16385), 4), (dict(max_blocks_per_seq=1 << 27), 4)):
        assert _build(lib, _dims(**kw)) == st, kw
        assert _release(lib, _dims(**kw)) == st, kw
    for name in ("table", "lens", "released", "free", "count", "count_out", "lens_out"):
        assert _release(lib, d, **{name: None}) == 1, name
        if name != "released":
            assert _release(lib, d, **{name: 0x1002}) == 5, name
    assert lib.build_block_tables(*([16] * 2), 4, *([16] * 8), None, None, None) == 1
    assert lib.release_blocks(*([16] * 7), None, None, None) == 1


def _norm(lib, rows=4, N=256, norm=256, scale=256, bf16=0, f32=0, kind=0, x=16, w=16, out=16, out_scale=16, res=None,
          res_out=None, eps=1e-5, gain=1.0):
    d = binding.PdNormDims(rows, N, norm, scale, bf16, f32, kind)
    return lib.rms_norm(x, res, w, eps, gain, res_out, out, out_scale, ctypes.byref(d), None)


def test_rms_norm_refusals(lib):
    for kw in (dict(rows=-1), dict(N=0), dict(norm=0), dict(norm=100), dict(kind=1, scale=0), dict(kind=2, scale=100),
               dict(eps=-1.0), dict(eps=float("inf")), dict(gain=float("nan"))):
        assert _norm(lib, **kw) == 2, kw
    assert _norm(lib, kind=3) == 3
    assert _norm(lib, N=32769, norm=32769) == 4
    for kw in (dict(x=None), dict(w=None), dict(out=None), dict(kind=1, out_scale=None)):
        assert _norm(lib, **kw) == 1, kw
    for kw in (dict(x=17), dict(w=18, f32=1), dict(out=17), dict(res=17), dict(res_out=17), dict(kind=1, out_scale=18)):
        assert _norm(lib, **kw) == 5, kw
    assert _norm(lib, rows=0) == 0
    assert lib.rms_norm(16, None, 16, 1e-5, 1.0, None, 16, None, None, None) == 1


def test_python_refusals():
    """What the binding refuses before it asks for a device."""
    h, i32, f32 = torch.float16, torch.int32, torch.float32
    x, w = torch.zeros(2, 64, dtype=h), torch.ones(64, dtype=h)
    with pytest.raises(TypeError):
        pd.rms_norm(x.float(), w.float())
    with pytest.raises(TypeError):
        pd.rms_norm(x, w, out_dtype=torch.bfloat16)
    for kw in (dict(norm_size=48), dict(norm_size=32), dict(scale_size=0), dict(residual=x[:1]), dict(residual_out=x[:1]),
               dict(out=torch.zeros(2, 32, dtype=h)), dict(out_scale=torch.zeros(2, 1)),
               dict(out_dtype=torch.int8, out_scale=torch.zeros(3))):
        with pytest.raises(ValueError):
            pd.rms_norm(x, w, **kw)
    with pytest.raises(TypeError):
        pd.rms_norm(x, w)  # not on a GPU
    table, lens = torch.zeros(2, 3, dtype=i32), torch.zeros(2, dtype=i32)
    free, count = torch.zeros(6, dtype=i32), torch.zeros(1, dtype=i32)
    for args, kw in (((lens[:1], lens, table, free, count, 16, 2), {}), ((lens, lens, table, free, count, 16), {}),
                     ((lens, lens, table[0], free, count, 16, 2), {}), ((lens, lens, table, free, lens, 16, 2), {}),
                     ((lens, lens, table, free, count, 16, 2), dict(seq_lens=free)),
                     ((lens, lens, table, free, count, 16, 2), dict(query_start_loc=lens)),
                     ((lens, lens, table, free, count, 16, 2), dict(positions=free)),
                     ((lens, lens, table, free, count, 16, 2), dict(slot_mapping=torch.zeros(3, dtype=torch.int64)))):
        with pytest.raises(ValueError):
            pd.build_block_tables(*args, **kw)
    with pytest.raises(ValueError):
        pd.release_blocks(table, lens, lens[:1].bool(), free, count, 16)
    with pytest.raises(ValueError):
        pd.release_blocks(table, lens, lens.bool(), free, count, 16, seq_lens_out=free)
    q, c = torch.zeros(2, 8, 128, dtype=h), torch.zeros(4, 16, 4, 128, dtype=h)
    lam = torch.zeros(8, dtype=f32)
    for kw in (dict(qlen=2), dict(lam=lam[:4]), dict(norm_weight=w), dict(out=q[:1]), dict(query_start_loc=lens),
               dict(v_cache=c[:1])):
        a = dict(q=q, k_cache=c, v_cache=c, block_table=table, seq_lens=lens, lam=lam, scale=0.1)
        a.update(kw)
        with pytest.raises(ValueError):
            pd.decode_paged_diff(**a)


def test_the_library_is_built_without_the_python_headers(tmp_path, monkeypatch):
    """A compiled binding that does not build (no PyTorch or Python headers) is
    reported and leaves the library built; the calls that need it say why."""
    src = tmp_path / "one.cu"
    src.write_text('extern "C" __attribute__((visibility("default"))) int answer() { return 42; }\n')
    for name, path in (("BUILD", "_build"), ("LIB", "lib.so"), ("BIND", "_bind.so"), ("BIND_FOR", "bind.for")):
        monkeypatch.setattr(build, name, str(tmp_path / path))
    monkeypatch.setattr(build, "sources", lambda: [str(src)])
    command = build._bind_command
    monkeypatch.setattr(build, "_bind_command", lambda out: ["false"])
    with pytest.warns(RuntimeWarning, match="bind.cpp"):
        assert build.build() == str(tmp_path / "lib.so")
    assert ctypes.CDLL(build.LIB).answer() == 42 and not (tmp_path / "_bind.so").exists()
    # the next build does not compile the library again, and builds the binding once that works
    before = (tmp_path / "lib.so").stat().st_mtime_ns
    monkeypatch.setattr(build, "_bind_command", lambda out: ["touch", out])
    assert build.build() == build.LIB
    assert (tmp_path / "lib.so").stat().st_mtime_ns == before and (tmp_path / "_bind.so").exists()
    # a binding left from other sources does not stand in for one that fails
    (tmp_path / "bind.for").write_text("another PyTorch")
    monkeypatch.setattr(build, "_bind_command", lambda out: ["false"])
    with pytest.warns(RuntimeWarning):
        build.build()
    assert not (tmp_path / "_bind.so").exists()
    monkeypatch.setattr(build, "_bind_command", command)


def test_rms_norm_refuses_overlaps(lib):
    """Outputs over inputs or each other; what the header allows is tested where it can run."""
    m = 1 << 20  # 4 x 256 fp16 values are 2 KiB, as codes 1 KiB; 4 scales 16 bytes
    kw = dict(x=m, w=2 * m, out=3 * m, out_scale=4 * m)
    for bad in (dict(res=5 * m, res_out=3 * m), dict(res=5 * m, res_out=3 * m + 2046), dict(res_out=m + 2), dict(out=m + 16),
                dict(out=2 * m), dict(out=2 * m - 2046), dict(res=5 * m, res_out=5 * m, out=5 * m), dict(res=5 * m, out=5 * m + 64),
                dict(res=m + 1024, res_out=m), dict(kind=1, out=m), dict(kind=2, res=5 * m, out=5 * m + 2047),
                dict(kind=1, out_scale=m + 2044), dict(kind=1, out_scale=3 * m + 1020), dict(kind=2, out_scale=2 * m),
                dict(kind=2, res=5 * m, out_scale=5 * m), dict(kind=1, res_out=4 * m - 2044)):
        assert _norm(lib, **{**kw, **bad}) == 2, bad
