"""Host-side validation of the dense-cache entry points (nothing here launches a kernel:
every call is refused, or has nothing to do)."""
import ctypes

import pytest

FAKE = 1 << 20                      # an aligned address that no refused call follows


@pytest.fixture(scope="module")
def csa2():
    from __graft_entry__ import build
    build()
    from fp4_kv_cache_04_b200 import csa2 as c
    return c


def _rope(csa2, **kw):
    a = csa2.RopeArgs(rows=4, heads=16, dim=512, rope_dim=64, in_type=0, out_type=0, flags=1, x_row_stride=8192,
                      x_head_stride=512, out_row_stride=8192, out_head_stride=512, x=FAKE, out=2 * FAKE, pos=FAKE,
                      inv_freq=FAKE, weight=FAKE, eps=1e-6)
    for k, v in kw.items():
        setattr(a, k, v)
    return csa2.lib().csa2_norm_rope(ctypes.byref(a), None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 1), (dict(heads=0), 1), (dict(heads=1025), 2), (dict(dim=4), 1), (dict(dim=12), 1),
    (dict(dim=1032, x_head_stride=1032, out_head_stride=1032, x_row_stride=16512, out_row_stride=16512), 2),
    (dict(rope_dim=3), 1), (dict(rope_dim=514), 1), (dict(rope_dim=-2), 1), (dict(in_type=3), 1), (dict(out_type=-1), 1),
    (dict(flags=8), 1), (dict(flags=0), 1),                       # a weight without the norm
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(reserved0=1), 1), (dict(x=None), 1), (dict(out=None), 1),
    (dict(pos=None), 1), (dict(inv_freq=None), 1), (dict(x=FAKE + 8), 1), (dict(out=FAKE + 2), 1),
    (dict(weight=FAKE + 4), 1), (dict(x_row_stride=8196), 1), (dict(x_head_stride=-512), 1),
    (dict(out_head_stride=504), 1), (dict(out_row_stride=8184), 1), (dict(out_row_stride=0), 1),
    (dict(out=FAKE, out_type=2), 1), (dict(out=FAKE, out_row_stride=8200), 1),
])
def test_norm_rope_refuses(csa2, kw, status):
    assert _rope(csa2, **kw) == status


def test_nothing_to_do_is_ok(csa2):
    assert _rope(csa2, rows=0, x=None, out=None) == 0
    assert _append(csa2, n=0, latent=None) == 0
    assert csa2.lib().csa2_dequantize_kv(None, None, 0, None, 0, None, None) == 0
    assert csa2.lib().csa2_norm_rope(None, None) == 1
    assert csa2.lib().csa2_append_rope(None, None) == 1
    assert csa2.lib().csa2_attend_cache(None, None) == 1
    assert csa2.lib().csa2_cache_workspace_size(None) == 0


def _append(csa2, **kw):
    a = csa2.AppendArgs(n=4, batch=4, rope_dim=64, idx_rope_dim=64, in_type=0, flags=1, eps=1e-6, latent_stride=512,
                        idx_stride=64, total_rows=100, latent=FAKE, idx_proj=FAKE, seq=FAKE, pos=FAKE, kv_offsets=FAKE,
                        inv_freq=FAKE, idx_inv_freq=FAKE, weight=FAKE, codes=FAKE, scales=FAKE, idx_k=FAKE, idx_kscale=FAKE)
    for k, v in kw.items():
        setattr(a, k, v)
    return csa2.lib().csa2_append_rope(ctypes.byref(a), None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), 1), (dict(batch=0), 1), (dict(rope_dim=514), 1), (dict(rope_dim=1), 1), (dict(idx_rope_dim=66), 1),
    (dict(in_type=7), 1), (dict(flags=2), 1), (dict(flags=0), 1), (dict(eps=-0.5), 1), (dict(latent_stride=508), 1),
    (dict(latent_stride=516), 1), (dict(idx_stride=62), 1), (dict(idx_stride=65), 1), (dict(total_rows=0), 1),
    (dict(latent=None), 1), (dict(pos=None), 1), (dict(codes=None), 1), (dict(scales=None), 1), (dict(idx_k=None), 1),
    (dict(idx_kscale=None), 1), (dict(inv_freq=None), 1), (dict(idx_inv_freq=None), 1), (dict(kv_offsets=None), 1),
    (dict(page_table=FAKE, page_rows=128, pages_per_seq=1), 1),   # both ways of addressing
    (dict(kv_offsets=None, page_table=FAKE, page_rows=64, pages_per_seq=1), 1),
    (dict(kv_offsets=None, page_table=FAKE, page_rows=128, pages_per_seq=0), 1),
    (dict(seq=None, n=5), 1), (dict(latent=FAKE + 8), 1), (dict(codes=FAKE + 4), 1), (dict(workspace=FAKE + 64), 3),
])
def test_append_rope_refuses(csa2, kw, status):
    assert _append(csa2, **kw) == status


@pytest.mark.parametrize("args,status", [
    ((FAKE, FAKE, 8, None, -1, FAKE), 1), ((FAKE, FAKE, -1, None, 1, FAKE), 1), ((None, FAKE, 8, None, 8, FAKE), 1),
    ((FAKE, None, 8, None, 8, FAKE), 1), ((FAKE, FAKE, 8, None, 8, None), 1), ((FAKE, FAKE, 8, None, 9, FAKE), 1),
    ((FAKE + 4, FAKE, 8, None, 8, FAKE), 1), ((FAKE, FAKE, 8, None, 8, FAKE + 8), 1), ((FAKE, FAKE, 8, FAKE + 4, 8, FAKE), 1),
    ((FAKE, FAKE, 8, FAKE, 1 << 36, FAKE), 2),
])
def test_dequantize_refuses(csa2, args, status):
    assert csa2.lib().csa2_dequantize_kv(*args, None) == status


def _cache(csa2, **kw):
    a = csa2.CacheArgs(batch=2, q_per_seq=1, ratio=1, out_type=0, max_n=1000, total_n=2000, kv_offsets=FAKE, codes=FAKE,
                       scales=FAKE, q=FAKE, sm_scale=1.0, out=FAKE, workspace=FAKE, workspace_bytes=1 << 30)
    for k, v in kw.items():
        setattr(a, k, v)
    return csa2.lib().csa2_attend_cache(ctypes.byref(a), None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), 1), (dict(q_per_seq=0), 1), (dict(q_per_seq=65537), 1), (dict(ratio=3), 1), (dict(out_type=1), 2),
    (dict(out_type=9), 1), (dict(max_n=0), 1), (dict(max_n=1 << 31), 2), (dict(total_n=0), 1), (dict(total_n=1 << 31), 1),
    (dict(window=-1), 1), (dict(sinks=-1), 1), (dict(kv_offsets=None), 1), (dict(codes=None), 1), (dict(scales=None), 1),
    (dict(q=None), 1), (dict(out=None), 1), (dict(codes=FAKE + 8), 1), (dict(q=FAKE + 8), 1), (dict(out=FAKE + 4), 1),
    (dict(sm_scale=float("inf")), 1), (dict(sm_scale=float("nan")), 1), (dict(reserved0=2), 1),
    (dict(page_table=FAKE, page_rows=100, pages_per_seq=10), 1), (dict(page_table=FAKE, page_rows=128, pages_per_seq=7), 1),
    (dict(batch=1 << 20, q_per_seq=65536), 2), (dict(workspace=None), 3), (dict(workspace=FAKE + 128), 3),
    (dict(workspace_bytes=256), 3),
])
def test_attend_cache_refuses(csa2, kw, status):
    assert _cache(csa2, **kw) == status


def test_workspace_is_bounded_and_covers_the_call(csa2):
    def size(**kw):
        a = csa2.CacheArgs(batch=1, q_per_seq=1, ratio=1, max_n=1)
        for k, v in kw.items():
            setattr(a, k, v)
        return csa2.lib().csa2_cache_workspace_size(ctypes.byref(a))
    one = size()
    assert 256 < one < size(max_n=1500) < size(max_n=1 << 20)
    assert size(max_n=1 << 20) == size(batch=64, max_n=1 << 20) == size(batch=1000, q_per_seq=64, max_n=1 << 31 - 1)
    assert size(max_n=1 << 20, window=128, sinks=4) < size(max_n=1 << 20)
    assert size(max_n=1 << 20, window=1 << 40, sinks=1 << 40) == size(max_n=1 << 20)


def test_struct_layouts_match_the_header(csa2, tmp_path):
    from tests.test_abi_layout_cpu import _c_layout
    pairs = [("csa2_rope_args", csa2.RopeArgs), ("csa2_append_args", csa2.AppendArgs), ("csa2_cache_args", csa2.CacheArgs)]
    table = _c_layout(tmp_path, [(c, [f for f, _ in py._fields_]) for c, py in pairs])
    for cname, py in pairs:
        assert table[(cname, "size")] == ctypes.sizeof(py), cname
        for f, _ in py._fields_:
            assert table[(cname, f)] == getattr(py, f).offset, f"{cname}.{f}"


def test_binding_refuses_host_tensors(csa2):
    import torch
    x = torch.zeros(2, 16, 512, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        csa2.rope_args(x=x, out=x)
    with pytest.raises(ValueError):
        csa2.rope_args(x=x, out=x[:1])


def test_workspace_size_of_a_refused_call_is_zero(csa2):
    for kw in (dict(max_n=0), dict(max_n=(1 << 63) - 1), dict(max_n=1 << 31), dict(batch=0), dict(q_per_seq=0),
               dict(batch=(1 << 31) - 1, q_per_seq=65536), dict(window=-1), dict(sinks=-1)):
        a = csa2.CacheArgs(**{**dict(batch=1, q_per_seq=1, ratio=1, max_n=1), **kw})
        assert csa2.lib().csa2_cache_workspace_size(ctypes.byref(a)) == 0, kw


def test_norm_rope_strides_beyond_64_bits_are_seen_to_overlap_or_not(csa2):
    """(rows - 1) * stride passes 2^63: the heads would lie between the rows."""
    far = 1 << 62
    assert _rope(csa2, rows=1 << 20, heads=2, out_row_stride=far, out_head_stride=far) == 1


def test_workspace_of_a_larger_call_serves_smaller_ones(csa2):
    """The size never falls as any of the sizes grows, also where whole rows are dealt out."""
    def size(**kw):
        a = csa2.CacheArgs(**{**dict(batch=1, q_per_seq=1, ratio=1, max_n=1), **kw})
        return csa2.lib().csa2_cache_workspace_size(ctypes.byref(a))
    lengths = [1, 128, 129, 256, 384, 512, 640, 768, 896, 1000, 1024, 1025, 1280, 5000, 18944, 20000, 1 << 20]
    for window, sinks in ((0, 0), (1, 0), (128, 4), (700, 300), (4096, 4)):
        table = [[size(batch=b, max_n=n, window=window, sinks=sinks) for n in lengths] for b in range(1, 301)]
        assert all(x <= y for row in table for x, y in zip(row, row[1:]))
        assert all(x <= y for a, b in zip(table, table[1:]) for x, y in zip(a, b))
        assert [size(batch=12, q_per_seq=k, max_n=1000, window=window, sinks=sinks) for k in (1, 2, 5)] == \
            [size(batch=12 * k, max_n=1000, window=window, sinks=sinks) for k in (1, 2, 5)]
    for rows in (1, 30, 62, 64, 200):
        for n in (300, 1000, 5000):
            by_window = [size(batch=rows, max_n=n, window=w, sinks=4) for w in (1, 2, 128, 129, 500, 900, 4096, 0)]
            by_sinks = [size(batch=rows, max_n=n, window=200, sinks=s) for s in (0, 1, 128, 129, 500, 4096)]
            assert by_window == sorted(by_window) and by_sinks == sorted(by_sinks)
    assert size(batch=1 << 20, max_n=1 << 20) <= 9.8e6


def test_a_workspace_below_the_stated_size_is_refused(csa2):
    for rows in (30, 32, 62, 64):
        need = csa2.lib().csa2_cache_workspace_size(ctypes.byref(csa2.CacheArgs(batch=rows, q_per_seq=1, ratio=1, max_n=1024)))
        assert _cache(csa2, batch=rows, max_n=1024, workspace_bytes=need - 1) == 3


def test_positions_whose_last_tile_ends_past_32_bits_are_refused(csa2):
    """A tile's end is counted in 32 bits: a sequence may be that long where its pages repeat."""
    last = (1 << 31) - 128
    size = lambda n: csa2.lib().csa2_cache_workspace_size(ctypes.byref(csa2.CacheArgs(batch=1, q_per_seq=1, ratio=1, max_n=n)))  # noqa: E731
    assert size(last) == size(1 << 20) and size(last + 1) == size((1 << 31) - 1) == 0
    assert _cache(csa2, batch=1, max_n=last, workspace_bytes=256) == 3
    for n in (last + 1, (1 << 31) - 1):
        assert _cache(csa2, batch=1, max_n=n, workspace_bytes=256) == 2


@pytest.mark.parametrize("codes,scales", [((4, 128, 256), (4, 128, 32)), ((512, 256), (511, 32)), ((512, 256), (4, 128, 32)),
                                          ((512, 2, 256), (512, 32)), ((256,), (32,))])
def test_binding_refuses_a_cache_that_is_not_two_matrices(csa2, codes, scales):
    """The first dimension counts rows: of a cache given as [pages][page_rows][256] it would count
    pages, and the rows behind would be taken for missing ones."""
    import torch
    q = torch.zeros(1, 16, 512, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match=r"codes uint8 \[rows\]\[256\]"):
        csa2.cache_args(batch=1, max_n=512, kv_offsets=torch.zeros(2, dtype=torch.int64), q=q, out=q,
                        codes=torch.zeros(codes, dtype=torch.uint8), scales=torch.zeros(scales, dtype=torch.uint8))
