"""GPU: the dense-cache operators against float64 on the same inputs, with the bounds derived
here (u = half a unit in the last place of the type named)."""
import math

import numpy as np
import pytest
import torch

from oracle import csa2_oracle as O

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


@pytest.fixture(scope="module")
def csa2():
    from __graft_entry__ import build
    build()
    from fp4_kv_cache_04_b200 import csa2 as c
    return c


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def freqs(r, base=10000.0):
    return (base ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)).float().to(DEV) if r else None


def turned(y, pos, f, half=False, sign=1.0):
    """y [n][...][dim] float64, its last 2 len(f) channels turned by sign * pos * f."""
    if f is None:
        return y
    r = 2 * f.numel()
    a = sign * (pos.double().view(-1, *([1] * (y.dim() - 1))) * f.double())
    y = y.clone()
    t = y[..., -r:]
    i = torch.arange(r // 2, device=y.device)
    iu, iv = (i, i + r // 2) if half else (2 * i, 2 * i + 1)
    u, v = t[..., iu].clone(), t[..., iv].clone()
    t[..., iu] = u * a.cos() - v * a.sin()
    t[..., iv] = v * a.cos() + u * a.sin()
    return y


def normed(x, w, eps):
    y = x / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    return y if w is None else y * w.double()


def rows64(codes, scales):
    """FP4 rows as float64."""
    c = codes.long()
    v = E2M1.to(codes.device)[torch.stack([c & 15, c >> 4], -1).flatten(-2)]
    return v * scales.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)


# ------------------------------------------------------------------ norm + rotation

@pytest.mark.parametrize("rows,heads,dim,r,src,dst,half,inverse,norm,cut", [
    (1, 16, 512, 64, BF, BF, False, False, True, False),
    (65, 16, 512, 64, BF, BF, False, False, True, True),
    (33, 4, 64, 64, BF, BF, True, False, True, True),
    (7, 3, 192, 2, HF, FP, True, False, True, False),
    (129, 1, 8, 8, FP, HF, False, True, True, False),
    (5, 7, 72, 30, BF, FP, True, True, False, True),
    (40, 2, 1024, 1024, FP, FP, True, False, True, False),
    (9, 2, 1024, 600, BF, HF, False, False, True, True),
    (300, 5, 256, 0, HF, BF, False, False, True, True),
    (50, 16, 512, 64, FP, BF, False, True, False, False),
    (17, 1024, 16, 6, BF, BF, False, False, True, False),
])
def test_norm_rope(csa2, rows, heads, dim, r, src, dst, half, inverse, norm, cut):
    g = gen(rows + dim)
    wide = torch.randn(rows, heads * dim + (24 if cut else 0), generator=g, device=DEV).mul_(3).to(src)
    x = wide[:, :heads * dim].unflatten(1, (heads, dim))
    pos = torch.randint(0, 1 << 30, (rows,), generator=g, device=DEV)
    pos[0] = 0
    w = torch.rand(dim, generator=g, device=DEV) + 0.5 if norm and dim != 192 else None
    buf = torch.full((rows, heads, dim + (16 if cut else 0)), 7.0, dtype=dst, device=DEV)
    out = buf[..., :dim]
    f = freqs(r)
    csa2.norm_rope(csa2.rope_args(x=x, out=out, pos=pos if r else None, inv_freq=f, weight=w, norm=norm, eps=1e-5,
                                  inverse=inverse, half=half))
    x64 = x.double()
    y = normed(x64, w, 1e-5) if norm else x64
    want = turned(y, pos, f, half, -1.0 if inverse else 1.0)
    # fp32: the sum of squares is <= 32 + 5 additions deep (half of it reaches 1 / sqrt), a
    # division, a root and three products round: 24 u32.  cos and sin: the fraction of a turn
    # rounded (pi u32), sincospi to 2 units (4 u32), two products and a sum: 12 u32 of |u| + |v|.
    # Angles: pos * f / 2 pi in 64 bits, 3 roundings of up to 2^30 turns: 2^-22 turns = 24 u32.
    mag = y.abs().clone()
    if f is not None:
        t = mag[..., -r:]
        i = torch.arange(r // 2, device=DEV)
        iu, iv = (i, i + r // 2) if half else (2 * i, 2 * i + 1)
        both = t[..., iu] + t[..., iv]
        t[..., iu], t[..., iv] = both.clone(), both
    tol = (24 + 12 + 24) * 2.0 ** -24 * mag + torch.finfo(dst).eps / 2 * want.abs() + torch.finfo(dst).smallest_normal * torch.finfo(dst).eps
    assert ((out.double() - want).abs() <= tol).all()
    if cut:
        assert (buf[..., dim:] == 7.0).all()


def test_norm_rope_in_place_twice_is_identity_turned_back(csa2):
    x = torch.randn(20, 16, 512, generator=gen(3), device=DEV)
    keep, pos, f = x.clone(), torch.arange(20, device=DEV) * 1001, freqs(64)
    csa2.norm_rope(csa2.rope_args(x=x, out=x, pos=pos, inv_freq=f, norm=False))
    assert not torch.equal(x, keep)
    csa2.norm_rope(csa2.rope_args(x=x, out=x, pos=pos, inv_freq=f, norm=False, inverse=True))
    assert (x - keep).abs().max() <= 24 * 2.0 ** -24 * 2 * keep.abs().max()


def test_norm_rope_of_zeros_and_other_stream(csa2):
    x = torch.zeros(3, 2, 64, dtype=BF, device=DEV)
    out = torch.full_like(x, 5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    csa2.norm_rope(csa2.rope_args(x=x, out=out, norm=True, eps=1e-6), stream=s)
    s.synchronize()
    assert (out == 0).all()


# ------------------------------------------------------------------ append

def table_for(batch, pages, total_pages, seed):
    return torch.randperm(total_pages, generator=gen(seed), device=DEV)[:batch * pages].to(torch.int32).view(batch, pages)


def row_of(seq, pos, offs, table, page):
    if table is None:
        return offs[seq.long()] + pos
    return table[seq.long(), pos // page].long() * page + pos % page


def blank_cache(rows):
    return (torch.full((rows, 256), 0xAB, dtype=torch.uint8, device=DEV), torch.full((rows, 32), 0x2B, dtype=torch.uint8, device=DEV),
            torch.full((rows, 64), 0xCD, dtype=torch.uint8, device=DEV), torch.full((rows,), -3.0, device=DEV))


@pytest.mark.parametrize("src,r,ri,half,norm,paged,idx,cut", [
    (BF, 64, 64, False, True, True, True, True),
    (BF, 64, 32, True, True, False, True, False),
    (HF, 2, 6, True, True, True, True, True),
    (FP, 512, 0, False, True, False, True, True),
    (FP, 512, 64, True, True, True, False, False),
    (BF, 130, 2, False, False, True, True, False),
    (BF, 0, 0, False, False, False, True, True),
])
def test_append_rope_rows_are_exact(csa2, src, r, ri, half, norm, paged, idx, cut):
    g = gen(r + ri)
    batch, n = 5, 83
    lens = torch.tensor([300, 1, 777, 130, 257])
    page = 128
    offs = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)]).to(DEV)
    table = table_for(batch, 7, 40, 1) if paged else None
    total = 40 * page if paged else int(lens.sum())
    seq = torch.randint(0, batch, (n,), generator=g, device=DEV).to(torch.int32)
    seq[seq == 1] = 2
    pos = torch.empty(n, dtype=torch.int64, device=DEV)
    for b in range(batch):                                  # distinct positions of each sequence
        m = seq == b
        pos[m] = torch.randperm(int(lens[b]), generator=g, device=DEV)[:int(m.sum())]
    pos[5], pos[50] = -1, -7                                # padding
    lat = torch.randn(n, 512 + (40 if cut else 0), generator=g, device=DEV) * torch.exp(torch.randn(n, 1, generator=g, device=DEV) * 2)
    lat = lat.to(src)[:, :512]
    proj = (torch.randn(n, 64 + (6 if cut else 0), generator=g, device=DEV))[:, :64] if idx else None
    if idx:
        proj[7] = 0
    w = torch.rand(512, generator=g, device=DEV) + 0.5 if norm else None
    codes, scales, ik, iks = blank_cache(total)
    f, fi = freqs(r), freqs(ri) if idx else None
    ws = csa2.alloc_workspace(256)
    csa2.append_rope(csa2.append_args(
        latent=lat, pos=pos, seq=seq, codes=codes, scales=scales, kv_offsets=None if paged else offs, page_table=table,
        page_rows=page if paged else 0, weight=w, norm=norm, eps=1e-6, inv_freq=f, half=half, idx_proj=proj, idx_inv_freq=fi,
        idx_k=ik if idx else None, idx_kscale=iks if idx else None, workspace=ws))
    assert csa2.check_device_status(ws) == 0
    live = pos >= 0
    y = lat.double()
    y = turned(normed(y, w, float(np.float32(1e-6))) if norm else y, pos, f, half)[live]
    oc, os_ = O.quantize_rows(O.f64_to_bf16(y.cpu().numpy()))
    rows = row_of(seq, pos, offs, table, page)[live]
    want = blank_cache(total)
    want[0][rows], want[1][rows] = torch.from_numpy(oc).to(DEV), torch.from_numpy(os_).to(DEV)
    assert torch.equal(scales, want[1]) and torch.equal(codes, want[0])    # and every other row as it was
    if not idx:
        assert torch.equal(ik, want[2]) and torch.equal(iks, want[3])
        return
    k = turned(proj.double(), pos, fi, half)[live]
    ks = k.abs().amax(-1) / 448
    got_s, got_k = iks[rows].double(), ik[rows].view(torch.float8_e4m3fn).double()
    # fp32 rotation and division: 12 + 24 u32 as above, of |u| + |v| <= 2 * amax
    assert ((got_s - ks).abs() <= 80 * 2.0 ** -24 * ks).all()
    step = torch.where(got_k.abs() < 2 ** -6, torch.full_like(got_k, 2.0 ** -10), got_k.abs() * 2.0 ** -4)   # half a step of E4M3
    assert ((got_k * ks[:, None] - k).abs() <= (step + 1e-4 * 448) * ks[:, None] + 1e-30).all()
    iks[rows], ik[rows] = want[3][rows], want[2][rows]
    assert torch.equal(ik, want[2]) and torch.equal(iks, want[3])


@pytest.mark.parametrize("ri,half", [(64, False), (64, True), (32, False), (6, True), (30, True)])
def test_append_rope_indexer_rows_are_exact(csa2, ri, half):
    """The real rotation rounded once to fp32, then the plain append's scale and codes: equal, over
    half a million values."""
    n = 8192
    g = gen(50 + ri)
    lat = torch.zeros(n, 512, dtype=BF, device=DEV)
    proj = torch.randn(n, 64, generator=g, device=DEV)
    pos = torch.randperm(1 << 17, generator=g, device=DEV)[:n]
    seq, offs = torch.zeros(n, dtype=torch.int32, device=DEV), torch.tensor([0, 1 << 17], device=DEV)
    codes, scales, ik, iks = blank_cache(1 << 17)
    csa2.append_rope(csa2.append_args(latent=lat, pos=pos, seq=seq, codes=codes, scales=scales, kv_offsets=offs, norm=False,
                                      half=half, idx_proj=proj, idx_inv_freq=freqs(ri), idx_k=ik, idx_kscale=iks))
    k = turned(proj.double(), pos, freqs(ri), half).float().cpu().numpy()
    ks = np.abs(k).max(-1) / np.float32(448)
    assert ks.dtype == np.float32 and np.array_equal(iks[pos].cpu().numpy(), ks)
    want = torch.from_numpy(k / ks[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(ik[pos].cpu(), want)


def test_append_rope_is_append_kv_without_norm_and_rotation(csa2):
    n = 70
    lat = torch.randn(n, 512, generator=gen(5), device=DEV).to(BF)
    proj = torch.randn(n, 64, generator=gen(6), device=DEV)
    rows = torch.randperm(200, generator=gen(7), device=DEV)[:n]
    a, b = blank_cache(200), blank_cache(200)
    csa2.append_kv(lat, proj, rows, *a)
    offs = torch.tensor([0, 200], device=DEV)
    csa2.append_rope(csa2.append_args(latent=lat, pos=rows, seq=torch.zeros(n, dtype=torch.int32, device=DEV), codes=b[0],
                                      scales=b[1], kv_offsets=offs, norm=False, idx_proj=proj, idx_k=b[2], idx_kscale=b[3]))
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_append_rope_rounds_like_the_quantiser_everywhere(csa2):
    """Rows of every bf16 value beside scales of every size: ties, saturation, subnormal and zero
    scales, signs of zero."""
    bits = torch.arange(1 << 16, dtype=torch.int32, device=DEV).to(torch.int16).view(BF)
    bits = bits[bits.isfinite()]
    bits = torch.cat([bits, bits[: (-bits.numel()) % 512]])
    rows = [bits.view(-1, 512)]
    tops = 2.0 ** torch.arange(-12, 12, device=DEV).double()[:, None] * (1 + torch.arange(0, 128, device=DEV).double() / 128)[None]
    half = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, 0.0], device=DEV).double()
    t = tops.reshape(-1)
    s = (t / 6).float().clamp(max=448).to(torch.float8_e4m3fn).double()
    rows.append(torch.cat([t[:, None], half * s[:, None]], 1).to(BF).view(-1, 512))
    x = torch.cat(rows)
    n = x.shape[0]
    a, b = blank_cache(n), blank_cache(n)
    csa2.quantize_kv(x, 1, a[0], a[1])
    csa2.append_rope(csa2.append_args(latent=x, pos=torch.arange(n, device=DEV), seq=torch.zeros(n, dtype=torch.int32, device=DEV),
                                      codes=b[0], scales=b[1], kv_offsets=torch.tensor([0, n], device=DEV), norm=False))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_append_not_finite_values_keep_the_quantiser_s_codes(csa2):
    """Infinities and NaN: the FP4 row of append_kv; indexer codes of 448 (126) with the value's sign,
    NaN counting as positive, against the largest of the others."""
    inf, nan = math.inf, math.nan
    x = torch.randn(6, 512, generator=gen(40), device=DEV).to(BF)
    x[0, 3], x[1, 20], x[2, 37], x[3, :16], x[4, 500:], x[5, 64] = inf, -inf, nan, nan, -nan, 3e38
    proj = torch.full((6, 64), 1.0, device=DEV)
    proj[0, 3], proj[1, 4], proj[2, 5], proj[3, 6:8], proj[4, :] = nan, inf, -inf, torch.tensor([448.0, -1e-9], device=DEV), nan
    want = torch.full((6, 64), 126, dtype=torch.uint8)         # 1 / (1 / 448) = 448
    want[1:3] = 0                                              # 1 / inf = 0
    want[1, 4], want[2, 5] = 126, 126                          # inf / inf = NaN
    want[3], want[3, 6], want[3, 7] = 0x38, 126, 0x80          # 1.0, 448, -0
    want[4] = 0                                                # nothing but NaN: so is the scale
    caches = [blank_cache(6) for _ in range(2)]
    offs, pos = torch.arange(7, device=DEV), torch.zeros(6, dtype=torch.int64, device=DEV)
    c, s, ik, iks = caches[0]
    csa2.append_kv(x, proj, offs[:6].contiguous(), c, s, ik, iks)
    c2, s2, ik2, iks2 = caches[1]
    csa2.append_rope(csa2.append_args(latent=x, pos=pos, codes=c2, scales=s2, kv_offsets=offs, norm=False, idx_proj=proj,
                                      idx_k=ik2, idx_kscale=iks2))
    for a, b in zip(*caches):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert torch.equal(ik.cpu(), want)
    assert iks.tolist()[0] == np.float32(1) / np.float32(448) and iks.tolist()[1:3] == [inf, inf] and iks[4].isnan()


@pytest.mark.parametrize("gain,wgain", [(1e-25, 1.0), (1e37, 1.0), (1e-18, 1e25), (1e18, 1e-20), (1.0, 1e30)])
def test_append_rope_far_magnitudes(csa2, gain, wgain):
    """fp32 latents whose squares, or whose weights times 1 / rms, leave the range of fp32."""
    x = torch.randn(9, 512, generator=gen(41), device=DEV) * gain
    w = (torch.rand(512, generator=gen(42), device=DEV) + 0.5) * wgain
    pos, offs, f = torch.zeros(9, dtype=torch.int64, device=DEV), torch.arange(10, device=DEV), freqs(64)
    c, s, _, _ = blank_cache(9)
    csa2.append_rope(csa2.append_args(latent=x, pos=pos, codes=c, scales=s, kv_offsets=offs, weight=w, eps=0.0, inv_freq=f))
    y = turned(normed(x.double(), w, 0.0), pos, f)
    wc, ws = O.quantize_rows(O.f64_to_bf16(y.cpu().numpy()))
    assert np.array_equal(c.cpu().numpy(), wc) and np.array_equal(s.cpu().numpy(), ws)


def test_append_rope_skips_and_reports_what_lies_outside(csa2):
    lat = torch.randn(6, 512, generator=gen(8), device=DEV).to(BF)
    table = torch.tensor([[0, 1], [2, 9], [-1, 3]], dtype=torch.int32, device=DEV)     # page 9 of 4, page -1
    codes, scales, _, _ = blank_cache(4 * 128)
    ws = csa2.alloc_workspace(256)
    want = codes.clone()
    seq = torch.tensor([1, 2, 3, -1, 0, 0], dtype=torch.int32, device=DEV)
    pos = torch.tensor([128, 0, 0, 0, 256, 3], device=DEV)
    csa2.append_rope(csa2.append_args(latent=lat, pos=pos, seq=seq, codes=codes, scales=scales, page_table=table, page_rows=128,
                                      norm=False, workspace=ws))
    assert csa2.check_device_status(ws) == 6 and csa2.check_device_status(ws) == 0
    c5, _ = O.quantize_rows(lat[5:].cpu().view(torch.int16).numpy().view(np.uint16))
    want[3] = torch.from_numpy(c5[0]).to(DEV)
    assert torch.equal(codes, want)
    offs = torch.tensor([0, 100, 90, 700], device=DEV)                                  # a negative length; rows past the cache
    codes, scales, _, _ = blank_cache(4 * 128)
    want = codes.clone()
    csa2.append_rope(csa2.append_args(latent=lat[:3], pos=torch.tensor([100, 0, 600], device=DEV), codes=codes, scales=scales,
                                      kv_offsets=offs, norm=False, workspace=ws))
    assert csa2.check_device_status(ws) == 6 and torch.equal(codes, want)


# ------------------------------------------------------------------ read-back

def test_dequantize_is_exact_for_every_code_and_scale(csa2):
    scales = torch.arange(0, 127, device=DEV).to(torch.uint8).repeat_interleave(32).view(-1, 32).contiguous()
    codes = torch.arange(256, device=DEV).to(torch.uint8).repeat(127, 1).contiguous()
    out = torch.empty(127, 512, dtype=BF, device=DEV)
    csa2.dequantize_kv(codes, scales, out)
    assert torch.equal(out.double(), rows64(codes, scales))


@pytest.mark.parametrize("n", [1, 3, 4, 33, 1000])
def test_dequantize_gathers_and_zeroes_padding(csa2, n):
    g = gen(n)
    codes = torch.randint(0, 256, (500, 256), generator=g, device=DEV).to(torch.uint8)
    scales = torch.randint(0, 126, (500, 32), generator=g, device=DEV).to(torch.uint8)
    rows = torch.randint(-1, 501, (n,), generator=g, device=DEV)
    buf = torch.full((n + 1, 512), 9.0, dtype=BF, device=DEV)
    csa2.dequantize_kv(codes, scales, buf[:n], src_row=rows)
    ok = (rows >= 0) & (rows < 500)
    want = rows64(codes, scales)[rows.clamp(0, 499)] * ok[:, None]
    assert torch.equal(buf[:n].double(), want) and (buf[n] == 9.0).all()


# ------------------------------------------------------------------ attention

def make_cache(rows, seed, spread=1.0):
    """Codes and scales as the quantiser writes them for N(0, spread) rows."""
    x = torch.randn(rows, 512, generator=gen(seed), device=DEV) * spread
    x[:, ::64] *= 4
    s = (x.view(rows, 32, 16).abs().amax(-1) / 6).to(torch.float8_e4m3fn)
    y = x.view(rows, 32, 16).abs() / s.float().unsqueeze(-1).clamp(min=1e-9)
    mag = sum((y > t).to(torch.uint8) for t in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)).view(rows, 256, 2)
    code = mag + (x < 0).view(rows, 256, 2) * 8
    return (code[..., 0] + 16 * code[..., 1]).to(torch.uint8).contiguous(), s.view(torch.uint8).contiguous()


def seen_positions(n, t, ratio, window, sinks):
    vis = n if t is None else max(0, min(n, (t + 1) // ratio))
    p = torch.arange(vis, device=DEV)
    return p if not window else p[(p < sinks) | (p >= vis - window)]


def check_attend(csa2, lens, window=0, sinks=0, q_per_seq=1, q_pos=None, ratio=1, page=0, out_type=BF, seed=0, sm_scale=None,
                 q_gain=2.0, spread=1.0, max_n=None, spoil=False, want_lse=True, stream=None, cache=None, graph=False, every=1):
    B = len(lens)
    lens_t = torch.tensor(lens)
    offs = torch.cat([torch.zeros(1, dtype=torch.int64), lens_t.cumsum(0)]).to(DEV)
    max_n = max_n or max(1, max(lens))
    if page:
        pages = -(-max_n // page)
        table = table_for(B, pages, B * pages + 3, seed + 1)
        total = (B * pages + 3) * page
    else:
        table, total = None, max(1, sum(lens))
    codes, scales = cache or make_cache(total, seed, spread)
    if spoil:                                     # every row that no query sees: NaN scales, any codes
        used = torch.zeros(total, dtype=torch.bool, device=DEV)
        for b in range(B):
            for i in range(q_per_seq):
                p = seen_positions(lens[b], None if q_pos is None else q_pos[b] + i, ratio, window, sinks)
                used[row_of(torch.full_like(p, b), p, offs, table, page)] = True
        codes[~used], scales[~used] = 0x77, 0x7F
    R = B * q_per_seq
    q = (torch.randn(R, 16, 512, generator=gen(seed + 2), device=DEV) * q_gain).to(BF)
    out = torch.full((R + 1, 16, 512), 3.0, dtype=out_type, device=DEV)
    lse = torch.full((R + 1, 16), 3.0, device=DEV) if want_lse else None
    sm_scale = 1 / math.sqrt(512) if sm_scale is None else sm_scale
    kw = dict(batch=B, q_per_seq=q_per_seq, max_n=max_n, kv_offsets=offs, codes=codes, scales=scales, q=q, out=out[:R],
              q_pos=None if q_pos is None else torch.tensor(q_pos, device=DEV), ratio=ratio, window=window, sinks=sinks,
              sm_scale=sm_scale, lse=lse[:R] if want_lse else None, page_table=table, page_rows=page)
    ws = csa2.alloc_workspace(csa2.cache_workspace_size(csa2.cache_args(**kw)))
    a = csa2.cache_args(workspace=ws, **kw)
    if graph:
        csa2.attend_cache(a)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            csa2.attend_cache(a)
        out.fill_(3.0)
        for _ in range(3):
            gr.replay()
    else:
        csa2.attend_cache(a, stream=stream)
    torch.cuda.synchronize()
    assert csa2.check_device_status(ws) == 0
    assert (out[R] == 3.0).all()
    worst = 0.0
    for r in range(0, R, every):
        b, i = divmod(r, q_per_seq)
        p = seen_positions(lens[b], None if q_pos is None else q_pos[b] + i, ratio, window, sinks)
        if not p.numel():
            assert (out[r] == 0).all() and (lse is None or (lse[r] == -math.inf).all())
            continue
        rows = row_of(torch.full_like(p, b), p, offs, table, page)
        kv = rows64(codes[rows], scales[rows])
        q64 = q[r].double()
        s = q64 @ kv.T * sm_scale
        w = torch.softmax(s, -1)
        want, mag = w @ kv, w @ kv.abs()
        # the query's fixed point is off by half of 2^-15 of the head's largest element at
        # most; the products' fp32 sum by 640 u32 of their magnitudes' sum; 2^-20 for exp2
        qmax = q64.abs().amax(-1, keepdim=True)
        ds = abs(sm_scale) * (2.0 ** -16 * qmax * kv.abs().sum(-1) + 640 * 2.0 ** -24 * (q64.abs() @ kv.abs().T)).amax(-1, keepdim=True)
        rel = 2 * ds + 2.0 ** -20
        n_add = 2.0 ** -23 * (p.numel() / 16 + 32)             # P V adds 16 positions per step
        # P is kept in f16 times 2^11 against a reference that the true maximum never lies below:
        # below 2^-14 f16 rounds by up to 2^-25, which is 2^-36 of the largest weight for each key
        tol = (rel + 2.0 ** -11 + n_add) * mag + 2.0 ** -36 * kv.abs().sum(0) + torch.finfo(out_type).eps / 2 * want.abs() * 1.01 + 1e-30
        err = (out[r].double() - want).abs()
        worst = max(worst, float((err / tol).max()))
        assert (err <= tol).all(), f"row {r}: {float((err / tol).max())} of the bound"
        if lse is not None:
            le = torch.logsumexp(s, -1)
            assert ((lse[r].double() - le).abs() <= ds[:, 0] + n_add + 2.0 ** -20 + 2.0 ** -22 * le.abs()).all()
    return out, worst


@pytest.mark.parametrize("lens", [[1], [2], [127], [128], [129], [300, 1, 0, 128], [1501], [0], [0, 0, 5]])
@pytest.mark.parametrize("page", [0, 128])
def test_attend_cache_lengths(csa2, lens, page):
    check_attend(csa2, lens, page=page)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (128, 0), (128, 4), (100, 130), (129, 1), (1000, 4), (64, 10000),
                                          (1 << 40, 1 << 40)])
def test_attend_cache_window_and_first_positions(csa2, window, sinks):
    check_attend(csa2, [700, 90, 1, 128, 129, 2000, 0], window=window, sinks=sinks, page=256, spoil=True, seed=window % 97)


@pytest.mark.parametrize("ratio", [1, 2])
@pytest.mark.parametrize("window,sinks", [(0, 0), (130, 5)])
def test_attend_cache_drafted_tokens(csa2, ratio, window, sinks):
    # the first queries of sequence 0 see little or nothing; those of sequence 1 end on the last row
    check_attend(csa2, [300, 260, 17, 0], window=window, sinks=sinks, q_per_seq=5, ratio=ratio,
                 q_pos=[0, 260 * ratio - 5, 1000, 3], spoil=True, out_type=FP)


def test_attend_cache_masked_tail_holds_nan(csa2):
    check_attend(csa2, [200, 65, 129], page=128, spoil=True)


def test_attend_cache_many_rows(csa2):
    check_attend(csa2, [(37 * i) % 400 for i in range(600)], window=200, sinks=3, seed=9)


def test_attend_cache_many_empty_rows_and_one_long(csa2):
    check_attend(csa2, [0] * 700 + [5000] + [0] * 300 + [1], seed=10)


@pytest.mark.parametrize("long", [0, 1000])
def test_attend_cache_more_rows_in_a_range_than_its_table_holds(csa2, long):
    """12,000 rows of 0 to 4 positions: over 60 that see anything for each of 148 ranges, uncut, and
    (with one longer row among them) cut."""
    lens = [i % 5 for i in range(12000)]
    if long:
        lens[7001] = long
    check_attend(csa2, lens, seed=11, every=7)


def test_attend_cache_gives_up_in_order_and_recovers(csa2):
    """With a bound of one poll the kernel's waits run out: the call ends with the timeout flag, and
    the same workspace serves the next call."""
    codes, scales = make_cache(6000, 31)
    offs = torch.tensor([0, 5000, 5003, 5003, 6000], device=DEV)
    q = torch.randn(4, 16, 512, generator=gen(32), device=DEV).to(BF)
    outs = [torch.empty(4, 16, 512, device=DEV) for _ in range(2)]
    kw = dict(batch=4, max_n=5000, kv_offsets=offs, codes=codes, scales=scales, q=q, sm_scale=512 ** -0.5)
    ws = csa2.alloc_workspace(csa2.cache_workspace_size(csa2.cache_args(out=outs[0], **kw)))
    csa2.attend_cache(csa2.cache_args(out=outs[0], workspace=ws, **kw))
    assert csa2.check_device_status(ws) == 0
    csa2.set_wait_limit(ws, 1)
    csa2.attend_cache(csa2.cache_args(out=outs[1], workspace=ws, **kw))
    assert csa2.check_device_status(ws) == 5
    csa2.set_wait_limit(ws, 0)
    csa2.attend_cache(csa2.cache_args(out=outs[1], workspace=ws, **kw))
    assert csa2.check_device_status(ws) == 0
    assert torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("gain,spread", [(0.01, 1.0), (20.0, 1.0), (2.0, 60.0), (1e-30, 1.0), (0.0, 1.0), (2.0, 0.004)])
def test_attend_cache_magnitudes(csa2, gain, spread):
    check_attend(csa2, [500, 3], q_gain=gain, spread=spread, out_type=FP)


def test_attend_cache_growing_logits(csa2):
    """Every tile holds a larger logit than the tiles before it: the running maximum moves."""
    n = 1024
    codes, scales = make_cache(n, 12)
    q = (torch.randn(1, 16, 512, generator=gen(2), device=DEV) * 2).to(BF)    # check_attend's own query (seed 0)
    kv = rows64(codes, scales)
    order = torch.argsort(kv @ q[0, 3].double())
    check_attend(csa2, [n], cache=(codes[order].contiguous(), scales[order].contiguous()), sm_scale=1.0, out_type=FP)


def test_attend_cache_negative_scale_and_no_lse(csa2):
    check_attend(csa2, [333], sm_scale=-0.03, want_lse=False)


def test_attend_cache_long_row(csa2):
    check_attend(csa2, [70001, 5], out_type=FP)


def test_attend_cache_max_n_above_the_lengths(csa2):
    check_attend(csa2, [100, 40], max_n=100000, page=512)


def test_attend_cache_other_stream_and_repeat(csa2):
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    a, _ = check_attend(csa2, [900, 31, 5000], stream=s, seed=4)
    b, _ = check_attend(csa2, [900, 31, 5000], seed=4)
    assert torch.equal(a, b)


def test_attend_cache_captured_and_replayed(csa2):
    a, _ = check_attend(csa2, [900, 31, 5000], graph=True, seed=4)
    b, _ = check_attend(csa2, [900, 31, 5000], seed=4)
    assert torch.equal(a, b)


def test_attend_cache_bad_page_is_reported(csa2):
    codes, scales = make_cache(4 * 128, 1)
    offs = torch.tensor([0, 300, 600], device=DEV)
    q = torch.randn(2, 16, 512, generator=gen(1), device=DEV).to(BF)
    out = torch.empty(2, 16, 512, dtype=BF, device=DEV)
    for bad in (4, -1, 1 << 30, -(1 << 31)):
        table = torch.tensor([[0, bad, 1], [2, 3, 0]], dtype=torch.int32, device=DEV)
        kw = dict(batch=2, max_n=300, kv_offsets=offs, codes=codes, scales=scales, q=q, out=out, page_table=table, page_rows=128)
        ws = csa2.alloc_workspace(csa2.cache_workspace_size(csa2.cache_args(**kw)))
        csa2.attend_cache(csa2.cache_args(workspace=ws, **kw))
        assert csa2.check_device_status(ws) == 6
        kv = rows64(codes, scales)[torch.arange(300, device=DEV) % 128 + torch.tensor([2, 3, 0], device=DEV)[torch.arange(300, device=DEV) // 128] * 128]
        w = torch.softmax(q[1].double() @ kv.T, -1) @ kv          # the other sequence is untouched by it
        assert (out[1].double() - w).norm() <= 4e-3 * w.norm()


def test_attend_cache_rows_behind_the_packed_cache_are_reported(csa2):
    """Offsets that reach past the last row, by whole tiles or inside one."""
    codes, scales = make_cache(300, 1)
    q = torch.randn(2, 16, 512, generator=gen(1), device=DEV).to(BF)
    out = torch.empty(2, 16, 512, dtype=BF, device=DEV)
    for last, status in ((300, 0), (301, 6), (384, 6), (700, 6)):
        offs = torch.tensor([0, 100, last], device=DEV)
        kw = dict(batch=2, max_n=600, kv_offsets=offs, codes=codes, scales=scales, q=q, out=out)
        ws = csa2.alloc_workspace(csa2.cache_workspace_size(csa2.cache_args(**kw)))
        csa2.attend_cache(csa2.cache_args(workspace=ws, **kw))
        assert csa2.check_device_status(ws) == status
        kv = rows64(codes, scales)[:100]
        w = torch.softmax(q[0].double() @ kv.T, -1) @ kv          # the other sequence is untouched by it
        assert (out[0].double() - w).norm() <= 4e-3 * w.norm()


def test_attend_cache_query_position_without_end(csa2):
    check_attend(csa2, [300, 20], q_per_seq=2, q_pos=[(1 << 63) - 1, -(1 << 63)], ratio=2)


@pytest.mark.parametrize("n", [50, 5000])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_attend_cache_not_finite_query_stays_in_its_head(csa2, n, bad):
    codes, scales = make_cache(n, 3)
    q = torch.randn(1, 16, 512, generator=gen(4), device=DEV).to(BF)
    outs = []
    for value in (1.0, bad):
        q[0, 5, 77] = value
        out, lse = torch.empty(1, 16, 512, dtype=BF, device=DEV), torch.empty(1, 16, device=DEV)
        kw = dict(batch=1, max_n=n, kv_offsets=torch.tensor([0, n], device=DEV), codes=codes, scales=scales, q=q, out=out,
                  lse=lse, sm_scale=512 ** -0.5)
        ws = csa2.alloc_workspace(csa2.cache_workspace_size(csa2.cache_args(**kw)))
        csa2.attend_cache(csa2.cache_args(workspace=ws, **kw))
        assert csa2.check_device_status(ws) == 0
        outs.append((out, lse))
    assert outs[1][0][0, 5].isnan().all() and outs[1][1][0, 5].isnan()
    rest = [h for h in range(16) if h != 5]
    assert torch.equal(outs[0][0][:, rest], outs[1][0][:, rest]) and torch.equal(outs[0][1][:, rest], outs[1][1][:, rest])


def test_attend_cache_two_calls_at_once(csa2):
    """Two streams, each with its own workspace and output."""
    alone = check_attend(csa2, [4000, 31, 900], seed=6)[0]
    codes, scales = make_cache(4931, 6)
    offs = torch.tensor([0, 4000, 4031, 4931], device=DEV)
    q = (torch.randn(3, 16, 512, generator=gen(8), device=DEV) * 2).to(BF)
    jobs = []
    for _ in range(2):
        out = torch.zeros(4, 16, 512, dtype=BF, device=DEV)
        kw = dict(batch=3, max_n=4000, kv_offsets=offs, codes=codes, scales=scales, q=q, out=out[:3], sm_scale=512 ** -0.5)
        ws = csa2.alloc_workspace(csa2.cache_workspace_size(csa2.cache_args(**kw)))
        jobs.append((torch.cuda.Stream(), csa2.cache_args(workspace=ws, **kw), out))
    torch.cuda.synchronize()
    for _ in range(20):
        for s, a, _ in jobs:
            csa2.attend_cache(a, stream=s)
    torch.cuda.synchronize()
    for _, _, out in jobs:
        assert torch.equal(out[:3], alone[:3])


def test_argument_blocks_let_their_tensors_go(csa2):
    """A block that is dropped frees what it points at, without waiting for the cycle collector."""
    import gc
    gc.collect()
    gc.disable()
    try:
        x = torch.zeros(1, 16, 512, dtype=BF, device=DEV)
        before = torch.cuda.memory_allocated()
        for _ in range(3):
            csa2.norm_rope(csa2.rope_args(x=x, out=torch.empty_like(x)))
        assert torch.cuda.memory_allocated() == before
    finally:
        gc.enable()


# ------------------------------------------------------------------ together

def test_one_decode_step_of_a_dense_layer(csa2):
    """Three steps of a layer: the new token's latent goes into the paged cache normed and
    rotated, its query is normed and rotated, attends over the cache, and the output's rotated
    channels are turned back."""
    g = gen(77)
    B, page, start, r = 3, 128, [126, 0, 511], 64
    table = table_for(B, 5, 20, 3)
    codes, scales, _, _ = blank_cache(20 * page)
    wq, wk, f = torch.rand(512, generator=g, device=DEV) + 0.5, torch.rand(512, generator=g, device=DEV) + 0.5, freqs(r)
    history = [[] for _ in range(B)]
    q, out = torch.empty(B, 16, 512, dtype=BF, device=DEV), torch.empty(B, 16, 512, device=DEV)
    back = torch.empty(B, 16, 512, dtype=BF, device=DEV)

    def append(b, pos, lat):
        csa2.append_rope(csa2.append_args(latent=lat, pos=pos, seq=torch.full((len(pos),), b, dtype=torch.int32, device=DEV),
                                          codes=codes, scales=scales, page_table=table, page_rows=page, weight=wk, inv_freq=f))
        y = turned(normed(lat.double(), wk, float(np.float32(1e-6))), pos, f)
        c, s = O.quantize_rows(O.f64_to_bf16(y.cpu().numpy()))
        history[b].append(rows64(torch.from_numpy(c).to(DEV), torch.from_numpy(s).to(DEV)))

    for b in range(B):
        if start[b]:
            append(b, torch.arange(start[b], device=DEV), torch.randn(start[b], 512, generator=g, device=DEV).to(BF))
    for step in range(3):
        n = torch.tensor([s + step + 1 for s in start], device=DEV)
        offs = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), n.cumsum(0)])
        proj = torch.randn(B, 16 * 512 + 512, generator=g, device=DEV).to(BF)      # one projection: queries, latent
        x, lat = proj[:, :8192].unflatten(1, (16, 512)), proj[:, 8192:]
        csa2.append_rope(csa2.append_args(latent=lat, pos=n - 1, codes=codes, scales=scales, page_table=table, page_rows=page,
                                          weight=wk, inv_freq=f))
        csa2.norm_rope(csa2.rope_args(x=x, out=q, pos=n - 1, inv_freq=f, weight=wq))
        kw = dict(batch=B, max_n=600, kv_offsets=offs, codes=codes, scales=scales, q=q, out=out, sm_scale=512 ** -0.5,
                  page_table=table, page_rows=page)
        ws = csa2.alloc_workspace(csa2.cache_workspace_size(csa2.cache_args(**kw)))
        csa2.attend_cache(csa2.cache_args(workspace=ws, **kw))
        csa2.norm_rope(csa2.rope_args(x=out, out=back, pos=n - 1, inv_freq=f, norm=False, inverse=True))
        y = turned(normed(lat.double(), wk, float(np.float32(1e-6))), n - 1, f)
        c, s = O.quantize_rows(O.f64_to_bf16(y.cpu().numpy()))
        y = rows64(torch.from_numpy(c).to(DEV), torch.from_numpy(s).to(DEV))
        qe = turned(normed(x.double(), wq, 1e-6), n - 1, f)
        for b in range(B):
            history[b].append(y[b:b + 1])
            kv = torch.cat(history[b])
            want = turned((torch.softmax(qe[b] @ kv.T * 512 ** -0.5, -1) @ kv)[None], (n - 1)[b:b + 1], f, sign=-1.0)[0]
            # bf16 queries move each logit by u_bf16 of its terms' root sum of squares, about
            # 2^-9 * |q||k| / sqrt(512) <= 0.05 at these sizes; then one bf16 rounding
            rel = (back[b].double() - want).norm() / want.norm()
            assert rel <= 2.0 ** -8 + 0.05
        got = torch.empty(B, 512, dtype=BF, device=DEV)
        csa2.dequantize_kv(codes, scales, got, src_row=row_of(torch.arange(B, device=DEV), n - 1, None, table, page))
        assert torch.equal(got.double(), y)


def test_a_layer_may_attend_over_selected_and_all_positions(csa2):
    """With at most 512 positions the Top-512 selection is the whole context: csa2_attend's main
    rows and attend_cache agree once the window's part is joined through the lse."""
    n, B = 400, 2
    codes, scales = make_cache(B * n, 21)
    offs = torch.tensor([0, n, 2 * n], device=DEV)
    q = torch.randn(B, 16, 512, generator=gen(22), device=DEV).to(BF)
    swa = torch.randn(B, 128, 512, generator=gen(23), device=DEV).to(BF)
    topk = torch.full((B, 512), -1, dtype=torch.int32, device=DEV)
    topk[:, :n] = torch.arange(n, device=DEV)
    both = torch.empty(B, 16, 512, device=DEV)
    kw = dict(mode=csa2.MODE_REUSE, batch=B, q_per_seq=1, max_n=n, kv_offsets=offs, codes=codes, scales=scales, topk_idx=topk,
              q=q, swa_kv=swa, out=both, sm_scale=512 ** -0.5)
    csa2.attend(csa2.layer_args(workspace=csa2.alloc_workspace(csa2.workspace_size(csa2.layer_args(**kw))), **kw))
    main, lse = torch.empty(B, 16, 512, device=DEV), torch.empty(B, 16, device=DEV)
    kw = dict(batch=B, max_n=n, kv_offsets=offs, codes=codes, scales=scales, q=q, out=main, lse=lse, sm_scale=512 ** -0.5)
    csa2.attend_cache(csa2.cache_args(workspace=csa2.alloc_workspace(csa2.cache_workspace_size(csa2.cache_args(**kw))), **kw))
    s = torch.einsum("bhd,bjd->bhj", q.double(), swa.double()) * 512 ** -0.5
    ls = torch.logsumexp(s, -1)
    w = torch.softmax(s, -1) @ swa.double()
    a = torch.sigmoid(lse.double() - ls)[..., None]
    joined = main.double() * a + w * (1 - a)
    assert (joined - both.double()).norm() <= 1e-3 * both.double().norm()      # csa2_attend's own bound
